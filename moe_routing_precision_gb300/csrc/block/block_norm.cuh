// block_norm.cuh -- what the norms' forward and backward kernels share: the row
// sums, the gate, and the ring of staged rows.
#pragma once

#include "block/block_ops.cuh"

namespace moe {
namespace {

// Sums of N values over the threads of each row group (TPR threads, a multiple
// of 32), known to all of them on return.  buf: N * warps floats of shared
// memory that no thread still reads.  Whole-block barriers: every thread of
// the block calls it the same number of times.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* buf, int wpr, int row_in_block) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (wpr == 1) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) buf[warp * N + i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    // at most 32 warps per row: one value per lane
    const float p = lane < wpr ? buf[(row_in_block * wpr + lane) * N + i] : 0.0f;
    v[i] = warp_sum(p);
  }
}

// The gate's values from what is stored, and for the backward their derivatives.
template <int VEC>
__device__ __forceinline__ void gate_values(const NormArgs& a, float (&g)[VEC]) {
  if (a.gate_act == MOE_GATE_ACT_SIGMOID) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) g[i] = sigmoid_f32(g[i]);
  }
}
template <int VEC>
__device__ __forceinline__ void gate_values(const NormArgs& a, float (&g)[VEC], float (&g1)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) g1[i] = 1.0f;
  if (a.gate_act == MOE_GATE_ACT_SIGMOID) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) g[i] = sigmoid_f32(g[i], &g1[i]);
  }
}

// ---------------------------------------------------------------- the ring
// For H <= kRingMaxHidden and 16-byte aligned tensors: each block takes the rows
// congruent to its index, and one thread copies whole rows ahead of their use
// into a ring in shared memory (bulk copies counted by one barrier per stage),
// so that the loads never wait for a row's sums.  Every thread keeps the same
// channels for all rows (U units of V), so what depends on the channel alone
// (weights, per-channel gate, the gradients' sums) stays in its registers.
//
// V = 8: rows of whole 16-byte pieces (H % 8 == 0).  V = 1: any H.  A row then
// starts and ends inside 16-byte pieces that it shares with its neighbours; the
// copies take those pieces whole, except past the last row, whose last elements
// the copying thread moves itself.  Channels go to the threads one by one, so
// loads from the stage and stores stay consecutive across a warp.
//
// Wide rows take 16 channels per thread, one block of at most 512 threads per SM
// or more of fewer threads; narrower ones fewer channels, and as many blocks per
// SM as their registers allow.  With V = 1 the number of threads is NT, fixed at
// compile time: the offsets between a thread's 4 to 16 channels are then
// constants (computed, they were half of all instructions).
constexpr int kRingMaxHidden = 8192;
constexpr int kRingMaxStages = 4;
constexpr int kRingHeader = 1152;  // sums and barriers in front of the stages
constexpr int ring_max_threads(int U, int NT) { return NT ? NT : U == 1 ? 256 : 512; }
// Blocks per SM of that size: 512 threads of 128 registers, 640 of 102, 768 of
// 85 or 1024 of 64.
constexpr int ring_min_blocks(int V, int U, int NT) {
  const int n = (V * U == 16 ? 512 : V == 8 ? 768 : U == 8 ? 640 : 1024) / ring_max_threads(U, NT);
  return n > 0 ? n : 1;
}

struct Ring {
  int stages = 0;
  uint32_t stage_bytes = 0;
  uint32_t at[5] = {};  // where each stream's rows lie in a stage
};

// V elements of a staged row (its first byte at p) as f32, from channel c.
template <int V>
__device__ __forceinline__ void stage_elems(const uint8_t* p, int c, const Bf16*, float (&v)[V]) {
  if constexpr (V == 8)
    unpack8(*reinterpret_cast<const uint4*>(p + c * 2), v);
  else
    v[0] = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(p + c * 2) << 16);
}
template <int V>
__device__ __forceinline__ void stage_elems(const uint8_t* p, int c, const float*, float (&v)[V]) {
  if constexpr (V == 8) {
    const float4 a = *reinterpret_cast<const float4*>(p + c * 4);
    const float4 b = *reinterpret_cast<const float4*>(p + c * 4 + 16);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    v[0] = *reinterpret_cast<const float*>(p + c * 4);
  }
}
// V elements to a row: 8 f32 as one 32-byte store.
template <int V>
__device__ __forceinline__ void store_row(Bf16* p, const float (&v)[V]) {
  store_elems<V>(p, v);
}
template <int V>
__device__ __forceinline__ void store_row(float* p, const float (&v)[V]) {
  if constexpr (V == 8)
    asm volatile("st.global.cs.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]),
                 "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
  else
    st_stream_f32(p, v[0]);
}

// The copying side, run by thread 0, and the waiting side.
struct RingState {
  uint32_t bars, stages_at;
  int stage = 0;
  uint32_t parity = 0;
  bool ok = true;
  __device__ __forceinline__ void wait(unsigned* err) {
    if (ok && !mbar_wait(bars + stage * 8, parity)) {
      ok = false;  // reported; the results are not right
      flag_error(err, MOE_DEVERR_TIMEOUT);
    }
  }
  // The copying thread, before it leaves: after a wait that ran out, copies may
  // still be on their way.  A stage's barrier is in a phase of either parity;
  // waiting for the other one returns at once.
  __device__ __forceinline__ void drain(int stages) {
    if (ok || threadIdx.x != 0) return;
    for (int i = 0; i < 2 * stages; ++i) (void)mbar_wait(bars + i / 2 * 8, i & 1);
  }
  __device__ __forceinline__ void next(int stages) {
    if (++stage == stages) {
      stage = 0;
      parity ^= 1u;
    }
  }
};

// Starts the copies of rows t .. t + rows - 1 of every stream into a stage.
// V = 1: a row of the stream lies at its offset modulo 16.
template <int V>
__device__ __forceinline__ void ring_fill(const RingState& r, const Ring& ring, uint8_t* smem,
                                          int stage, const void* const (&src)[5],
                                          const uint32_t (&row_bytes)[5], int64_t t, int rows,
                                          int64_t T, unsigned* err) {
  const uint32_t bar = r.bars + stage * 8;
  const uint32_t dst = r.stages_at + stage * ring.stage_bytes;
  int64_t from[5];
  uint32_t bytes[5], total = 0;
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    from[i] = t * row_bytes[i];
    bytes[i] = 0;
    if (src[i] == nullptr) continue;
    int64_t to = from[i] + (int64_t)row_bytes[i] * rows;
    if (V == 1) {
      const int64_t whole = T * row_bytes[i] & ~(int64_t)15;
      const int64_t end = to;
      from[i] &= ~(int64_t)15;
      to = (to + 15) & ~(int64_t)15;
      if (to > whole) {  // the tensor's last elements
        to = whole;
        const int64_t first = t * row_bytes[i];
        for (int64_t b = to > first ? to : first; b < end; b += 2)
          *reinterpret_cast<uint16_t*>(smem + kRingHeader + stage * ring.stage_bytes + ring.at[i] +
                                       (b - from[i])) =
              *reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(src[i]) + b);
      }
    }
    bytes[i] = to > from[i] ? (uint32_t)(to - from[i]) : 0u;
    if (!MOE_DBG_OK(((reinterpret_cast<uintptr_t>(src[i]) | (uintptr_t)from[i] | bytes[i] |
                      (dst + ring.at[i])) & 15u) == 0 &&
                        ring.at[i] + bytes[i] <= ring.stage_bytes &&
                        kRingHeader + (stage + 1) * ring.stage_bytes <= dynamic_smem_bytes(),
                    err))
      bytes[i] = 0;
    total += bytes[i];
  }
  mbar_expect(bar, total);
#pragma unroll
  for (int i = 0; i < 5; ++i)
    if (bytes[i] > 0)
      bulk_load(dst + ring.at[i], static_cast<const uint8_t*>(src[i]) + from[i], bytes[i], bar);
}

// post_w * per-channel gate, and pre_w, of V channels.
template <int V>
__device__ __forceinline__ void channel_constants(const NormArgs& a, int c, float (&wg)[V],
                                                  float (&pw)[V]) {
#pragma unroll
  for (int q = 0; q < V; ++q) wg[q] = 1.0f, pw[q] = 0.0f;
  if (c >= a.H) return;
  float v[V];
  if (a.post_w) load_shared_f32<V>(a.post_w + c, wg);
  if (a.gate_kind == MOE_GATE_CHANNEL) {
    load_shared_f32<V>(static_cast<const float*>(a.gate) + c, v);
    gate_values<V>(a, v);
#pragma unroll
    for (int q = 0; q < V; ++q) wg[q] *= v[q];
  }
  if (a.pre_w) load_shared_f32<V>(a.pre_w + c, pw);
}

// The bits in which any [T, H] or [H] tensor's address is not aligned.
uintptr_t misalignment(const NormArgs& a) {
  const void* p[] = {a.residual, a.y, a.h, a.n, a.post_w, a.pre_w, a.grad_h, a.grad_n,
                     a.grad_residual, a.grad_y,
                     a.gate_kind == MOE_GATE_TOKEN ? nullptr : a.gate,
                     a.gate_kind == MOE_GATE_TOKEN ? nullptr : a.grad_gate};
  uintptr_t bits = 0;
  for (const void* q : p) bits |= reinterpret_cast<uintptr_t>(q);
  return bits;
}
bool vec_ok(const NormArgs& a) { return a.H % 8 == 0 && (misalignment(a) & 15u) == 0; }

// Threads per row (a multiple of 32) and rows per block for `units` accesses
// per row, NPT of them per thread.
struct Shape {
  int tpr, rows;
};
Shape row_shape(int units, int npt) {
  const int need = (units + npt - 1) / npt;
  Shape s;
  s.tpr = (need + 31) / 32 * 32;
  s.rows = s.tpr >= 256 ? 1 : 256 / s.tpr;
  return s;
}

// Elements per access of the ring for these tensors, 0 if they cannot use it.
int ring_vec(const NormArgs& a) {
  const uintptr_t bits = misalignment(a);
  if (a.H > kRingMaxHidden || (bits & 15u) != 0) return 0;
  return a.H % 8 == 0 && (bits & 31u) == 0 ? 8 : 1;
}

// The ring's shape; at least `least` stages, or none.
struct RingShape {
  Ring ring;
  int threads = 0, per_sm = 0;
};
template <int V, int U, int NT>
RingShape ring_shape(int H, int rows, const uint32_t (&row_bytes)[5], int least = 2) {
  RingShape s;
  for (int i = 0; i < 5; ++i) {
    s.ring.at[i] = s.ring.stage_bytes;
    // (up to 15 bytes before the rows and 15 behind them)
    if (row_bytes[i]) s.ring.stage_bytes += (rows * row_bytes[i] + 32 + 127) / 128 * 128;
  }
  s.threads = NT && V == 1 ? NT : (H + 32 * V * U - 1) / (32 * V * U) * 32;
  s.per_sm = ring_max_threads(U, NT) * ring_min_blocks(V, U, NT) / s.threads;
  if (s.per_sm > kNormMaxBlocksPerSm) s.per_sm = kNormMaxBlocksPerSm;
  for (; s.per_sm > 0; --s.per_sm) {  // (1 KB of each block's shared memory is the system's)
    const uint32_t room = 226u * 1024 / s.per_sm - 1024 - kRingHeader;
    s.ring.stages = (int)(room / s.ring.stage_bytes);
    if (s.ring.stages >= least) break;
    s.ring.stages = 0;
  }
  if (s.ring.stages > kRingMaxStages) s.ring.stages = kRingMaxStages;
  return s;
}

template <auto* kernel>
cudaError_t ring_launch(const LaunchCtx& c, const NormArgs& a, const RingShape& s,
                        int64_t max_blocks, int* blocks_out) {
  static SmemOptIn opt_in;
  cudaError_t e = opt_in.once(kernel);
  if (e != cudaSuccess) return e;
  int64_t blocks = (int64_t)c.num_sms * s.per_sm;
  if (blocks > max_blocks) blocks = max_blocks;
  *blocks_out = (int)blocks;
  const size_t smem = kRingHeader + (size_t)s.ring.stages * s.ring.stage_bytes;
  return launch_pdl(kernel, dim3((unsigned)blocks), s.threads, smem, c.stream, a, s.ring, c.err);
}

}  // namespace
}  // namespace moe
