// expert_matvec_fp4.cu -- products of routed rows with their expert's 4-bit
// weights (E2M1 codes, one scale per group of channels), for decode batches.
//
//   o[r, m] = sum_g w_sf[e, m, g] * sum_{c in g} x[src(r), c] * E2M1(w[e, m, c])
//
// With few rows per expert the weights are read once for little arithmetic,
// so HBM bounds it: K/2 bytes of codes and K/group scales per output.  At that
// rate an SM receives about 47 weights per clock.  Decoding them to f32 and
// multiplying on the FP32 lanes costs more issue slots than there are, so the
// products go to the tensor cores (mma.sync m16n8k16, f16 inputs, f32 sums):
// 16 outputs by up to 8 rows of x, the codes decoded two at a time by the
// hardware conversion E2M1 -> f16, which is exact.  (tcgen05.mma takes 4-bit
// weights only beside activations of 8 bits or fewer, which would round x.)
//
// x is bf16, which f16 cannot hold in range, so each block of 256 channels of
// a row is scaled by the power of two that brings its largest magnitude to
// [2^14, 2^15).  bf16's 8 significant bits fit f16's 11: a channel is exact
// unless it is below 2^-31 of its block's largest, and then off by less than
// 2^-39 of that largest.  The power of two is undone in f32.
//
// One CTA per SM.  Each computes, from the offsets, the list of (expert, run
// of up to C rows) items, and takes an equal share of all (item, tile of 16
// outputs) units, or of those of one item (kAloneSteps).  For each item the CTA converts the run's rows of x into
// shared memory once; then its 16 warps share the item's blocks of (tile, 256
// channels) in equal consecutive runs.  A tile that falls into several warps'
// runs is added up in warp order through shared memory.  Each warp streams its
// codes (TMA boxes) and scales (cp.async) through a ring of its own in shared
// memory, two blocks of 256 channels ahead, so no barrier stands in the stream.
//
// Measured: 64 tokens, top 8 of 256 experts, K = 2048, N = 7168, f32 scales per 128
// (1.74 GB): 244 us, 7.1 TB/s, above a plain copy's rate (reads alone run faster).
// Groups of 16: f32 scales (2.4 GB) 388 us, 6.3 TB/s, UE8M0 (1.8 GB) 372 us, 4.9 TB/s:
// the scaling of the groups' sums bounds those.
// One token, K = 7168, SwiGLU of 2 x 2048, UE8M0 scales per 32 (125 MB): 28 us, of
// which 8 us do not depend on N (launch, offsets, x, filling the rings); the
// slope is 6.4 TB/s.  At that rate a scheduler issues two thirds of its slots;
// what the warps execute per weight bounds it next: 64 conversions and 16 products
// per 4096 weights among 264 instructions.  A stage of 128 channels doubled
// the rest (42 us); cp.async for the codes filled the load queue ahead of the
// shared-memory reads (batch 292 us); 8 warps could not hide the latencies (51 us).
//
// With SwiGLU a tile is 8 gate outputs and the 8 up outputs of the same
// channels, which the fragment layout leaves in one lane.
#include "block/block_ops.cuh"

#include <cuda.h>
#include <cuda_fp16.h>

#include <type_traits>

namespace moe {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxRows = 8;   // columns of one mma
constexpr int kBlockK = 256;  // channels per ring stage
constexpr int kStages = 3;
// Few items: a CTA stays within one item, which saves a second start (about 2 us),
// if the largest share grows by no more than this many blocks of 256 channels.
// That against equal shares over all units, us: 29 tokens, top 2 of 16 experts, K =
// 1056, N = 1001 9.4 : 12.3; 20 tokens, 5 of 8, K = 5120, SwiGLU of 659 19.8 : 24.5.
// A limit of 300 instead: 6 tokens, 8 of 256, K = 2048, N = 7168 69 : 62.
constexpr int kAloneSteps = 32;
constexpr int kRowBytes = kBlockK / 2;  // codes of a row in a stage
constexpr int kCodeBytes = 16 * kRowBytes;

// A stage holds 16 rows of 128 code bytes (two TMA boxes of 8 rows, 128-byte
// swizzle: the 16-byte unit u of row r lies at unit u ^ (r % 8), so the 8 rows x
// 4 lanes of a fragment read meet 32 banks), and the rows' scales of the block.
// ALIGNED (K a multiple of 256 and 16-byte aligned scales): a row's scales of
// half a block start on a multiple of their own size, and each lane copies
// those of one half row.  Otherwise, and for bytes of G >= 64, 4-byte copies:
// f32 as above, or the aligned words that hold 256 / G bytes at any offset.
template <int G, bool U8, bool ALIGNED>
struct Stage {
  static constexpr int kGroups = kBlockK / G;
  static constexpr bool kHalves = ALIGNED && (!U8 || G <= 32);
  static constexpr int kWords = !U8 ? kGroups : kHalves ? kGroups / 4 : (kGroups + 6) / 4;
  static constexpr int kScaleBytes = 16 * kWords * 4;
};

// The two E2M1 codes of byte I of w as f16x2, element 0 (the low nibble) in
// the low half: the hardware conversion, exact.
template <int I>
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t w) {
  uint32_t r;
  if constexpr (I == 0)
    asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %1;\n"
        " cvt.rn.f16x2.e2m1x2 %0, b0;\n}" : "=r"(r) : "r"(w));
  else if constexpr (I == 1)
    asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %1;\n"
        " cvt.rn.f16x2.e2m1x2 %0, b1;\n}" : "=r"(r) : "r"(w));
  else if constexpr (I == 2)
    asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %1;\n"
        " cvt.rn.f16x2.e2m1x2 %0, b2;\n}" : "=r"(r) : "r"(w));
  else
    asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %1;\n"
        " cvt.rn.f16x2.e2m1x2 %0, b3;\n}" : "=r"(r) : "r"(w));
  return r;
}

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1, bool from_zero) {
  const float c[4] = {from_zero ? 0.0f : d[0], from_zero ? 0.0f : d[1], from_zero ? 0.0f : d[2],
                      from_zero ? 0.0f : d[3]};
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]),
        "f"(c[2]), "f"(c[3]));
}

// Asynchronous copies of 16, 8 or 4 bytes into shared memory; only the first
// `bytes` are read, the rest is zero.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A box of 8 rows of 128 bytes at byte column c and row r of the codes.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int c, int r,
                                        uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(dst),
      "l"(map), "r"(c), "r"(r), "r"(bar)
      : "memory");
}

// Shared-memory loads at a 32-bit address plus a constant.  Volatile: kept in
// program order, between the products that use them (grouped ahead of a block's
// products, as the compiler would have them, they fill the load queue: 16 warps
// then wait on it, 364 -> 448 us for 32768 outputs of 8 experts, K = 7168).
template <int OFF>
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1+%2];" : "=r"(v) : "r"(a), "n"(OFF));
  return v;
}
template <int OFF>
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1+%2];" : "=h"(v) : "r"(a), "n"(OFF));
  return v;
}
template <int OFF>
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2+%3];" : "=r"(v.x), "=r"(v.y) : "r"(a), "n"(OFF));
  return v;
}
template <int OFF>
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4+%5];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a), "n"(OFF));
  return v;
}
// f(0), ..., f(N - 1), the arguments compile-time constants.
template <int N, int I = 0, class F>
__device__ __forceinline__ void unrolled(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>());
    unrolled<N, I + 1>(static_cast<F&&>(f));
  }
}
// 2^(b - 127) of the four bytes of w: the hardware conversion to bf16, exact
// (2^-127 is a denormal there too).
__device__ __forceinline__ void ue8m0x4(uint32_t w, float (&s)[4]) {
  uint32_t lo, hi;
  asm("{\n .reg .b16 h0, h1;\n mov.b32 {h0, h1}, %2;\n cvt.rn.bf16x2.ue8m0x2 %0, h0;\n"
      " cvt.rn.bf16x2.ue8m0x2 %1, h1;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
  s[0] = bf16_lo(lo), s[1] = bf16_hi(lo), s[2] = bf16_lo(hi), s[3] = bf16_hi(hi);
}

// Shared memory: the warps' rings of codes (1024-byte aligned for the swizzle)
// and of scales, the x rows (f16, row stride 2 Kp + 64 bytes so that
// neighbouring rows fall into different halves of the banks), the powers of two
// [Kp / 256][8], the warps' partial sums, the barriers, and per expert the items
// before it, its first row and the end of its rows.
struct Smem {
  uint32_t codes, scales, x, xs, red, bars, first, rows, total;
};
__host__ __device__ inline int padded_k(int K) { return (K + kBlockK - 1) / kBlockK * kBlockK; }
__host__ __device__ inline uint32_t x_stride(int K) { return (uint32_t)padded_k(K) * 2 + 64; }
__host__ __device__ inline Smem smem_layout(int scale_bytes, int K, int E, int C) {
  Smem s;
  s.codes = 0;
  s.scales = (uint32_t)(kWarps * kStages * kCodeBytes);
  s.x = s.scales + (uint32_t)(kWarps * kStages * scale_bytes);
  s.xs = s.x + (uint32_t)C * x_stride(K);
  s.red = s.xs + (uint32_t)(padded_k(K) / kBlockK) * kMaxRows * 4;
  s.bars = s.red + kWarps * 512;
  s.first = s.bars + (uint32_t)(kWarps * kStages * 8);
  s.rows = s.first + (uint32_t)(E + 2) / 2 * 8;
  s.total = s.rows + (uint32_t)E * 8;
  return s;
}

// Row r's row of x, or -1 for a row of zeros.
__device__ __forceinline__ int64_t source_row(const MatvecArgs& a, int r, unsigned* err) {
  int64_t s = r;
  if (a.src != nullptr) {
    const int v = __ldg(a.src + r);
    if (v < 0) return -1;
    s = v / a.k;
  }
  if (s >= a.num_x) {
    flag_error(err, MOE_DEVERR_POS_RANGE);
    return -1;
  }
  return s;
}

template <int G, bool U8, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 1)
    expert_matvec_kernel(const MatvecArgs a, const __grid_constant__ CUtensorMap map,
                         const int C, unsigned* err) {
  // the map is a launch parameter: its fetch need not wait for earlier kernels
  if (threadIdx.x == 0)
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map) : "memory");
  pdl_enter();
  using St = Stage<G, U8, ALIGNED>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const Smem L = smem_layout(St::kScaleBytes, a.K, a.E, C);
  const uint32_t sbase = (uint32_t)__cvta_generic_to_shared(smem);
  int* first = reinterpret_cast<int*>(smem + L.first);
  int2* rows_of = reinterpret_cast<int2*>(smem + L.rows);
  float* xs = reinterpret_cast<float*>(smem + L.xs);
  float4* red = reinterpret_cast<float4*>(smem + L.red);
  const int tid = threadIdx.x, lane = tid & 31;
  // broadcast, so that what derives from it is known to be one value per warp
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int g = lane >> 2, q = lane & 3;
  const int M = a.swiglu ? 2 * a.N : a.N;
  const int per_tile = a.swiglu ? 8 : 16;  // outputs of one tile
  const int tiles = (a.N + per_tile - 1) / per_tile;
  const int nblk = (a.K + kBlockK - 1) / kBlockK;
  const uint32_t xrow_bytes = x_stride(a.K);
  const int64_t sf_row = a.K / G;  // scales of one weight row

  const uint32_t bar = sbase + L.bars + (uint32_t)(warp * kStages * 8);  // of this warp's stages
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(bar + i * 8);
    mbar_init_done();
  }

  // first[e]: items of the experts before e; each thread counts kPer experts
  {
    constexpr int kPer = (MOE_MAX_EXPERTS + kThreads - 1) / kThreads;
    int* totals = reinterpret_cast<int*>(red);
    int runs[kPer] = {};
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = kPer * tid + i;
      if (e >= a.E) continue;
      int64_t lo = 0, hi = a.R;
      if (a.offsets != nullptr) {
        lo = __ldg(a.offsets + e);
        hi = __ldg(a.offsets + e + 1);
        if (lo < 0 || hi > a.R) flag_error(err, MOE_DEVERR_POS_RANGE);
        if (lo < 0) lo = 0;
        if (hi > a.R) hi = a.R;
      }
      rows_of[e] = make_int2((int)lo, (int)hi);
      runs[i] = hi > lo ? (int)((hi - lo + C - 1) / C) : 0;
    }
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum += runs[i];
    const int own = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) totals[warp] = sum;
    __syncthreads();
    int before = sum - own;
    for (int w = 0; w < warp; ++w) before += totals[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (kPer * tid + i <= a.E) first[kPer * tid + i] = before;
      before += runs[i];
    }
    if (tid == kThreads - 1 && a.E == kPer * kThreads) first[a.E] = before;
    __syncthreads();
  }
  // this CTA's share of the units
  const uint32_t items = (uint32_t)first[a.E], grid = gridDim.x, b = blockIdx.x;
  int64_t u0, u1;
  bool alone = false;
  if (items > 0 && items <= grid && tiles <= 1 << 20) {
    const uint32_t few = grid / items, most = (items * tiles + grid - 1) / grid;
    alone = ((tiles + few - 1) / few - most) * nblk <= kAloneSteps;
  }
  if (alone) {
    const uint32_t i = ((b + 1) * items - 1) / grid, c0 = grid * i / items;
    const uint32_t ctas = grid * (i + 1) / items - c0;
    u0 = i * tiles + tiles * (b - c0) / ctas;
    u1 = i * tiles + tiles * (b - c0 + 1) / ctas;
  } else {
    const int64_t units = (int64_t)items * tiles;
    u0 = units * b / grid, u1 = units * (b + 1) / grid;
  }

  const uint32_t codes = sbase + L.codes + (uint32_t)(warp * kStages * kCodeBytes);
  const uint32_t scales = sbase + L.scales + (uint32_t)(warp * kStages * St::kScaleBytes);
  uint32_t phase = 0;  // bit i: the parity that stage i's barrier is at
  bool ok = true;      // no wait ran out

  int64_t u = u0;
  while (u < u1) {
    // the item of unit u, and the part of this CTA's share in it
    const int item = (int)(u / tiles);
    int e = 0;  // the last expert with first[e] <= item
    for (int hi = a.E; hi - e > 1;) {
      const int mid = (e + hi) >> 1;
      if (first[mid] <= item)
        e = mid;
      else
        hi = mid;
    }
    const int tile0 = (int)(u - (int64_t)item * tiles);
    const int64_t left = u1 - u;
    const int ntiles = (int)(left < tiles - tile0 ? left : tiles - tile0);
    u += ntiles;
    const int2 rows = rows_of[e];
    const int r0 = rows.x + (item - first[e]) * C;
    const int n = rows.y - r0 < C ? rows.y - r0 : C;

    // this warp's run of the item's (tile, block) steps
    const int all = ntiles * nblk;
    auto run_begin = [&](int w) { return (int)((int64_t)all * w / kWarps); };
    const int run0 = run_begin(warp), steps = run_begin(warp + 1) - run0;
    const int m_e = e * M;
    const int64_t sf_e = (int64_t)m_e * sf_row;
    // weight row, within the expert, of row i of a tile; past the last output
    // the last one, whose products are not stored
    auto weight_row = [&](int tile, int i) -> uint32_t {
      const int nn = tile * per_tile + (a.swiglu ? i & 7 : i);
      return (uint32_t)((nn < a.N ? nn : a.N - 1) + (a.swiglu ? (i >> 3) * a.N : 0));
    };

    // the stream of stages: where the next one comes from and goes to
    int ld_tile = tile0 + run0 / nblk, ld_blk = run0 % nblk, to_issue = ok ? steps : 0;
    int tile = ld_tile, blk = ld_blk;
    bool head = blk != 0;  // the current tile began in an earlier warp's run
    const char* sf_at = nullptr;  // kHalves: this lane's first scale of block ld_blk
    auto open_tile = [&]() {
      if (St::kHalves) {
        const int64_t at = sf_e + weight_row(ld_tile, lane >> 1) * (uint32_t)sf_row +
                           (uint32_t)(ld_blk * St::kGroups + (lane & 1) * (St::kGroups / 2));
        sf_at = static_cast<const char*>(a.sf) + at * (U8 ? 1 : 4);
      }
    };
    if (steps > 0) open_tile();
    // fills stage I with the next block
    auto issue = [&](auto I) {
      constexpr int ld_stage = I;
      if (to_issue > 0) {
        --to_issue;
        if (lane == 0) {
          // rows past the last output are another's, or past the tensor and zero
          const uint32_t b = bar + ld_stage * 8, dst = codes + ld_stage * kCodeBytes;
          const int r = m_e + ld_tile * per_tile;
          // the boxes' columns are whole 16 bytes; each fills 1024 bytes of the ring
          const bool box_ok =
              MOE_DBG_OK(dst % (kCodeBytes / 2) == 0 && dst + kCodeBytes <= sbase + L.scales &&
                             (ld_blk * kRowBytes) % 16 == 0 && ld_blk < nblk,
                         err);
          mbar_expect(b, box_ok ? kCodeBytes : 0);
          if (box_ok) {
            tma_box(dst, &map, ld_blk * kRowBytes, r, b);
            tma_box(dst + kCodeBytes / 2, &map, ld_blk * kRowBytes, r + (a.swiglu ? a.N : 8), b);
          }
        }
        const uint32_t sst = scales + ld_stage * St::kScaleBytes;
        if (St::kHalves) {
          constexpr int kBytes = St::kGroups / 2 * (U8 ? 1 : 4);  // of half a row
          if constexpr (kBytes >= 16) {
#pragma unroll
            for (int i = 0; i < kBytes; i += 16) cp_async16(sst + lane * kBytes + i, sf_at + i, 16);
          } else if constexpr (kBytes == 8) {
            cp_async8(sst + lane * 8, sf_at, 8);
          } else {
            cp_async4(sst + lane * 4, sf_at, 4);
          }
          sf_at += 2 * kBytes;
        } else if (U8) {
          // nothing past the row's own scales: beside the zero codes and channels past
          // K another row's 255 (a NaN) would not vanish
          const uint8_t* sf = static_cast<const uint8_t*>(a.sf);
#pragma unroll
          for (int i = 0; i < (St::kWords + 1) / 2; ++i) {
            const int p = lane + 32 * i, row = p / St::kWords, wi = p % St::kWords;
            if (St::kWords % 2 != 0 && p >= 16 * St::kWords) break;
            const int64_t row_at = sf_e + weight_row(ld_tile, row) * (uint32_t)sf_row;
            const int64_t at =
                ((row_at + (uint32_t)(ld_blk * St::kGroups)) & ~(int64_t)3) + 4 * wi;
            const int64_t left = row_at + sf_row - at;
            const int bytes = left < 0 ? 0 : left > 4 ? 4 : (int)left;
            cp_async4(sst + p * 4, sf + (bytes > 0 ? at : 0), bytes);
          }
        } else {
          const float* sf = static_cast<const float*>(a.sf) + sf_e;
#pragma unroll
          for (int i = 0; i < (16 * St::kGroups + 31) / 32; ++i) {
            const int p = lane + 32 * i, row = p / St::kGroups;
            const uint32_t gi = (uint32_t)(ld_blk * St::kGroups + p % St::kGroups);
            const bool ok = gi < (uint32_t)sf_row;
            cp_async4(sst + p * 4, sf + (ok ? weight_row(ld_tile, row) * (uint32_t)sf_row + gi : 0),
                      ok ? 4 : 0);
          }
        }
        if (++ld_blk == nblk) {
          ld_blk = 0;
          ++ld_tile;
          if (to_issue > 0) open_tile();
        }
      }
      cp_async_commit();
    };
    unrolled<kStages - 1>(issue);

    // x: each warp converts blocks of 256 channels of a row, two loads ahead
    const int64_t my_src = lane < n ? source_row(a, r0 + lane, err) : -1;
    auto fetch_x = [&](int t) {
      const int col = t / nblk, c = (t - col * nblk) * kBlockK + lane * 8;
      const int64_t sr = __shfl_sync(0xFFFFFFFFu, my_src, col & 7);
      uint4 v = make_uint4(0, 0, 0, 0);
      if (t < n * nblk && sr >= 0 && c < a.K)
        v = ld_v4(static_cast<const uint16_t*>(a.x) + sr * a.K + c);
      return v;
    };
    uint4 v0 = fetch_x(warp), v1 = fetch_x(warp + kWarps);
    for (int t = warp; t < n * nblk; t += kWarps) {
      const uint4 v = v0;
      v0 = v1;
      v1 = fetch_x(t + 2 * kWarps);
      const int col = t / nblk, b = t - col * nblk, c = b * kBlockK + lane * 8;
      float f[8];
      unpack8(v, f);
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
      // 2^ex brings m's exponent to 14; kept to 126 so that 2^-ex is normal
      int ex = (int)(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m)) >> 23);
      ex = 14 + 127 - ex;
      ex = ex > 126 ? 126 : ex;
      const float up = __uint_as_float((uint32_t)(127 + ex) << 23);
      uint4 h;
      uint32_t* hw = reinterpret_cast<uint32_t*>(&h);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 p = __floats2half2_rn(f[2 * i] * up, f[2 * i + 1] * up);
        hw[i] = *reinterpret_cast<const uint32_t*>(&p);
      }
      *reinterpret_cast<uint4*>(smem + L.x + col * xrow_bytes + c * 2) = h;
      if (lane == 0) xs[b * kMaxRows + col] = __uint_as_float((uint32_t)(127 - ex) << 23);
    }
    __syncthreads();

    // lanes of columns past the run read the last one's: their sums are not stored
    const uint32_t xcol =
        sbase + L.x + (g < n ? g : n - 1) * xrow_bytes + (G == 16 ? q * 8 : q * 16);
    // unit j of row g (and of row g + 8, 1024 bytes on) in a stage
    uint32_t frag[kBlockK / 32];
#pragma unroll
    for (int j = 0; j < kBlockK / 32; ++j)
      frag[j] = codes + (uint32_t)(g * kRowBytes + ((j ^ g) << 4) + (G == 16 ? q * 2 : q * 4));
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    // where a row's scales start in its first word
    constexpr bool kShift = U8 && !St::kHalves;
    int sf_off[2] = {0, 0};
    auto tile_offsets = [&]() {
      if (kShift) {
        sf_off[0] = (int)((sf_e + weight_row(tile, g) * (uint32_t)sf_row) & 3);
        sf_off[1] = (int)((sf_e + weight_row(tile, g + 8) * (uint32_t)sf_row) & 3);
      }
    };
    tile_offsets();
    // one block of this warp's tiles, from stage I
    auto block = [&](auto I) {
        constexpr int stage = I;
        cp_async_wait<kStages - 2>();
        if (ok && !mbar_wait(bar + stage * 8, (phase >> stage) & 1u)) {
          // reported; nothing more is fetched, and what may be on its way to the
          // other stages is waited for (bounded again)
          ok = false;
          to_issue = 0;
          flag_error(err, MOE_DEVERR_TIMEOUT);
          for (int i = 0; i < kStages; ++i)
            if (i != stage) (void)mbar_wait(bar + i * 8, (phase >> i) & 1u);
        }
        phase ^= 1u << stage;
        __syncwarp();
        issue(std::integral_constant<int, (stage + kStages - 1) % kStages>());
        const uint32_t sst = scales + stage * St::kScaleBytes + g * (St::kWords * 4);
        const float2 xc = *reinterpret_cast<const float2*>(xs + blk * kMaxRows + 2 * q);
        // scales of rows g and g + 8
        float s[2][St::kGroups < 4 ? 4 : St::kGroups];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t sw[St::kWords + 1];
          const uint32_t at = sst + 8 * i * (St::kWords * 4);
          if constexpr (St::kWords % 4 == 0) {
            unrolled<St::kWords / 4>([&](auto J) {
              const uint4 v = lds128<J * 16>(at);
              sw[J * 4] = v.x, sw[J * 4 + 1] = v.y, sw[J * 4 + 2] = v.z, sw[J * 4 + 3] = v.w;
            });
          } else if constexpr (St::kWords == 2) {
            const uint2 v = lds64<0>(at);
            sw[0] = v.x, sw[1] = v.y;
          } else {
            unrolled<St::kWords>([&](auto J) { sw[J] = lds32<J * 4>(at); });
          }
          sw[St::kWords] = 0;
          if constexpr (!U8) {
#pragma unroll
            for (int j = 0; j < St::kGroups; ++j) s[i][j] = __uint_as_float(sw[j]);
          } else {
#pragma unroll
            for (int j = 0; j < St::kGroups; j += 4) {
              uint32_t w = sw[j / 4];
              if constexpr (kShift)
                w = __funnelshift_r(w, sw[j / 4 + 1], 8 * ((sf_off[i] + blk * St::kGroups) & 3));
              float v[4];
              ue8m0x4(w, v);
#pragma unroll
              for (int b = 0; b < 4; ++b) s[i][j + b] = v[b];
            }
          }
        }
        float part[4] = {0.0f, 0.0f, 0.0f, 0.0f}, blk_acc[4];
        auto flush = [&](int gi) {  // a group is complete: scale its sums
#pragma unroll
          for (int i = 0; i < 4; ++i)
            blk_acc[i] = gi == 0 ? s[i >> 1][gi] * part[i]
                                 : __fmaf_rn(s[i >> 1][gi], part[i], blk_acc[i]);
        };
        const uint32_t xb = xcol + (uint32_t)blk * (2 * kBlockK);
        constexpr int kSt = stage * kCodeBytes, kHi = kSt + 8 * kRowBytes;  // from row g to row g + 8
        unrolled<kBlockK / 32>([&](auto J) {
          constexpr int j = J;
          const uint32_t row = frag[j];
          uint32_t a0[4], a1[4];
          uint4 x;
          if constexpr (G == 16) {
            // the 16 channels of a group: 2 bytes of codes per lane
            const uint32_t w0 = lds16<kSt>(row), w1 = lds16<kSt + 8>(row);
            const uint32_t w2 = lds16<kHi>(row), w3 = lds16<kHi + 8>(row);
            a0[0] = e2m1x2_to_f16x2<0>(w0), a0[2] = e2m1x2_to_f16x2<1>(w0);
            a0[1] = e2m1x2_to_f16x2<0>(w2), a0[3] = e2m1x2_to_f16x2<1>(w2);
            a1[0] = e2m1x2_to_f16x2<0>(w1), a1[2] = e2m1x2_to_f16x2<1>(w1);
            a1[1] = e2m1x2_to_f16x2<0>(w3), a1[3] = e2m1x2_to_f16x2<1>(w3);
            const uint2 p = lds64<j * 64>(xb), r = lds64<j * 64 + 32>(xb);
            x = make_uint4(p.x, p.y, r.x, r.y);
          } else {
            const uint32_t w0 = lds32<kSt>(row), w1 = lds32<kHi>(row);
            x = lds128<j * 64>(xb);
            a0[0] = e2m1x2_to_f16x2<0>(w0), a0[2] = e2m1x2_to_f16x2<1>(w0);
            a0[1] = e2m1x2_to_f16x2<0>(w1), a0[3] = e2m1x2_to_f16x2<1>(w1);
            a1[0] = e2m1x2_to_f16x2<2>(w0), a1[2] = e2m1x2_to_f16x2<3>(w0);
            a1[1] = e2m1x2_to_f16x2<2>(w1), a1[3] = e2m1x2_to_f16x2<3>(w1);
          }
          mma_16816(part, a0, x.x, x.y, G <= 32 || (j * 32) % G == 0);
          if constexpr (G == 16) flush(2 * j);
          mma_16816(part, a1, x.z, x.w, G == 16);
          if constexpr (G == 16)
            flush(2 * j + 1);
          else if constexpr ((j * 32 + 32) % G == 0)
            flush((j * 32) / G);
        });
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = __fmaf_rn(i & 1 ? xc.y : xc.x, blk_acc[i], acc[i]);
        ++blk;
    };
    auto write_out = [&]() {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int col = 2 * q + (i & 1);
        float o = acc[i];
        int nn;
        if (a.swiglu) {
          if (i >= 2) break;
          o = o / (1.0f + expf(-o)) * acc[i + 2];
          nn = tile * 8 + g;
        } else {
          nn = tile * 16 + g + (i >> 1) * 8;
        }
        if (col >= n || nn >= a.N) continue;
        const int64_t at = (int64_t)(r0 + col) * a.N + nn;
        if (a.out_f32)
          static_cast<float*>(a.out)[at] = o;
        else
          static_cast<uint16_t*>(a.out)[at] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
      }
    };
    auto leave = [&]() { red[warp * 32 + lane] = make_float4(acc[0], acc[1], acc[2], acc[3]); };
    // whole turns of the ring, so that every stage address is a constant; the
    // next item starts at stage 0 again
    for (int step = 0; step < steps; step += kStages)
      unrolled<kStages>([&](auto I) {
        if (step + I >= steps) return;
        block(I);
        if (blk < nblk) return;
        // the tile ends here
        if (head)
          leave();
        else
          write_out();
        head = false;
        acc[0] = acc[1] = acc[2] = acc[3] = 0.0f;
        blk = 0;
        ++tile;
        tile_offsets();
      });
    // a tile that goes on in the next run: its first warp adds the others' sums
    const bool open = steps > 0 && blk > 0;
    if (open && head) leave();
    __syncthreads();
    if (open && !head) {
      const int end = (tile - tile0 + 1) * nblk;
      for (int w = warp + 1; w < kWarps && run_begin(w) < end; ++w) {
        if (run_begin(w) == run_begin(w + 1)) continue;
        const float4 v = red[w * 32 + lane];
        acc[0] += v.x, acc[1] += v.y, acc[2] += v.z, acc[3] += v.w;
      }
      write_out();
    }
    cp_async_wait<0>();
    __syncthreads();  // x and the sums are free for the next item
  }
}

// The codes as a tensor of rows of K / 2 bytes, in boxes of 8 rows of 128 bytes.
cudaError_t code_map(const MatvecArgs& a, CUtensorMap* map) {
  using Encode = decltype(&cuTensorMapEncodeTiled);
  static const Encode encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                                           cudaEnableDefault, &found);
    return e == cudaSuccess && found == cudaDriverEntryPointSuccess ? reinterpret_cast<Encode>(fn)
                                                                    : nullptr;
  }();
  if (encode == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {(cuuint64_t)a.K / 2,
                              (cuuint64_t)a.E * a.N * (a.swiglu ? 2 : 1)};
  const cuuint64_t strides[1] = {(cuuint64_t)a.K / 2};
  const cuuint32_t box[2] = {kRowBytes, 8}, unit[2] = {1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(a.w), dims,
                            strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int G, bool U8, bool ALIGNED>
cudaError_t launch_t(const LaunchCtx& c, const MatvecArgs& a) {
  constexpr int kScaleBytes = Stage<G, U8, ALIGNED>::kScaleBytes;
  // rows per item: the 8 columns of the mma, but no more than an expert can get
  // (a token's experts are distinct: one row per token; more would only take
  // more items), and fewer where a long x would not fit
  int C = kMaxRows;
  while (C > 1 && C / 2 >= (a.R + a.k - 1) / a.k) C >>= 1;
  while (C > 1 && smem_layout(kScaleBytes, a.K, a.E, C).total > 227 * 1024) C >>= 1;
  const size_t smem = smem_layout(kScaleBytes, a.K, a.E, C).total;
  auto* kernel = expert_matvec_kernel<G, U8, ALIGNED>;
  static SmemOptIn opt_in;
  cudaError_t e = opt_in.once(kernel);
  if (e != cudaSuccess) return e;
  CUtensorMap map;
  e = code_map(a, &map);
  if (e != cudaSuccess) return e;
  int64_t items = (a.offsets ? a.E : 1) + a.R / C;
  if (items > a.R) items = a.R;
  const int per_tile = a.swiglu ? 8 : 16;
  const int64_t units = items * ((a.N + per_tile - 1) / per_tile);
  const int64_t blocks = units < c.num_sms ? units : c.num_sms;
  return launch_pdl(kernel, dim3((unsigned)blocks), kThreads, smem, c.stream, a, map, C, c.err);
}

template <int G>
cudaError_t launch_g(const LaunchCtx& c, const MatvecArgs& a) {
  const bool al = a.K % kBlockK == 0 && (reinterpret_cast<uintptr_t>(a.sf) & 15u) == 0;
  if (a.sf_type == MOE_WSF_UE8M0)
    return al ? launch_t<G, true, true>(c, a) : launch_t<G, true, false>(c, a);
  return al ? launch_t<G, false, true>(c, a) : launch_t<G, false, false>(c, a);
}

}  // namespace

cudaError_t launch_expert_matvec_fp4(const LaunchCtx& c, const MatvecArgs& a) {
  switch (a.group) {
    case 16: return launch_g<16>(c, a);
    case 32: return launch_g<32>(c, a);
    case 64: return launch_g<64>(c, a);
    default: return launch_g<128>(c, a);
  }
}

}  // namespace moe
