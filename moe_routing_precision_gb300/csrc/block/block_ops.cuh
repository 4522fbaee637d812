// block_ops.cuh -- what the operators around the routed experts share: element
// access, and the launchers that api_block.cu validates for and calls.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace moe {

// bf16 in memory; f32 is float itself.
struct Bf16 {
  uint16_t bits;
};

// Two f32 values rounded to nearest even bf16, `lo` in the low half: one paired
// conversion (the single one runs at a quarter of its rate).
__device__ __forceinline__ uint32_t pack_bf16x2_rn(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

__device__ __forceinline__ void unpack8(const uint4& a, float (&v)[8]) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(w[i]);
    v[2 * i + 1] = bf16_hi(w[i]);
  }
}

// 16-byte load of data read once, through the coherent path: an output may
// share its address (in-place updates), each element read before it is stored.
__device__ __forceinline__ uint4 ld_once_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// VEC consecutive elements as f32: one element, or eight through 16-byte
// accesses (p 16-byte aligned).  Loads are read-once (no L1 allocation);
// stores are evict-first.
template <int VEC>
__device__ __forceinline__ void load_elems(const Bf16* p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    unpack8(ld_once_v4(p), v);
  } else {
    static_assert(VEC == 1, "one or eight elements");
    v[0] = __uint_as_float((uint32_t)p->bits << 16);
  }
}

template <int VEC>
__device__ __forceinline__ void load_elems(const float* p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    const uint4 a = ld_once_v4(p), b = ld_once_v4(p + 4);
    v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y);
    v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
    v[4] = __uint_as_float(b.x), v[5] = __uint_as_float(b.y);
    v[6] = __uint_as_float(b.z), v[7] = __uint_as_float(b.w);
  } else {
    static_assert(VEC == 1, "one or eight elements");
    v[0] = *p;
  }
}

// f32 values other rows re-read (weights, per-channel gates): the cached path.
template <int VEC>
__device__ __forceinline__ void load_shared_f32(const float* p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    v[0] = __ldg(p);
  }
}

template <int VEC>
__device__ __forceinline__ void store_elems(Bf16* p, const float (&v)[VEC]) {
  if constexpr (VEC == 8)
    st_stream_v4(p, make_uint4(pack_bf16x2_rn(v[0], v[1]), pack_bf16x2_rn(v[2], v[3]),
                               pack_bf16x2_rn(v[4], v[5]), pack_bf16x2_rn(v[6], v[7])));
  else
    p->bits = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
}

template <int VEC>
__device__ __forceinline__ void store_elems(float* p, const float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    st_stream_v4(p, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]),
                               __float_as_uint(v[2]), __float_as_uint(v[3])));
    st_stream_v4(p + 4, make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]),
                                   __float_as_uint(v[6]), __float_as_uint(v[7])));
  } else {
    *p = v[0];
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// 1 / x for 2^-126 <= x < 2^126, to an ulp: the hardware estimate and one Newton step.
__device__ __forceinline__ float rcp_f32(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return __fmaf_rn(y, __fmaf_rn(-x, y, 1.0f), y);
}

// g = 1 / (1 + e^-x) and g' = g (1 - g), both to a few ulp for every x: with
// e = e^-|x| the larger of g and 1 - g is 1 / (1 + e), the smaller e / (1 + e).
__device__ __forceinline__ float sigmoid_f32(float x, float* deriv = nullptr) {
  const float e = expf(-fabsf(x));
  const float big = rcp_f32(1.0f + e), small = e * big;
  if (deriv) *deriv = big * small;
  return x < 0.0f ? small : big;
}

// 1 / sqrt(x) for x > 0: the hardware estimate and one Newton step, whose x is kept
// finite: 0 for +inf, not 0 * inf.  (Beside the estimate; a choice after the step
// stood in every row's chain: 16384 rows of 7168, bf16, 140.3 : 139.4 us.)
__device__ __forceinline__ float rsqrt_f32(float x) {
  const float y = rsqrtf(x), v = fminf(x, 3.402823466e38f);
  return __fmaf_rn(0.5f * y, __fmaf_rn(-v * y, y, 1.0f), y);
}

// ----------------------------------------------------------- pairs of f32

// y = a b, y += a b, s += a . b, y = a + b of V values, a scalar operand taken V times.
// PAIRS: two values per instruction.
__device__ __forceinline__ void mul2(float* y, const float* a, const float* b) {
  asm("{\n .reg .b64 p, q;\n mov.b64 p, {%2, %3};\n mov.b64 q, {%4, %5};\n"
      " mul.rn.f32x2 p, p, q;\n mov.b64 {%0, %1}, p;\n}"
      : "=f"(y[0]), "=f"(y[1])
      : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]));
}
__device__ __forceinline__ void fma2(float* y, const float* a, const float* b) {
  asm("{\n .reg .b64 p, q, r;\n mov.b64 p, {%2, %3};\n mov.b64 q, {%4, %5};\n"
      " mov.b64 r, {%0, %1};\n fma.rn.f32x2 r, p, q, r;\n mov.b64 {%0, %1}, r;\n}"
      : "+f"(y[0]), "+f"(y[1])
      : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]));
}
template <bool PAIRS, int V>
__device__ __forceinline__ void mul_v(float (&y)[V], const float (&a)[V], const float (&b)[V]) {
  if constexpr (PAIRS && V % 2 == 0) {
#pragma unroll
    for (int q = 0; q < V; q += 2) mul2(y + q, a + q, b + q);
  } else {
#pragma unroll
    for (int q = 0; q < V; ++q) y[q] = a[q] * b[q];
  }
}
template <bool PAIRS, int V>
__device__ __forceinline__ void fma_v(float (&y)[V], const float (&a)[V], const float (&b)[V]) {
  if constexpr (PAIRS && V % 2 == 0) {
#pragma unroll
    for (int q = 0; q < V; q += 2) fma2(y + q, a + q, b + q);
  } else {
#pragma unroll
    for (int q = 0; q < V; ++q) y[q] = __fmaf_rn(a[q], b[q], y[q]);
  }
}
template <int V>
__device__ __forceinline__ void fill_v(float (&y)[V], float a) {
#pragma unroll
  for (int q = 0; q < V; ++q) y[q] = a;
}
template <bool PAIRS, int V>
__device__ __forceinline__ void mul_v(float (&y)[V], float a, const float (&b)[V]) {
  float p[V];
  fill_v(p, a);
  mul_v<PAIRS>(y, p, b);
}
template <bool PAIRS, int V>
__device__ __forceinline__ void fma_v(float (&y)[V], float a, const float (&b)[V]) {
  float p[V];
  fill_v(p, a);
  fma_v<PAIRS>(y, p, b);
}
template <bool PAIRS, int V>
__device__ __forceinline__ void dot_v(float (&s)[2], const float (&a)[V], const float (&b)[V]) {
  if constexpr (PAIRS && V % 2 == 0) {
#pragma unroll
    for (int q = 0; q < V; q += 2) fma2(s, a + q, b + q);
  } else {
#pragma unroll
    for (int q = 0; q < V; ++q) s[0] = __fmaf_rn(a[q], b[q], s[0]);
  }
}
template <bool PAIRS, int V>
__device__ __forceinline__ void add_v(float (&y)[V], const float (&a)[V], float b) {
  if constexpr (PAIRS && V % 2 == 0) {
#pragma unroll
    for (int q = 0; q < V; q += 2)
      asm("{\n .reg .b64 p, q;\n mov.b64 p, {%2, %3};\n mov.b64 q, {%4, %4};\n"
          " add.rn.f32x2 p, p, q;\n mov.b64 {%0, %1}, p;\n}"
          : "=f"(y[q]), "=f"(y[q + 1])
          : "f"(a[q]), "f"(a[q + 1]), "f"(b));
  } else {
#pragma unroll
    for (int q = 0; q < V; ++q) y[q] = a[q] + b;
  }
}

// ------------------------------------------------ barriers of bulk copies

__device__ __forceinline__ void mbar_init(uint32_t bar) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// Waits for the phase `parity` of the barrier; false if that took over a second (`bound` ns).
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity,
                                          uint64_t bound = 1000000000ull) {
  uint64_t begin = 0;
  for (;;) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    if (done) return true;
    const uint64_t t = now_ns();
    if (begin == 0) begin = t;
    if (t - begin > bound) return false;
  }
}
// Copies `bytes` (a multiple of 16) from global to shared memory, both 16-byte
// aligned, and counts them at the barrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
// Makes barriers that this thread initialised known to the copy engine.
__device__ __forceinline__ void mbar_init_done() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ------------------------------------------------------------- launchers

// allow_max_dynamic_smem, called once per device for each kernel: a launch that
// needs more than the default must not pay the call every time (0.6 us each on
// a Grace host).  One object per kernel instance.
class SmemOptIn {
 public:
  template <typename... KArgs>
  cudaError_t once(void (*kernel)(KArgs...)) {
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (device & 63);  // context() admits 64 devices
    if (done_.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = allow_max_dynamic_smem(kernel);
    if (e == cudaSuccess) done_.fetch_or(bit, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<uint64_t> done_{0};
};

// moe_block_norm and its backward (block_norm.cu); the fields are the
// arguments of the C calls, checked by the caller.
struct NormArgs {
  const void* residual = nullptr;  // forward only
  const void* y = nullptr;
  const void* gate = nullptr;
  const float* post_w = nullptr;
  const float* pre_w = nullptr;
  int64_t T = 0;
  int H = 0;
  int gate_kind = 0;
  int gate_act = 0;
  float scale = 1.0f;
  float eps = 0.0f;
  void* h = nullptr;  // written by the forward, read by the backward
  void* n = nullptr;
  float* rstd_post = nullptr;
  float* rstd_pre = nullptr;
  // backward
  const void* grad_h = nullptr;
  const void* grad_n = nullptr;
  void* grad_residual = nullptr;
  void* grad_y = nullptr;
  void* grad_gate = nullptr;
  float* grad_post_w = nullptr;
  float* grad_pre_w = nullptr;
  float* partials = nullptr;  // workspace: [2][blocks][H] sums over a block's tokens
};
cudaError_t launch_block_norm(const LaunchCtx& c, const NormArgs& a, bool stream_f32,
                              bool block_f32);
cudaError_t launch_block_norm_backward(const LaunchCtx& c, const NormArgs& a, bool stream_f32,
                                       bool block_f32);
// Blocks of the backward that leave partial sums over tokens: at most this
// many (160 SMs at most, each with as many blocks as its 8192 channels in
// registers make rows, at most kNormMaxBlocksPerSm), and at most one per token.
constexpr int kNormMaxBlocksPerSm = 24;
inline int64_t norm_partial_blocks(int64_t T, int H) {
  int64_t per_sm = (8192 + H - 1) / H;
  if (per_sm > kNormMaxBlocksPerSm) per_sm = kNormMaxBlocksPerSm;
  if (per_sm < 1) per_sm = 1;
  return T < 160 * per_sm ? T : 160 * per_sm;
}

// moe_balance_loss (balance_loss.cu).
struct BalanceArgs {
  const float* scores = nullptr;
  const int32_t* idx = nullptr;
  int64_t T = 0;
  int E = 0, k = 0, func = 0, S = 1;
  const int32_t* seq = nullptr;
  const uint8_t* mask = nullptr;
  float* balance = nullptr;
  float* z = nullptr;
  int32_t* counts = nullptr;
  float* probs = nullptr;
  int32_t* tokens = nullptr;
  void* ws = nullptr;
  // backward
  const float* grad_balance = nullptr;
  const float* grad_z = nullptr;
  const float* w = nullptr;
  const float* grad_w = nullptr;
  float* grad_scores = nullptr;
};
// aligned: whether scores are 16-byte aligned.
size_t balance_workspace_bytes(int64_t T, int E, int S, bool aligned);
cudaError_t launch_balance_loss(const LaunchCtx& c, const BalanceArgs& a);
cudaError_t launch_balance_loss_backward(const LaunchCtx& c, const BalanceArgs& a);

cudaError_t launch_combine_backward(const LaunchCtx& c, const void* grad_out, bool grad_f32,
                                    const void* y, const float* w, const int32_t* pos,
                                    const int32_t* src, int64_t T, int H, int k, int64_t R,
                                    void* grad_y, float* grad_w);

// moe_expert_matvec_fp4 (expert_matvec_fp4.cu).
struct MatvecArgs {
  const void* x = nullptr;
  int64_t num_x = 0;
  const uint8_t* w = nullptr;
  const void* sf = nullptr;
  int sf_type = 0, group = 0;
  const int32_t* offsets = nullptr;
  const int32_t* src = nullptr;
  int E = 1, k = 1;
  int64_t R = 0;
  int K = 0, N = 0, swiglu = 0;
  void* out = nullptr;
  bool out_f32 = false;
};
cudaError_t launch_expert_matvec_fp4(const LaunchCtx& c, const MatvecArgs& a);

// moe_router_gate and its backward (router_gate.cu).
struct RouterArgs {
  const float* scores = nullptr;
  int64_t T = 0;
  int E = 0, k = 0, func = 0;
  const float* bias = nullptr;
  int G = 1, g = 1, group_score = 0;
  bool renorm = true;
  float scale = 1.0f;
  int32_t* idx = nullptr;  // written by the forward, read by the backward
  float* w = nullptr;
  // backward
  const float* grad_w = nullptr;
  const float* add = nullptr;
  float* grad_scores = nullptr;
};
cudaError_t launch_router_gate(const LaunchCtx& c, const RouterArgs& a);
cudaError_t launch_router_gate_backward(const LaunchCtx& c, const RouterArgs& a);

// moe_cast_int8 (cast_int8.cu).
cudaError_t launch_cast_int8(const LaunchCtx& c, const void* x, bool f32, int64_t T, int H,
                             int8_t* out, float* sf);

// moe_expert_matmul_int8 (expert_matmul_int8.cu).
struct MatmulInt8Args {
  const int8_t* x = nullptr;
  const float* x_sf = nullptr;
  int64_t num_x = 0;
  const int8_t* w = nullptr;
  const float* w_sf = nullptr;
  const int32_t* offsets = nullptr;
  const int32_t* src = nullptr;
  int E = 1, k = 1;
  int64_t R = 0;
  int K = 0, N = 0, swiglu = 0;
  void* out = nullptr;
  bool out_f32 = false;
  // test hooks (moe_debug_set): the bound of every wait, and how many stages of weights a
  // CTA asks for
  uint64_t wait_ns = 1000000000ull;
  int64_t stages = INT64_MAX;
};
cudaError_t launch_expert_matmul_int8(const LaunchCtx& c, const MatmulInt8Args& a);
// The form that it takes (MOE_MATMUL_INT8_*), by the sizes alone, and a cluster's CTAs.
cudaError_t expert_matmul_int8_form(const LaunchCtx& c, const MatmulInt8Args& a, int* form,
                                    int* ctas);

}  // namespace moe
