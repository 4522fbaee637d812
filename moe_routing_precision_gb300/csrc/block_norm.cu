// block_norm.cu -- the norms before and after a block, with the block's gate
// and residual scale, and their gradients.
//
// Forward, per token (f32 throughout, each output rounded once):
//   z = y * rsqrt(mean(y^2) + eps) * post_w,  h = r + scale * g * z,
//   n = h * rsqrt(mean(h^2) + eps) * pre_w
// A row stays in registers from its load to its stores, so HBM sees r, y (and
// an elementwise gate) once and h, n once; that traffic bounds it.
//
// Backward, with u = gn * pre_w and c = scale * g * post_w, per token:
//   A = sum u h,  B = sum c y (gh + rho u),  C = sum c y h
//   d  = gh + rho u - h rho^3 A / H
//   D  = sum c d y = B - C rho^3 A / H
//   gy = rho_y c d - y rho_y^3 D / H
// D needs d, which needs A; written through B and C the three sums are taken
// together, so a row costs one reduction over the block instead of two.  (The
// terms of B and of C rho^3 A / H are those that d itself subtracts element by
// element, so this cancels no more than d does.)
#include "block_ops.cuh"

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

// Accesses a thread holds as loaded (a row waits in registers for its norm).
template <class T, int VEC>
struct Raw {
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ void zero() { v = T(); }
  __device__ __forceinline__ void get(float (&f)[VEC]) const { load_elems<1>(&v, f); }
};
template <>
struct Raw<Bf16, 8> {
  uint4 v;
  __device__ __forceinline__ void load(const Bf16* p) { v = ld_once_v4(p); }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&f)[8]) const { unpack8(v, f); }
};
template <>
struct Raw<float, 8> {
  float v[8];
  __device__ __forceinline__ void load(const float* p) { load_elems<8>(p, v); }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = v[i];
  }
};

template <class RT, class YT, int VEC, int NPT, int MAXT>
__global__ void __launch_bounds__(MAXT) block_norm_kernel(const NormArgs a, int tpr) {
  pdl_enter();
  __shared__ float red[2][32];
  const int row_in_block = threadIdx.x / tpr, tid = threadIdx.x - row_in_block * tpr;
  const int wpr = tpr >> 5;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x / tpr) + row_in_block;
  const bool live = t < a.T;
  const int64_t base = t * a.H;
  const bool has_y = a.y != nullptr;

  float h[NPT][VEC];
  Raw<RT, VEC> r_raw[NPT];
  Raw<YT, VEC> y_raw[NPT];
#pragma unroll
  for (int i = 0; i < NPT; ++i) {
    const int c = (i * tpr + tid) * VEC;
    if (has_y) {
      if (live && c < a.H)
        y_raw[i].load(static_cast<const YT*>(a.y) + base + c);
      else
        y_raw[i].zero();
    }
  }
#pragma unroll
  for (int i = 0; i < NPT; ++i) {
    const int c = (i * tpr + tid) * VEC;
    if (live && c < a.H)
      r_raw[i].load(static_cast<const RT*>(a.residual) + base + c);
    else
      r_raw[i].zero();
  }
  if (!has_y) {
#pragma unroll
    for (int i = 0; i < NPT; ++i) r_raw[i].get(h[i]);
  } else {
    float rho = 1.0f;
    if (a.post_w) {
      float ss[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < NPT; ++i) {
        float y[VEC];
        y_raw[i].get(y);
#pragma unroll
        for (int q = 0; q < VEC; ++q) ss[0] = __fmaf_rn(y[q], y[q], ss[0]);
      }
      row_sum<1>(ss, red[0], wpr, row_in_block);
      rho = rsqrt_f32(ss[0] / (float)a.H + a.eps);
      if (live && tid == 0 && a.rstd_post) a.rstd_post[t] = rho;
    }
    float gt[1] = {1.0f};
    if (live && a.gate_kind == MOE_GATE_TOKEN) {
      gt[0] = __ldg(static_cast<const float*>(a.gate) + t);
      gate_values<1>(a, gt);
    }
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
      const int c = (i * tpr + tid) * VEC;
      if (!live || c >= a.H) {
#pragma unroll
        for (int q = 0; q < VEC; ++q) h[i][q] = 0.0f;
        continue;
      }
      float z[VEC], g[VEC];
      y_raw[i].get(z);
      r_raw[i].get(h[i]);
#pragma unroll
      for (int q = 0; q < VEC; ++q) z[q] *= rho;
      if (a.post_w) {
        load_shared_f32<VEC>(a.post_w + c, g);
#pragma unroll
        for (int q = 0; q < VEC; ++q) z[q] *= g[q];
      }
      if (a.gate_kind == MOE_GATE_CHANNEL || a.gate_kind == MOE_GATE_ELEMENT) {
        if (a.gate_kind == MOE_GATE_CHANNEL)
          load_shared_f32<VEC>(static_cast<const float*>(a.gate) + c, g);
        else
          load_elems<VEC>(static_cast<const YT*>(a.gate) + base + c, g);
        gate_values<VEC>(a, g);
#pragma unroll
        for (int q = 0; q < VEC; ++q) z[q] *= g[q];
      }
#pragma unroll
      for (int q = 0; q < VEC; ++q) h[i][q] = __fmaf_rn(a.scale * gt[0], z[q], h[i][q]);
      store_elems<VEC>(static_cast<RT*>(a.h) + base + c, h[i]);
    }
  }
  if (a.pre_w) {
    float ss[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NPT; ++i)
#pragma unroll
      for (int q = 0; q < VEC; ++q) ss[0] = __fmaf_rn(h[i][q], h[i][q], ss[0]);
    row_sum<1>(ss, red[1], wpr, row_in_block);
    const float rho = rsqrt_f32(ss[0] / (float)a.H + a.eps);
    if (live && tid == 0 && a.rstd_pre) a.rstd_pre[t] = rho;
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
      const int c = (i * tpr + tid) * VEC;
      if (!live || c >= a.H) continue;
      float w[VEC];
      load_shared_f32<VEC>(a.pre_w + c, w);
#pragma unroll
      for (int q = 0; q < VEC; ++q) w[q] *= h[i][q] * rho;
      store_elems<VEC>(static_cast<YT*>(a.n) + base + c, w);
    }
  }
}

// The [H] gradients are sums over tokens.  With A[c] = sum_t scale g' d y rho_y,
// where g' is the gate without its per-channel kind,
//   grad_post_w = g A,  grad_gate = post_w A [g (1 - g)]   (per-channel gate g)
// so two sums per channel serve all three: A and sum_t gn h rho.  Each block
// keeps those of its own tokens (the ones congruent to its index) in registers
// and leaves them in partials[sum][block][H]; norm_partials_kernel adds the
// blocks in ascending order.
enum { kPartPost = 0, kPartPre = 1 };

template <class RT, class YT, int VEC, int NPT>
__global__ void __launch_bounds__(1024) block_norm_backward_kernel(const NormArgs a, int tpr) {
  pdl_enter();
  extern __shared__ float smem[];  // 2 x 4 x 32 reduction floats, then the rows' column sums
  const int rows = blockDim.x / tpr;
  const int row_in_block = threadIdx.x / tpr, tid = threadIdx.x - row_in_block * tpr;
  const int wpr = tpr >> 5;
  const bool has_y = a.y != nullptr, pre = a.pre_w != nullptr, post = a.post_w != nullptr;
  const bool gch = a.gate_kind == MOE_GATE_CHANNEL, gel = a.gate_kind == MOE_GATE_ELEMENT;
  const bool gtok = a.gate_kind == MOE_GATE_TOKEN;
  const float inv_h = 1.0f / (float)a.H;

  float s_post[NPT][VEC], s_pre[NPT][VEC];
#pragma unroll
  for (int i = 0; i < NPT; ++i)
#pragma unroll
    for (int q = 0; q < VEC; ++q) s_post[i][q] = s_pre[i][q] = 0.0f;

  const int64_t step = (int64_t)gridDim.x * rows;
  int parity = 0;
  for (int64_t t0 = (int64_t)blockIdx.x * rows; t0 < a.T; t0 += step, parity ^= 1) {
    const int64_t t = t0 + row_in_block;
    const bool live = t < a.T;
    const int64_t base = t * a.H;
    const float rho = live && pre ? __ldg(a.rstd_pre + t) : 0.0f;
    const float rho_y = live && post ? __ldg(a.rstd_post + t) : 1.0f;
    float gt[1] = {1.0f}, gt1[1] = {1.0f};
    if (live && gtok) {
      gt[0] = __ldg(static_cast<const float*>(a.gate) + t);
      gate_values<1>(a, gt, gt1);
    }
    float d[NPT][VEC], h[NPT][VEC], y[NPT][VEC], g[NPT][VEC];
    float sums[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
      const int c = (i * tpr + tid) * VEC;
#pragma unroll
      for (int q = 0; q < VEC; ++q) d[i][q] = h[i][q] = y[i][q] = 0.0f, g[i][q] = 1.0f;
      if (!live || c >= a.H) continue;
      float w[VEC], gn[VEC];
      if (a.grad_h) load_elems<VEC>(static_cast<const RT*>(a.grad_h) + base + c, d[i]);
      if (has_y) {
        load_elems<VEC>(static_cast<const YT*>(a.y) + base + c, y[i]);
        if (gch) load_shared_f32<VEC>(static_cast<const float*>(a.gate) + c, g[i]);
        if (gel) load_elems<VEC>(static_cast<const YT*>(a.gate) + base + c, g[i]);
      }
      if (pre) {
        load_elems<VEC>(static_cast<const RT*>(a.h) + base + c, h[i]);
        load_elems<VEC>(static_cast<const YT*>(a.grad_n) + base + c, gn);
        load_shared_f32<VEC>(a.pre_w + c, w);
#pragma unroll
        for (int q = 0; q < VEC; ++q) {
          const float u = gn[q] * w[q];
          sums[0] = __fmaf_rn(u, h[i][q], sums[0]);
          d[i][q] = __fmaf_rn(rho, u, d[i][q]);
          s_pre[i][q] = __fmaf_rn(gn[q] * rho, h[i][q], s_pre[i][q]);
        }
      }
      if (has_y) {
        if (post) {
          load_shared_f32<VEC>(a.post_w + c, w);
        } else {
#pragma unroll
          for (int q = 0; q < VEC; ++q) w[q] = 1.0f;
        }
        float gv[VEC];
#pragma unroll
        for (int q = 0; q < VEC; ++q) gv[q] = g[i][q];
        if (gch || gel) gate_values<VEC>(a, gv);
#pragma unroll
        for (int q = 0; q < VEC; ++q) {
          const float cy = w[q] * gv[q] * y[i][q];  // without scale and the token's gate
          sums[1] = __fmaf_rn(cy, d[i][q], sums[1]);
          sums[2] = __fmaf_rn(cy, h[i][q], sums[2]);
        }
      }
    }
    // two buffers: the next row's first writes cannot meet this row's reads
    row_sum<3>(sums, smem + parity * 96, wpr, row_in_block);
    const float m = rho * rho * rho * sums[0] * inv_h;
    const float dot = a.scale * (sums[1] - m * sums[2]);  // sum scale g_c d w y
    if (live && gtok && tid == 0) {
      static_cast<float*>(a.grad_gate)[t] = dot * rho_y * gt1[0];
    }
    const float cs = a.scale * gt[0];
    const float my = post ? rho_y * rho_y * rho_y * dot * gt[0] * inv_h : 0.0f;
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
      const int c = (i * tpr + tid) * VEC;
      if (!live || c >= a.H) continue;
#pragma unroll
      for (int q = 0; q < VEC; ++q) d[i][q] = __fmaf_rn(-h[i][q], m, d[i][q]);
      store_elems<VEC>(static_cast<RT*>(a.grad_residual) + base + c, d[i]);
      if (!has_y) continue;
      float w[VEC], gg[VEC], g1[VEC];
      if (gch || gel) gate_values<VEC>(a, g[i], g1);
      if (post) {
        load_shared_f32<VEC>(a.post_w + c, w);
      } else {
#pragma unroll
        for (int q = 0; q < VEC; ++q) w[q] = 1.0f;
      }
#pragma unroll
      for (int q = 0; q < VEC; ++q) {
        const float yn = y[i][q] * rho_y;
        const float dg = a.scale * d[i][q] * w[q] * yn;  // scale d z
        gg[q] = gel ? dg * g1[q] : dg;
        const float b = cs * g[i][q] * d[i][q];
        s_post[i][q] = __fmaf_rn(gel ? b : cs * d[i][q], yn, s_post[i][q]);
        w[q] = __fmaf_rn(rho_y * b, w[q], -y[i][q] * my);
      }
      store_elems<VEC>(static_cast<YT*>(a.grad_y) + base + c, w);
      if (gel) store_elems<VEC>(static_cast<YT*>(a.grad_gate) + base + c, gg);
    }
  }

  // this block's column sums: rows of the block added in order
  float* cols = smem + 192;
  const int64_t plane = (int64_t)gridDim.x * a.H;
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    const bool want = o == kPartPost ? post || gch : pre;
    if (!want) continue;
    float* dst = a.partials + o * plane + (int64_t)blockIdx.x * a.H;
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
      const int c = (i * tpr + tid) * VEC;
      if (c >= a.H) continue;
#pragma unroll
      for (int q = 0; q < VEC; ++q) {
        const float v = o == kPartPost ? s_post[i][q] : s_pre[i][q];
        if (rows == 1)
          dst[c + q] = v;
        else
          cols[(int64_t)row_in_block * a.H + c + q] = v;
      }
    }
    if (rows > 1) {
      __syncthreads();
      for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
        float v = 0.0f;
        for (int r = 0; r < rows; ++r) v += cols[r * a.H + c];
        dst[c] = v;
      }
      __syncthreads();
    }
  }
}

// The channels' sums over the blocks' partials, 32 columns per CTA: warp w adds
// the blocks w, w + 8, ...; then the warps' sums are added in order.
constexpr int kSumWarps = 8;
__global__ void __launch_bounds__(32 * kSumWarps)
    norm_partials_kernel(const NormArgs a, int blocks) {
  pdl_enter();
  __shared__ float part[kSumWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int o = blockIdx.y, c = blockIdx.x * 32 + lane;
  const bool channel = a.gate_kind == MOE_GATE_CHANNEL;
  if (o == kPartPost ? !a.grad_post_w && !channel : !a.grad_pre_w) return;
  float v = 0.0f;
  if (c < a.H) {
    const float* src = a.partials + (int64_t)o * blocks * a.H + c;
#pragma unroll 8
    for (int b = warp; b < blocks; b += kSumWarps) v += src[(int64_t)b * a.H];
  }
  part[warp][lane] = v;
  __syncthreads();
  if (warp != 0 || c >= a.H) return;
  v = 0.0f;
#pragma unroll
  for (int i = 0; i < kSumWarps; ++i) v += part[i][lane];
  if (o == kPartPre) {
    a.grad_pre_w[c] = v;
    return;
  }
  float g = 1.0f, g1 = 1.0f;
  if (channel) {
    g = static_cast<const float*>(a.gate)[c];
    if (a.gate_act == MOE_GATE_ACT_SIGMOID) g = sigmoid_f32(g, &g1);
    static_cast<float*>(a.grad_gate)[c] = v * (a.post_w ? a.post_w[c] : 1.0f) * g1;
  }
  if (a.grad_post_w) a.grad_post_w[c] = v * g;
}

// ---------------------------------------------------------------- the ring
// For rows that come in 16-byte pieces, H <= kRingMaxHidden and many tokens:
// each block takes the rows congruent to its index, and one thread copies whole
// rows ahead of their use into a ring in shared memory (bulk copies counted by
// one barrier per stage), so that the loads never wait for a row's sums.  Every
// thread keeps the same two 8-channel units for all rows, so what depends on
// the channel alone (weights, per-channel gate, the gradients' sums) stays in
// its registers.  Blocks of H / 16 threads; as many per SM as make 512 threads.
constexpr int kRingMaxHidden = 8192;
constexpr int kRingThreads = kRingMaxHidden / 16;
constexpr int kRingMaxStages = 4;
constexpr int kRingHeader = 1024;  // sums and barriers in front of the stages

struct Ring {
  int stages = 0;
  uint32_t stage_bytes = 0;
  uint32_t at[5] = {};  // where each stream's row lies in a stage
};

// 8 elements of a staged row as f32.
__device__ __forceinline__ void stage_elems(const uint8_t* p, int unit, const Bf16*, float (&v)[8]) {
  unpack8(*reinterpret_cast<const uint4*>(p + unit * 16), v);
}
__device__ __forceinline__ void stage_elems(const uint8_t* p, int unit, const float*, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p + unit * 32);
  const float4 b = *reinterpret_cast<const float4*>(p + unit * 32 + 16);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
// 8 elements to a row: f32 as one 32-byte store.
__device__ __forceinline__ void store8(Bf16* p, const float (&v)[8]) { store_elems<8>(p, v); }
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  asm volatile("st.global.cs.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]),
               "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
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
  __device__ __forceinline__ void next(int stages) {
    if (++stage == stages) {
      stage = 0;
      parity ^= 1u;
    }
  }
};
__device__ __forceinline__ void ring_fill(const RingState& r, const Ring& ring, int stage,
                                          const void* const (&src)[5], const uint32_t (&bytes)[5],
                                          int64_t t, int rows) {
  const uint32_t bar = r.bars + stage * 8;
  uint32_t total = 0;
#pragma unroll
  for (int i = 0; i < 5; ++i) total += src[i] ? bytes[i] * rows : 0u;
  mbar_expect(bar, total);
#pragma unroll
  for (int i = 0; i < 5; ++i)
    if (src[i])
      bulk_load(r.stages_at + stage * ring.stage_bytes + ring.at[i],
                static_cast<const uint8_t*>(src[i]) + t * bytes[i], bytes[i] * rows, bar);
}

// post_w * per-channel gate, and pre_w, of this thread's units.
__device__ __forceinline__ void channel_constants(const NormArgs& a, int c, bool in, float (&wg)[8],
                                                  float (&pw)[8]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) wg[q] = 1.0f, pw[q] = 0.0f;
  if (!in) return;
  float v[8];
  if (a.post_w) load_shared_f32<8>(a.post_w + c, wg);
  if (a.gate_kind == MOE_GATE_CHANNEL) {
    load_shared_f32<8>(static_cast<const float*>(a.gate) + c, v);
    gate_values<8>(a, v);
#pragma unroll
    for (int q = 0; q < 8; ++q) wg[q] *= v[q];
  }
  if (a.pre_w) load_shared_f32<8>(a.pre_w + c, pw);
}

// Forward: R consecutive rows per turn of a block, whose sums are reduced
// together.
template <class RT, class YT, bool GEL, int R>
__global__ void __launch_bounds__(kRingThreads, 1)
    norm_ring_kernel(const NormArgs a, const Ring ring, unsigned* err) {
  pdl_enter();
  extern __shared__ __align__(128) uint8_t ring_smem[];
  float* red = reinterpret_cast<float*>(ring_smem);  // 2 x 2 x 16 R sums
  const uint32_t sbase = (uint32_t)__cvta_generic_to_shared(ring_smem);
  RingState rs;
  rs.bars = sbase + kRingHeader - 64;
  rs.stages_at = sbase + kRingHeader;
  const int tid = threadIdx.x, nt = blockDim.x, wpr = nt >> 5;
  const bool has_y = a.y != nullptr, post = a.post_w != nullptr, pre = a.pre_w != nullptr;
  const bool gtok = a.gate_kind == MOE_GATE_TOKEN;
  const void* const src[5] = {a.residual, a.y, GEL ? a.gate : nullptr, nullptr, nullptr};
  const uint32_t rb = (uint32_t)(a.H * sizeof(RT)), yb = (uint32_t)(a.H * sizeof(YT));
  const uint32_t bytes[5] = {rb, yb, yb, 0u, 0u};
  const int64_t step = (int64_t)gridDim.x * R, first = (int64_t)blockIdx.x * R;
  auto fill = [&](int stage, int64_t t) {
    ring_fill(rs, ring, stage, src, bytes, t, a.T - t < R ? (int)(a.T - t) : R);
  };
  if (tid == 0) {
    for (int i = 0; i < ring.stages; ++i) mbar_init(rs.bars + i * 8);
    mbar_init_done();
    for (int i = 0; i < ring.stages; ++i)
      if (first + i * step < a.T) fill(i, first + i * step);
  }
  __syncthreads();
  float wg[2][8], pw[2][8];
  bool in[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = (i * nt + tid) * 8;
    in[i] = c < a.H;
    channel_constants(a, c, in[i], wg[i], pw[i]);
  }
  const float inv_h = 1.0f / (float)a.H;
  // the tokens' gates, loaded one turn ahead
  float next_gt[R];
  auto scalars = [&](int64_t t) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      next_gt[r] = gtok && t + r < a.T ? __ldg(static_cast<const float*>(a.gate) + t + r) : 1.0f;
  };
  scalars(first);
  int buf = 0;
  for (int64_t t = first; t < a.T; t += step, buf ^= 1) {
    float gt[R];
#pragma unroll
    for (int r = 0; r < R; ++r) gt[r] = next_gt[r];
    if (t + step < a.T) scalars(t + step);
    if (gtok) gate_values<R>(a, gt);
    rs.wait(err);
    const uint8_t* st = ring_smem + kRingHeader + rs.stage * ring.stage_bytes;
    // (the second row of a last single one is what the stage held before: its
    // sums are its own and nothing of it is stored)
    float h[R][2][8], z[R][2][8], ss[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      ss[r] = 0.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int u = i * nt + tid;
#pragma unroll
        for (int q = 0; q < 8; ++q) h[r][i][q] = z[r][i][q] = 0.0f;
        if (!in[i]) continue;
        if (has_y) {
          stage_elems(st + ring.at[1] + r * yb, u, static_cast<const YT*>(nullptr), z[r][i]);
#pragma unroll
          for (int q = 0; q < 8; ++q) ss[r] = __fmaf_rn(z[r][i][q], z[r][i][q], ss[r]);
          if (GEL) {
            float g[8];
            stage_elems(st + ring.at[2] + r * yb, u, static_cast<const YT*>(nullptr), g);
            gate_values<8>(a, g);
#pragma unroll
            for (int q = 0; q < 8; ++q) z[r][i][q] *= g[q];
          }
        }
        stage_elems(st + ring.at[0] + r * rb, u, static_cast<const RT*>(nullptr), h[r][i]);
      }
    }
    row_sum<R>(ss, red + buf * 16 * R, wpr, 0);
    // every thread holds its part of the rows: the stage is free
    if (wpr == 1) __syncwarp();
    if (tid == 0 && rs.ok && t + ring.stages * step < a.T) fill(rs.stage, t + ring.stages * step);
    rs.next(ring.stages);
    if (has_y) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float rho = 1.0f;
        if (post) {
          rho = rsqrt_f32(ss[r] * inv_h + a.eps);
          if (tid == 0 && a.rstd_post && t + r < a.T) a.rstd_post[t + r] = rho;
        }
        const float f = a.scale * gt[r] * rho;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            h[r][i][q] = __fmaf_rn(f * wg[i][q], z[r][i][q], h[r][i][q]);
          if (in[i] && t + r < a.T)
            store8(static_cast<RT*>(a.h) + (t + r) * a.H + (i * nt + tid) * 8, h[r][i]);
        }
      }
    }
    if (pre) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        ss[r] = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int q = 0; q < 8; ++q) ss[r] = __fmaf_rn(h[r][i][q], h[r][i][q], ss[r]);
      }
      row_sum<R>(ss, red + (2 + buf) * 16 * R, wpr, 0);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float rho = rsqrt_f32(ss[r] * inv_h + a.eps);
        if (t + r >= a.T) continue;
        if (tid == 0 && a.rstd_pre) a.rstd_pre[t + r] = rho;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int q = 0; q < 8; ++q) h[r][i][q] *= rho * pw[i][q];
          if (in[i])
            store8(static_cast<YT*>(a.n) + (t + r) * a.H + (i * nt + tid) * 8, h[r][i]);
        }
      }
    }
  }
  if (!rs.ok && tid == 0)
    for (int i = 0; i < ring.stages; ++i) (void)mbar_wait(rs.bars + i * 8, rs.parity);
}

template <class RT, class YT, bool GEL>
__global__ void __launch_bounds__(kRingThreads, 1)
    norm_backward_ring_kernel(const NormArgs a, const Ring ring, unsigned* err) {
  pdl_enter();
  extern __shared__ __align__(128) uint8_t ring_smem[];
  float* red = reinterpret_cast<float*>(ring_smem);  // 2 x 3 x 16 sums
  const uint32_t sbase = (uint32_t)__cvta_generic_to_shared(ring_smem);
  RingState rs;
  rs.bars = sbase + kRingHeader - 64;
  rs.stages_at = sbase + kRingHeader;
  const int tid = threadIdx.x, nt = blockDim.x, wpr = nt >> 5;
  const bool has_y = a.y != nullptr, post = a.post_w != nullptr, pre = a.pre_w != nullptr;
  const bool gtok = a.gate_kind == MOE_GATE_TOKEN;
  const void* const src[5] = {a.grad_h, pre ? a.h : nullptr, pre ? a.grad_n : nullptr, a.y,
                              GEL ? a.gate : nullptr};
  const uint32_t rb = (uint32_t)(a.H * sizeof(RT)), yb = (uint32_t)(a.H * sizeof(YT));
  const uint32_t bytes[5] = {rb, rb, yb, yb, yb};
  const int64_t step = gridDim.x;
  if (tid == 0) {
    for (int i = 0; i < ring.stages; ++i) mbar_init(rs.bars + i * 8);
    mbar_init_done();
    for (int i = 0; i < ring.stages; ++i) {
      const int64_t t = blockIdx.x + i * step;
      if (t < a.T) ring_fill(rs, ring, i, src, bytes, t, 1);
    }
  }
  __syncthreads();
  float wg[2][8], pw[2][8], s_post[2][8], s_pre[2][8];
  bool in[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = (i * nt + tid) * 8;
    in[i] = c < a.H;
    channel_constants(a, c, in[i], wg[i], pw[i]);
#pragma unroll
    for (int q = 0; q < 8; ++q) s_post[i][q] = s_pre[i][q] = 0.0f;
  }
  const float inv_h = 1.0f / (float)a.H;
  // the row's scalars, loaded one row ahead
  float next_rho = 0.0f, next_rho_y = 1.0f, next_gt = 1.0f;
  auto scalars = [&](int64_t t) {
    if (pre) next_rho = __ldg(a.rstd_pre + t);
    if (post) next_rho_y = __ldg(a.rstd_post + t);
    if (gtok) next_gt = __ldg(static_cast<const float*>(a.gate) + t);
  };
  if (blockIdx.x < a.T) scalars(blockIdx.x);
  int buf = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += step, buf ^= 1) {
    const float rho = next_rho, rho_y = next_rho_y;
    float gt[1] = {next_gt}, gt1[1] = {1.0f};
    if (t + step < a.T) scalars(t + step);
    if (gtok) gate_values<1>(a, gt, gt1);
    rs.wait(err);
    const uint8_t* st = ring_smem + kRingHeader + rs.stage * ring.stage_bytes;
    float d[2][8], h[2][8], y[2][8], g[2][8];
    float sums[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int u = i * nt + tid;
#pragma unroll
      for (int q = 0; q < 8; ++q) d[i][q] = h[i][q] = y[i][q] = 0.0f, g[i][q] = 1.0f;
      if (!in[i]) continue;
      if (a.grad_h) stage_elems(st + ring.at[0], u, static_cast<const RT*>(nullptr), d[i]);
      if (pre) {
        float gn[8];
        stage_elems(st + ring.at[1], u, static_cast<const RT*>(nullptr), h[i]);
        stage_elems(st + ring.at[2], u, static_cast<const YT*>(nullptr), gn);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float v = gn[q] * pw[i][q];
          sums[0] = __fmaf_rn(v, h[i][q], sums[0]);
          d[i][q] = __fmaf_rn(rho, v, d[i][q]);
          s_pre[i][q] = __fmaf_rn(gn[q] * rho, h[i][q], s_pre[i][q]);
        }
      }
      if (has_y) {
        stage_elems(st + ring.at[3], u, static_cast<const YT*>(nullptr), y[i]);
        if (GEL) {
          stage_elems(st + ring.at[4], u, static_cast<const YT*>(nullptr), g[i]);
        }
        float gv[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) gv[q] = g[i][q];
        if (GEL) gate_values<8>(a, gv);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float cy = (GEL ? wg[i][q] * gv[q] : wg[i][q]) * y[i][q];
          sums[1] = __fmaf_rn(cy, d[i][q], sums[1]);
          sums[2] = __fmaf_rn(cy, h[i][q], sums[2]);
        }
      }
    }
    row_sum<3>(sums, red + buf * 48, wpr, 0);
    // every thread holds its part of the row: the stage is free
    if (wpr == 1) __syncwarp();
    if (tid == 0 && rs.ok && t + ring.stages * step < a.T)
      ring_fill(rs, ring, rs.stage, src, bytes, t + ring.stages * step, 1);
    rs.next(ring.stages);
    const float m = rho * rho * rho * sums[0] * inv_h;
    const float dot = a.scale * (sums[1] - m * sums[2]);
    if (gtok && tid == 0) {
      static_cast<float*>(a.grad_gate)[t] = dot * rho_y * gt1[0];
    }
    const float cs = a.scale * gt[0];
    const float my = post ? rho_y * rho_y * rho_y * dot * gt[0] * inv_h : 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t at = t * a.H + (i * nt + tid) * 8;
#pragma unroll
      for (int q = 0; q < 8; ++q) d[i][q] = __fmaf_rn(-h[i][q], m, d[i][q]);
      if (in[i]) store8(static_cast<RT*>(a.grad_residual) + at, d[i]);
      if (!has_y) continue;
      float gg[8], gy[8], g1[8];
      if (GEL) gate_values<8>(a, g[i], g1);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float yn = y[i][q] * rho_y;
        if (GEL) {
          const float dg = a.scale * d[i][q] * wg[i][q] * yn;  // scale d z
          gg[q] = dg * g1[q];
        }
        const float b = cs * (GEL ? g[i][q] * d[i][q] : d[i][q]);
        s_post[i][q] = __fmaf_rn(b, yn, s_post[i][q]);
        gy[q] = __fmaf_rn(rho_y * b, wg[i][q], -y[i][q] * my);
      }
      if (!in[i]) continue;
      store8(static_cast<YT*>(a.grad_y) + at, gy);
      if (GEL) store8(static_cast<YT*>(a.grad_gate) + at, gg);
    }
  }
  const int64_t plane = (int64_t)gridDim.x * a.H;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (!in[i]) continue;
    float* p = a.partials + (int64_t)blockIdx.x * a.H + (i * nt + tid) * 8;
    if (post || a.gate_kind == MOE_GATE_CHANNEL) store_elems<8>(p, s_post[i]);
    if (pre) store_elems<8>(p + plane, s_pre[i]);
  }
  if (!rs.ok && tid == 0)
    for (int i = 0; i < ring.stages; ++i) (void)mbar_wait(rs.bars + i * 8, rs.parity);
}

// Every tensor's address a multiple of `bytes`, and rows of whole 8-element units.
bool vec_ok(const NormArgs& a, uintptr_t bytes = 16) {
  if (a.H % 8 != 0) return false;
  const void* p[] = {a.residual, a.y, a.h, a.n, a.post_w, a.pre_w, a.grad_h, a.grad_n,
                     a.grad_residual, a.grad_y,
                     a.gate_kind == MOE_GATE_TOKEN ? nullptr : a.gate,
                     a.gate_kind == MOE_GATE_TOKEN ? nullptr : a.grad_gate};
  uintptr_t bits = 0;
  for (const void* q : p) bits |= reinterpret_cast<uintptr_t>(q);
  return (bits & (bytes - 1)) == 0;
}

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

template <class RT, class YT, int VEC, int NPT, int MAXT>
cudaError_t fwd_t(const LaunchCtx& c, const NormArgs& a) {
  const Shape s = row_shape((a.H + VEC - 1) / VEC, NPT);
  const int64_t blocks = (a.T + s.rows - 1) / s.rows;
  if (blocks >= ((int64_t)1 << 31)) return cudaErrorInvalidConfiguration;
  return launch_pdl(block_norm_kernel<RT, YT, VEC, NPT, MAXT>, dim3((unsigned)blocks),
                    s.tpr * s.rows, 0, c.stream, a, s.tpr);
}

cudaError_t launch_partials(const LaunchCtx& c, const NormArgs& a, int blocks) {
  if (!a.grad_post_w && !a.grad_pre_w && a.gate_kind != MOE_GATE_CHANNEL) return cudaSuccess;
  return launch_pdl(norm_partials_kernel, dim3((unsigned)((a.H + 31) / 32), 2), 32 * kSumWarps, 0,
                    c.stream, a, blocks);
}

template <class RT, class YT, int VEC, int NPT>
cudaError_t bwd_t(const LaunchCtx& c, const NormArgs& a) {
  const Shape s = row_shape((a.H + VEC - 1) / VEC, NPT);
  const size_t smem = 192 * sizeof(float) + (s.rows > 1 ? (size_t)s.rows * a.H * sizeof(float) : 0);
  auto* kernel = block_norm_backward_kernel<RT, YT, VEC, NPT>;
  static SmemOptIn opt_in;
  cudaError_t e = opt_in.once(c, kernel);
  if (e != cudaSuccess) return e;
  // blocks per SM, looked up when the shape changes (1 us a call)
  thread_local int known = -1, per_sm = 0;
  if (known != a.H) {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, s.tpr * s.rows, smem);
    if (e != cudaSuccess) return e;
    known = a.H;
  }
  int64_t blocks = (a.T + s.rows - 1) / s.rows;
  const int64_t cap = (int64_t)c.num_sms * (per_sm > 0 ? per_sm : 1);
  if (blocks > cap) blocks = cap;
  const int64_t room = norm_partial_blocks(a.T, a.H);
  if (blocks > room) blocks = room;
  e = launch_pdl(kernel, dim3((unsigned)blocks), s.tpr * s.rows, smem, c.stream, a, s.tpr);
  if (e != cudaSuccess) return e;
  return launch_partials(c, a, (int)blocks);
}

// Rows enough that every SM's ring turns over: below, one block per row has the
// lower latency.
bool ring_ok(const NormArgs& a) {
  return a.H <= kRingMaxHidden && a.T >= 512 && vec_ok(a, 32);
}

template <auto* kernel>
cudaError_t ring_launch(const LaunchCtx& c, const NormArgs& a, int rows,
                        const uint32_t (&row_bytes)[5], int64_t max_blocks, int* blocks_out) {
  Ring ring;
  for (int i = 0; i < 5; ++i) {
    ring.at[i] = ring.stage_bytes;
    ring.stage_bytes += (rows * row_bytes[i] + 127) / 128 * 128;
  }
  const int threads = (a.H + 511) / 512 * 32;
  int per_sm = kRingThreads / threads;
  if (per_sm > 16) per_sm = 16;
  for (;; --per_sm) {  // (1 KB of each block's shared memory is the system's)
    ring.stages = (int)((226u * 1024 / per_sm - 1024 - kRingHeader) / ring.stage_bytes);
    if (ring.stages >= 2 || per_sm == 1) break;
  }
  if (ring.stages > kRingMaxStages) ring.stages = kRingMaxStages;
  const size_t smem = kRingHeader + (size_t)ring.stages * ring.stage_bytes;
  static SmemOptIn opt_in;
  cudaError_t e = opt_in.once(c, kernel);
  if (e != cudaSuccess) return e;
  int64_t blocks = (int64_t)c.num_sms * per_sm;
  if (blocks > max_blocks) blocks = max_blocks;
  *blocks_out = (int)blocks;
  return launch_pdl(kernel, dim3((unsigned)blocks), threads, smem, c.stream, a, ring, c.err);
}

// A ring of at least two stages of `rows` rows fits (H = 8192 with every stream
// in f32 does not).
template <class RT, class YT>
bool ring_fits(const NormArgs& a, int rows, int rt_rows, int yt_rows) {
  return 2 * rows * (size_t)a.H * (rt_rows * sizeof(RT) + yt_rows * sizeof(YT)) <= 200 * 1024;
}

template <class RT, class YT>
cudaError_t fwd_types(const LaunchCtx& c, const NormArgs& a) {
  const bool gel = a.gate_kind == MOE_GATE_ELEMENT;
  const int y_rows = (a.y != nullptr) + gel;
  if (ring_ok(a) && ring_fits<RT, YT>(a, 1, 1, y_rows)) {
    const uint32_t rb = (uint32_t)(a.H * sizeof(RT)), yb = (uint32_t)(a.H * sizeof(YT));
    const uint32_t bytes[5] = {rb, a.y ? yb : 0u, gel ? yb : 0u, 0u, 0u};
    int blocks = 0;
    if (ring_fits<RT, YT>(a, 2, 1, y_rows)) {
      const int64_t room = (a.T + 1) / 2;
      return gel ? ring_launch<norm_ring_kernel<RT, YT, true, 2>>(c, a, 2, bytes, room, &blocks)
                 : ring_launch<norm_ring_kernel<RT, YT, false, 2>>(c, a, 2, bytes, room, &blocks);
    }
    return gel ? ring_launch<norm_ring_kernel<RT, YT, true, 1>>(c, a, 1, bytes, a.T, &blocks)
               : ring_launch<norm_ring_kernel<RT, YT, false, 1>>(c, a, 1, bytes, a.T, &blocks);
  }
  if (vec_ok(a)) {
    const int units = a.H / 8;
    if (units <= 256) return fwd_t<RT, YT, 8, 1, 256>(c, a);
    if (units <= 512) return fwd_t<RT, YT, 8, 2, 256>(c, a);
    if (units <= 1024) return fwd_t<RT, YT, 8, 4, 256>(c, a);
    return fwd_t<RT, YT, 8, 4, 512>(c, a);
  }
  if (a.H <= 1024) return fwd_t<RT, YT, 1, 4, 256>(c, a);
  if (a.H <= 4096) return fwd_t<RT, YT, 1, 4, 1024>(c, a);
  return fwd_t<RT, YT, 1, 16, 1024>(c, a);
}

template <class RT, class YT>
cudaError_t bwd_types(const LaunchCtx& c, const NormArgs& a) {
  const bool gel = a.gate_kind == MOE_GATE_ELEMENT, pre = a.pre_w != nullptr;
  if (ring_ok(a) &&
      ring_fits<RT, YT>(a, 1, (a.grad_h != nullptr) + pre, pre + (a.y != nullptr) + gel)) {
    const uint32_t rb = (uint32_t)(a.H * sizeof(RT)), yb = (uint32_t)(a.H * sizeof(YT));
    const uint32_t bytes[5] = {a.grad_h ? rb : 0u, pre ? rb : 0u, pre ? yb : 0u, a.y ? yb : 0u,
                               gel ? yb : 0u};
    int blocks = 0;
    const int64_t room = norm_partial_blocks(a.T, a.H);
    const cudaError_t e =
        gel ? ring_launch<norm_backward_ring_kernel<RT, YT, true>>(c, a, 1, bytes, room, &blocks)
            : ring_launch<norm_backward_ring_kernel<RT, YT, false>>(c, a, 1, bytes, room, &blocks);
    return e == cudaSuccess ? launch_partials(c, a, blocks) : e;
  }
  if (vec_ok(a)) {
    if (a.H <= 8192) return bwd_t<RT, YT, 8, 1>(c, a);
    return bwd_t<RT, YT, 8, 2>(c, a);
  }
  if (a.H <= 4096) return bwd_t<RT, YT, 1, 4>(c, a);
  return bwd_t<RT, YT, 1, 16>(c, a);
}

}  // namespace

cudaError_t launch_block_norm(const LaunchCtx& c, const NormArgs& a, bool stream_f32,
                              bool block_f32) {
  if (stream_f32)
    return block_f32 ? fwd_types<float, float>(c, a) : fwd_types<float, Bf16>(c, a);
  return block_f32 ? fwd_types<Bf16, float>(c, a) : fwd_types<Bf16, Bf16>(c, a);
}

cudaError_t launch_block_norm_backward(const LaunchCtx& c, const NormArgs& a, bool stream_f32,
                                       bool block_f32) {
  if (stream_f32)
    return block_f32 ? bwd_types<float, float>(c, a) : bwd_types<float, Bf16>(c, a);
  return block_f32 ? bwd_types<Bf16, float>(c, a) : bwd_types<Bf16, Bf16>(c, a);
}

}  // namespace moe
