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

// g and, for the backward, g' of VEC gate values.
template <int VEC>
__device__ __forceinline__ void gate_values(const NormArgs& a, float (&g)[VEC]) {
  if (a.gate_act == MOE_GATE_ACT_SIGMOID) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) g[i] = sigmoid_f32(g[i]);
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
      rho = 1.0f / sqrtf(ss[0] / (float)a.H + a.eps);
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
    const float rho = 1.0f / sqrtf(ss[0] / (float)a.H + a.eps);
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

// The three [H] gradients are sums over tokens: each block keeps the sums of
// its own tokens (those congruent to its index) in registers, leaves them in
// partials[output][block][H], and norm_partials_kernel adds the blocks in
// ascending order.
enum { kPartPost = 0, kPartGate = 1, kPartPre = 2 };

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
  const bool sig = a.gate_act == MOE_GATE_ACT_SIGMOID;
  const float inv_h = 1.0f / (float)a.H;

  float s_post[NPT][VEC], s_gate[NPT][VEC], s_pre[NPT][VEC];
#pragma unroll
  for (int i = 0; i < NPT; ++i)
#pragma unroll
    for (int q = 0; q < VEC; ++q) s_post[i][q] = s_gate[i][q] = s_pre[i][q] = 0.0f;

  const int64_t step = (int64_t)gridDim.x * rows;
  int parity = 0;
  for (int64_t t0 = (int64_t)blockIdx.x * rows; t0 < a.T; t0 += step, parity ^= 1) {
    const int64_t t = t0 + row_in_block;
    const bool live = t < a.T;
    const int64_t base = t * a.H;
    const float rho = live && pre ? __ldg(a.rstd_pre + t) : 0.0f;
    const float rho_y = live && post ? __ldg(a.rstd_post + t) : 1.0f;
    float gt[1] = {1.0f};
    if (live && gtok) {
      gt[0] = __ldg(static_cast<const float*>(a.gate) + t);
      gate_values<1>(a, gt);
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
        if (gch || gel) gate_values<VEC>(a, g[i]);
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
#pragma unroll
        for (int q = 0; q < VEC; ++q) {
          const float cy = w[q] * g[i][q] * y[i][q];  // without scale and the token's gate
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
      const float gp = sig ? gt[0] * (1.0f - gt[0]) : 1.0f;
      static_cast<float*>(a.grad_gate)[t] = dot * rho_y * gp;
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
      float w[VEC], gg[VEC];
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
        gg[q] = gel && sig ? dg * g[i][q] * (1.0f - g[i][q]) : dg;
        s_gate[i][q] += dg;
        const float b = cs * g[i][q] * d[i][q];
        s_post[i][q] = __fmaf_rn(b, yn, s_post[i][q]);
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
  for (int o = 0; o < 3; ++o) {
    const bool want = o == kPartPost ? post : o == kPartGate ? gch : pre;
    if (!want) continue;
    float* dst = a.partials + o * plane + (int64_t)blockIdx.x * a.H;
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
      const int c = (i * tpr + tid) * VEC;
      if (c >= a.H) continue;
#pragma unroll
      for (int q = 0; q < VEC; ++q) {
        const float v = o == kPartPost ? s_post[i][q] : o == kPartGate ? s_gate[i][q] : s_pre[i][q];
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

// grad[c] = sum over the blocks' partials, 32 columns per CTA: warp w adds the
// blocks w, w + 8, ...; then the warps' sums are added in order.
constexpr int kSumWarps = 8;
__global__ void __launch_bounds__(32 * kSumWarps)
    norm_partials_kernel(const NormArgs a, int blocks) {
  pdl_enter();
  __shared__ float part[kSumWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int o = blockIdx.y, c = blockIdx.x * 32 + lane;
  float* out = o == kPartPost ? a.grad_post_w
               : o == kPartGate
                   ? (a.gate_kind == MOE_GATE_CHANNEL ? static_cast<float*>(a.grad_gate) : nullptr)
                   : a.grad_pre_w;
  if (out == nullptr) return;
  float v = 0.0f;
  if (c < a.H) {
    const float* src = a.partials + (int64_t)o * blocks * a.H + c;
#pragma unroll 4
    for (int b = warp; b < blocks; b += kSumWarps) v += src[(int64_t)b * a.H];
  }
  part[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < a.H) {
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < kSumWarps; ++i) v += part[i][lane];
    if (o == kPartGate && a.gate_act == MOE_GATE_ACT_SIGMOID) {
      const float g = sigmoid_f32(static_cast<const float*>(a.gate)[c]);
      v *= g * (1.0f - g);
    }
    out[c] = v;
  }
}

bool vec_ok(const NormArgs& a) {
  if (a.H % 8 != 0) return false;
  const void* p[] = {a.residual, a.y, a.h, a.n, a.post_w, a.pre_w, a.grad_h, a.grad_n,
                     a.grad_residual, a.grad_y,
                     a.gate_kind == MOE_GATE_TOKEN ? nullptr : a.gate,
                     a.gate_kind == MOE_GATE_TOKEN ? nullptr : a.grad_gate};
  uintptr_t bits = 0;
  for (const void* q : p) bits |= reinterpret_cast<uintptr_t>(q);
  return (bits & 15u) == 0;
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

template <class RT, class YT, int VEC, int NPT>
cudaError_t bwd_t(const LaunchCtx& c, const NormArgs& a) {
  const Shape s = row_shape((a.H + VEC - 1) / VEC, NPT);
  const size_t smem = 192 * sizeof(float) + (s.rows > 1 ? (size_t)s.rows * a.H * sizeof(float) : 0);
  auto* kernel = block_norm_backward_kernel<RT, YT, VEC, NPT>;
  cudaError_t e = allow_max_dynamic_smem(kernel);
  if (e != cudaSuccess) return e;
  int per_sm = 0;
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, s.tpr * s.rows, smem);
  if (e != cudaSuccess) return e;
  int64_t blocks = (a.T + s.rows - 1) / s.rows;
  const int64_t cap = (int64_t)c.num_sms * (per_sm > 0 ? per_sm : 1);
  if (blocks > cap) blocks = cap;
  if (blocks > kNormMaxPartials) blocks = kNormMaxPartials;
  e = launch_pdl(kernel, dim3((unsigned)blocks), s.tpr * s.rows, smem, c.stream, a, s.tpr);
  if (e != cudaSuccess) return e;
  if (!a.grad_post_w && !a.grad_pre_w && a.gate_kind != MOE_GATE_CHANNEL) return cudaSuccess;
  return launch_pdl(norm_partials_kernel, dim3((unsigned)((a.H + 31) / 32), 3), 32 * kSumWarps, 0,
                    c.stream, a, (int)blocks);
}

template <class RT, class YT>
cudaError_t fwd_types(const LaunchCtx& c, const NormArgs& a) {
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
  if (vec_ok(a)) {
    if (a.H <= 8192) return bwd_t<RT, YT, 8, 1>(c, a);
    return bwd_t<RT, YT, 8, 2>(c, a);
  }
  if (a.H <= 1024) return bwd_t<RT, YT, 1, 4>(c, a);
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
