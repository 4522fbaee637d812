// block_norm.cu -- the norms before and after a block, with the block's gate and
// residual scale.
//
// Forward, per token (f32 throughout, each output rounded once):
//   z = y * rsqrt(mean(y^2) + eps) * post_w,  h = r + scale * g * z,
//   n = h * rsqrt(mean(h^2) + eps) * pre_w
// A row stays in registers from its load to its stores, so HBM sees r, y (and
// an elementwise gate) once and h, n once; that traffic bounds it.
//
// Measured: 16384 tokens, H = 7168, bf16, gated per token (940 MB): 140 us, 6.7
// TB/s, 98 % of a plain copy, through the ring with two rows per turn (176 us
// with one block per row, whose loads stop while a row is summed; 206 us with
// the ring but one row per turn and single bf16 conversions).  One token, H =
// 4096: 2.9 us.  8192 tokens of widths that are no multiple of 8, all bf16 : f32 stream:
// H = 1001 17 : 19 us, 2047 38 : 41, 7161 115 : 123.  Above 8192, one block per row, 4096
// tokens: H = 12288 80 : 143 us, 16384 137 : 178 (their bytes 59 : 89 and 79 : 119).
#include "block/block_norm.cuh"

namespace moe {
namespace {

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

// Forward: R consecutive rows per turn of a block, whose sums are reduced
// together.  ALL: rows that fill the threads, with y and the pre-norm: no
// conditions between the loads.
template <class RT, class YT, bool GEL, int R, int V, int U, int NT, bool ALL>
__global__ void __launch_bounds__(ring_max_threads(U, NT), ring_min_blocks(V, U, NT))
    norm_ring_kernel(const NormArgs a, const Ring ring, unsigned* err) {
  pdl_enter();
  extern __shared__ __align__(128) uint8_t ring_smem[];
  float* red = reinterpret_cast<float*>(ring_smem);  // 2 x 2 x 32 R sums
  const uint32_t sbase = (uint32_t)__cvta_generic_to_shared(ring_smem);
  RingState rs;
  rs.bars = sbase + kRingHeader - 64;
  rs.stages_at = sbase + kRingHeader;
  const int tid = threadIdx.x, nt = NT && V == 1 ? NT : blockDim.x, wpr = nt >> 5;
  const bool has_y = ALL || a.y != nullptr, pre = ALL || a.pre_w != nullptr;
  const bool post = a.post_w != nullptr;
  const bool gtok = a.gate_kind == MOE_GATE_TOKEN;
  const void* const src[5] = {a.residual, a.y, GEL ? a.gate : nullptr, nullptr, nullptr};
  const uint32_t rb = (uint32_t)(a.H * sizeof(RT)), yb = (uint32_t)(a.H * sizeof(YT));
  const uint32_t bytes[5] = {rb, yb, yb, 0u, 0u};
  // (pairs of registers do not pay at 72 of them: H = 7168 139.5 us, in pairs 142)
  constexpr bool kPairs = ALL && NT < 896;
  const int64_t step = (int64_t)gridDim.x * R, first = (int64_t)blockIdx.x * R;
  auto fill = [&](int stage, int64_t t) {
    ring_fill<V>(rs, ring, ring_smem, stage, src, bytes, t, a.T - t < R ? (int)(a.T - t) : R, a.T,
                 err);
  };
  if (tid == 0) {
    for (int i = 0; i < ring.stages; ++i) mbar_init(rs.bars + i * 8);
    mbar_init_done();
    for (int i = 0; i < ring.stages; ++i)
      if (first + i * step < a.T) fill(i, first + i * step);
  }
  __syncthreads();
  float wg[U][V], pw[U][V];
#pragma unroll
  for (int i = 0; i < U; ++i) channel_constants<V>(a, (i * nt + tid) * V, wg[i], pw[i]);
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
    const uint32_t r_off = V == 1 ? (uint32_t)(t * rb) & 15u : 0u;
    const uint32_t y_off = V == 1 ? (uint32_t)(t * yb) & 15u : 0u;
    // (the second row of a last single one is what the stage held before: its
    // sums are its own and nothing of it is stored)
    float h[R][U][V], z[R][U][V], ss2[R][2] = {}, ss[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint8_t* r_row = st + ring.at[0] + r_off + r * rb;
      const uint8_t* y_row = st + ring.at[1] + y_off + r * yb;
      const uint8_t* g_row = st + ring.at[2] + y_off + r * yb;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int c = (i * nt + tid) * V;
#pragma unroll
        for (int q = 0; q < V; ++q) h[r][i][q] = z[r][i][q] = 0.0f;
        if (!ALL && c >= a.H) continue;
        if (has_y) {
          stage_elems<V>(y_row, c, static_cast<const YT*>(nullptr), z[r][i]);
          dot_v<kPairs>(ss2[r], z[r][i], z[r][i]);
          if (GEL) {
            float g[V];
            stage_elems<V>(g_row, c, static_cast<const YT*>(nullptr), g);
            gate_values<V>(a, g);
            mul_v<kPairs>(z[r][i], g, z[r][i]);
          }
        }
        stage_elems<V>(r_row, c, static_cast<const RT*>(nullptr), h[r][i]);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) ss[r] = ss2[r][0] + ss2[r][1];
    row_sum<R>(ss, red + buf * 32 * R, wpr, 0);
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
        RT* out = static_cast<RT*>(a.h) + (t + r) * a.H + tid * V;
#pragma unroll
        for (int i = 0; i < U; ++i) {
          mul_v<kPairs>(z[r][i], f, z[r][i]);
          fma_v<kPairs>(h[r][i], wg[i], z[r][i]);
          if ((ALL || (i * nt + tid) * V < a.H) && t + r < a.T) store_row<V>(out + i * nt * V, h[r][i]);
        }
      }
    }
    if (pre) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        ss2[r][0] = ss2[r][1] = 0.0f;
#pragma unroll
        for (int i = 0; i < U; ++i) dot_v<kPairs>(ss2[r], h[r][i], h[r][i]);
        ss[r] = ss2[r][0] + ss2[r][1];
      }
      row_sum<R>(ss, red + (2 + buf) * 32 * R, wpr, 0);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float rho = rsqrt_f32(ss[r] * inv_h + a.eps);
        if (t + r >= a.T) continue;
        if (tid == 0 && a.rstd_pre) a.rstd_pre[t + r] = rho;
        YT* out = static_cast<YT*>(a.n) + (t + r) * a.H + tid * V;
#pragma unroll
        for (int i = 0; i < U; ++i) {
          mul_v<kPairs>(h[r][i], rho, h[r][i]);
          mul_v<kPairs>(h[r][i], pw[i], h[r][i]);
          if (ALL || (i * nt + tid) * V < a.H) store_row<V>(out + i * nt * V, h[r][i]);
        }
      }
    }
  }
  rs.drain(ring.stages);
}

template <class RT, class YT, int VEC, int NPT, int MAXT>
cudaError_t fwd_t(const LaunchCtx& c, const NormArgs& a) {
  const Shape s = row_shape((a.H + VEC - 1) / VEC, NPT);
  const int64_t blocks = (a.T + s.rows - 1) / s.rows;
  if (blocks >= ((int64_t)1 << 31)) return cudaErrorInvalidConfiguration;
  return launch_pdl(block_norm_kernel<RT, YT, VEC, NPT, MAXT>, dim3((unsigned)blocks),
                    s.tpr * s.rows, 0, c.stream, a, s.tpr);
}

// Elements from which the forward goes through the ring; below, one block per
// row has the lower latency.  Ring against rows, us: H = 7168: 4.5 : 4.6 at
// T = 152, 7.2 : 9.3 at 512, 39.9 : 46.8 at 4096; H = 2048: 3.6 : 3.4 at 512,
// 5.5 : 5.6 at 1024, 7.7 : 8.6 at 2048; H = 512: 5.3 : 5.5 at 4096, 13.3 : 18.5 at
// 16384; H = 256: 4.0 : 3.1 at 4096, 7.4 : 7.5 at 16384, 25 : 29 at 65536.  Widths
// that are no multiple of 8, whose rows go element by element: H = 1155: 3.8 : 3.9
// at 256, 4.1 : 4.3 at 512, 6.3 : 7.8 at 1024.
constexpr int64_t kFwdRingElems = (int64_t)1 << 21, kFwdRingOddElems = (int64_t)1 << 19;

// The forward through the ring; false if it does not fit.
template <class RT, class YT, bool GEL, int V, int U, int NT, bool ALL>
bool fwd_ring(const LaunchCtx& c, const NormArgs& a, cudaError_t* e) {
  const uint32_t rb = (uint32_t)(a.H * sizeof(RT)), yb = (uint32_t)(a.H * sizeof(YT));
  const uint32_t bytes[5] = {rb, a.y ? yb : 0u, GEL ? yb : 0u, 0u, 0u};
  int blocks = 0;
  const RingShape two = ring_shape<V, U, NT>(a.H, 2, bytes);
  if (two.ring.stages) {
    *e = ring_launch<norm_ring_kernel<RT, YT, GEL, 2, V, U, NT, ALL>>(c, a, two, (a.T + 1) / 2,
                                                                      &blocks);
    return true;
  }
  // the widest rows of this form, where two stages of two rows may not fit
  constexpr int kWidest = NT ? NT * 8 : U == 1 ? 256 : ALL ? 1024 : kRingMaxHidden;
  if constexpr (V == 8 && 4 * kWidest * (sizeof(RT) + (GEL ? 2 : 1) * sizeof(YT)) > 220 * 1024) {
    const RingShape one = ring_shape<V, U, NT>(a.H, 1, bytes);
    if (one.ring.stages) {
      *e = ring_launch<norm_ring_kernel<RT, YT, GEL, 1, V, U, NT, ALL>>(c, a, one, a.T, &blocks);
      return true;
    }
  }
  return false;
}
template <class RT, class YT, bool GEL>
bool fwd_ring_vec(const LaunchCtx& c, const NormArgs& a, int vec, cudaError_t* e) {
  // one or two units of 8 channels per thread, us at 16384 tokens: H = 64: 7.3 :
  // 8.3, 256: 7.3 : 8.4, 512: 13.3 : 10.3, 1024: 27.4 : 23.4, 2048: 49.4 : 46.8.  From
  // 4096 on one unit and one block per SM (bf16, then with an element gate): 4096: 86
  // : 95, 116 : 105; 5120: 102 : 118, 136 : 167; 6144: 120 : 121, 159 : 169; 7168: 140 :
  // 143, 183 : 199; 8192: 160 : 180, 206 : 207; f32 rows alike within 2 %.  The form
  // without conditions, two units: 512: 8.4 : 10.0, 1024: 22.3 : 23.0, element gate
  // 2048: 59 : 54, 6144: 136 : 122, so it is taken up to 1024.
  if (vec == 8) {
    const bool all = a.y && a.pre_w;
    if (a.H <= 256)
      return all && a.H == 256 ? fwd_ring<RT, YT, GEL, 8, 1, 0, true>(c, a, e)
                               : fwd_ring<RT, YT, GEL, 8, 1, 0, false>(c, a, e);
    if (all && a.H % 256 == 0 && a.H > (GEL ? 4096 : 4095)) {
      if (a.H <= 4096) return fwd_ring<RT, YT, GEL, 8, 1, 512, true>(c, a, e);
      if (a.H <= 5120) return fwd_ring<RT, YT, GEL, 8, 1, 640, true>(c, a, e);
      if (a.H <= 6144) return fwd_ring<RT, YT, GEL, 8, 1, 768, true>(c, a, e);
      if (a.H <= 7168) return fwd_ring<RT, YT, GEL, 8, 1, 896, true>(c, a, e);
      return fwd_ring<RT, YT, GEL, 8, 1, 1024, true>(c, a, e);
    }
    return all && (a.H == 512 || a.H == 1024) ? fwd_ring<RT, YT, GEL, 8, 2, 0, true>(c, a, e)
                                              : fwd_ring<RT, YT, GEL, 8, 2, 0, false>(c, a, e);
  }
  // the smallest block that holds the row; the next larger one, us at 8192 tokens, all
  // bf16: H = 250: 8.5 : 31, 1001: 16 : 32, 2047: 36 : 61 (a block's threads past the
  // row are idle, and fewer blocks fit an SM)
  if (a.H <= 256) return fwd_ring<RT, YT, GEL, 1, 4, 64, false>(c, a, e);
  if (a.H <= 1024) return fwd_ring<RT, YT, GEL, 1, 8, 128, false>(c, a, e);
  if (a.H <= 2048) return fwd_ring<RT, YT, GEL, 1, 8, 256, false>(c, a, e);
  if (a.H <= 4096) return fwd_ring<RT, YT, GEL, 1, 8, 512, false>(c, a, e);
  return fwd_ring<RT, YT, GEL, 1, 16, 512, false>(c, a, e);
}

template <class RT, class YT>
cudaError_t fwd_types(const LaunchCtx& c, const NormArgs& a) {
  int vec = ring_vec(a);
  if (a.T * a.H < (vec == 8 ? kFwdRingElems : kFwdRingOddElems)) vec = 0;
  if (vec) {
    cudaError_t e;
    if (a.gate_kind == MOE_GATE_ELEMENT ? fwd_ring_vec<RT, YT, true>(c, a, vec, &e)
                                        : fwd_ring_vec<RT, YT, false>(c, a, vec, &e))
      return e;
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

}  // namespace

cudaError_t launch_block_norm(const LaunchCtx& c, const NormArgs& a, bool stream_f32,
                              bool block_f32) {
  if (stream_f32)
    return block_f32 ? fwd_types<float, float>(c, a) : fwd_types<float, Bf16>(c, a);
  return block_f32 ? fwd_types<Bf16, float>(c, a) : fwd_types<Bf16, Bf16>(c, a);
}

}  // namespace moe
