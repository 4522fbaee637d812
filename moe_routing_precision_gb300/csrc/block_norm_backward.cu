// block_norm_backward.cu -- gradients of the norms before and after a block.
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
//
// Measured: 8192 tokens, H = 7168, f32 stream, bf16 block, gate per channel (1.06
// GB): 161 us, 6.5 TB/s, 97 % of a plain copy (two rows of 86 KB in flight per
// SM); 321 us with one block per row and no ring.  What bounds the other types is the
// chain of a row (its sums) and the instructions: all bf16 125 us, 83 %.  Widths that
// are no multiple of 8 go element by element, 8192 tokens, all bf16 : f32 stream: H =
// 1001 40 : 42 us, 2047 67 : 67, 7161 356 : 377.  Above 8192 rows go through the kernel
// without the ring, whose threads' sums do not fit their registers: 4096 tokens, H =
// 12288 342 : 379, 16384 470 : 516 (their bytes 89 : 134 and 119 : 178).
#include "block/block_norm.cuh"
#include "known.cuh"

#include <cooperative_groups.h>

#include <utility>

namespace cg = cooperative_groups;

namespace moe {
namespace {

// The [H] gradients are sums over tokens.  With A[c] = sum_t scale g' d y rho_y,
// where g' is the gate without its per-channel kind,
//   grad_post_w = g A,  grad_gate = post_w A [g (1 - g)]   (per-channel gate g)
// so two sums per channel serve all three: A and sum_t gn h rho.  Each block
// keeps those of its own tokens (the ones congruent to its index) in registers
// and leaves them in partials[sum][block][H]; norm_partials_kernel adds the
// blocks in ascending order.
enum { kPartPost = 0, kPartPre = 1 };

// rho^3 x.  One factor at a time: the cube alone leaves f32's range for rows of
// magnitude 2^42 and more, and for rows below eps where eps is below 2^-85; x has
// the row's magnitude, so the products do not.
__device__ __forceinline__ float cubed(float rho, float x) { return rho * x * rho * rho; }

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
    const float m = cubed(rho, sums[0] * inv_h);
    const float dot = a.scale * (sums[1] - m * sums[2]);  // sum scale g_c d w y
    if (live && gtok && tid == 0) {
      static_cast<float*>(a.grad_gate)[t] = dot * rho_y * gt1[0];
    }
    const float cs = a.scale * gt[0];
    const float my = post ? cubed(rho_y, dot * gt[0] * inv_h) : 0.0f;
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
// the blocks w, w + 32, ... of the CTA's part; then the warps' sums are added in
// order.  Narrow rows leave up to 24 partials per SM and few columns: there a
// cluster of SPLIT CTAs shares the blocks, and its first CTA adds the others'
// sums in order through distributed shared memory.  (H = 256, 16384 tokens, the
// whole backward: 36 us with one CTA of 8 warps per 32 columns.)
constexpr int kSumWarps = 32, kSumSplit = 8;
template <int SPLIT>
__global__ void __launch_bounds__(32 * kSumWarps)
    norm_partials_kernel(const NormArgs a, int blocks) {
  pdl_enter();
  __shared__ float part[kSumWarps][33];
  __shared__ float whole[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int o = blockIdx.y, c = blockIdx.x * 32 + lane, rank = blockIdx.z;
  const bool channel = a.gate_kind == MOE_GATE_CHANNEL;
  if (o == kPartPost ? !a.grad_post_w && !channel : !a.grad_pre_w) return;  // the whole cluster
  float v = 0.0f;
  if (c < a.H) {
    const int b0 = blocks * rank / SPLIT, b1 = blocks * (rank + 1) / SPLIT;
    const float* src = a.partials + (int64_t)o * blocks * a.H + c;
#pragma unroll 8
    for (int b = b0 + warp; b < b1; b += kSumWarps) v += src[(int64_t)b * a.H];
  }
  part[warp][lane] = v;
  __syncthreads();
  if (warp == 0) {
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < kSumWarps; ++i) v += part[i][lane];
    if (SPLIT > 1) whole[lane] = v;
  }
  if (SPLIT > 1) {
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    if (rank == 0 && warp == 0) {
#pragma unroll
      for (int i = 1; i < SPLIT; ++i) v += *cluster.map_shared_rank(&whole[lane], i);
    }
    cluster.sync();  // no CTA leaves while its sums are read
  }
  if (rank != 0 || warp != 0 || c >= a.H) return;
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

// Starts the copies of channels [c0, c1) of row t of every stream into a stage
// (sizes: bytes per element).
__device__ __forceinline__ void ring_fill_piece(const RingState& r, const Ring& ring, int stage,
                                                const void* const (&src)[5],
                                                const uint32_t (&sizes)[5], int64_t t, int H,
                                                int c0, int c1, unsigned* err) {
  const uint32_t bar = r.bars + stage * 8;
  const uint32_t dst = r.stages_at + stage * ring.stage_bytes;
  uint32_t bytes[5], total = 0;
  int64_t from[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    bytes[i] = 0;
    if (src[i] == nullptr) continue;
    from[i] = (t * H + c0) * sizes[i];
    bytes[i] = (uint32_t)(c1 - c0) * sizes[i];
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

// ALL: rows that fill the threads, with every input: no conditions between the
// loads (H = 7168, 8192 tokens, bf16, two units: 127 us; 134 with them).
// P: stages per row.  Two (U = 2, V = 8, one unit of every thread each) where two
// whole rows do not fit: H = 7168, all f32, element gate, 4096 tokens 162 us; 251
// without the ring.  Whole rows where they fit (half rows take two turns of the
// copying thread: bf16, 8192 tokens, two units 127 : 134 us).
template <class RT, class YT, bool GEL, int V, int U, int NT, int P, bool ALL>
__global__ void __launch_bounds__(ring_max_threads(U, NT), ring_min_blocks(V, U, NT))
    norm_backward_ring_kernel(const NormArgs a, const Ring ring, unsigned* err) {
  pdl_enter();
  extern __shared__ __align__(128) uint8_t ring_smem[];
  float* red = reinterpret_cast<float*>(ring_smem);  // 2 x 3 x 32 sums
  const uint32_t sbase = (uint32_t)__cvta_generic_to_shared(ring_smem);
  RingState rs;
  rs.bars = sbase + kRingHeader - 64;
  rs.stages_at = sbase + kRingHeader;
  const int tid = threadIdx.x, nt = NT && V == 1 ? NT : blockDim.x, wpr = nt >> 5;
  const bool has_y = ALL || a.y != nullptr, pre = ALL || a.pre_w != nullptr;
  const bool post = a.post_w != nullptr, has_gh = ALL || a.grad_h != nullptr;
  const bool gtok = a.gate_kind == MOE_GATE_TOKEN;
  const void* const src[5] = {a.grad_h, pre ? a.h : nullptr, pre ? a.grad_n : nullptr, a.y,
                              GEL ? a.gate : nullptr};
  const uint32_t rb = (uint32_t)(a.H * sizeof(RT)), yb = (uint32_t)(a.H * sizeof(YT));
  const uint32_t bytes[5] = {rb, rb, yb, yb, yb};
  // (with an element gate and two units the pairs of registers cost spills: 4096
  // tokens, H = 7168, f32: 162 us, in pairs 170)
  constexpr bool kPairs = !(GEL && U == 2);
  const int64_t step = gridDim.x;
  // piece n of this block's rows (P each) into a stage
  auto fill_piece = [&](int stage, int n) {
    const int64_t t = blockIdx.x + n / P * step;
    const int half = nt * V, c0 = n % P ? half : 0, c1 = n % P ? a.H : half;
    if (t < a.T)
      ring_fill_piece(rs, ring, stage, src,
                      {sizeof(RT), sizeof(RT), sizeof(YT), sizeof(YT), sizeof(YT)}, t, a.H, c0, c1,
                      err);
  };
  if (tid == 0) {
    for (int i = 0; i < ring.stages; ++i) mbar_init(rs.bars + i * 8);
    mbar_init_done();
    for (int i = 0; i < ring.stages; ++i) {
      const int64_t t = blockIdx.x + i * step;
      if (P > 1)
        fill_piece(i, i);
      else if (t < a.T)
        ring_fill<V>(rs, ring, ring_smem, i, src, bytes, t, 1, a.T, err);
    }
  }
  __syncthreads();
  float wg[U][V], pw[U][V], s_post[U][V], s_pre[U][V];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    channel_constants<V>(a, (i * nt + tid) * V, wg[i], pw[i]);
#pragma unroll
    for (int q = 0; q < V; ++q) s_post[i][q] = s_pre[i][q] = 0.0f;
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
  int buf = 0, piece = 0;  // piece: this row's first
  for (int64_t t = blockIdx.x; t < a.T; t += step, buf ^= 1, piece += P) {
    const float rho = next_rho, rho_y = next_rho_y;
    float gt[1] = {next_gt}, gt1[1] = {1.0f};
    if (t + step < a.T) scalars(t + step);
    if (gtok) gate_values<1>(a, gt, gt1);
    rs.wait(err);
    const uint8_t* st = ring_smem + kRingHeader + rs.stage * ring.stage_bytes;
    const int stage0 = rs.stage;
    const uint32_t r_off = V == 1 ? (uint32_t)(t * rb) & 15u : 0u;
    const uint32_t y_off = V == 1 ? (uint32_t)(t * yb) & 15u : 0u;
    float d[U][V], h[U][V], y[U][V], g[U][V];
    float sum2[3][2] = {};
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int c = (i * nt + tid) * V;
#pragma unroll
      for (int q = 0; q < V; ++q) d[i][q] = h[i][q] = y[i][q] = 0.0f, g[i][q] = 1.0f;
      if (P > 1 && i > 0) {
        rs.next(ring.stages);
        rs.wait(err);
        st = ring_smem + kRingHeader + rs.stage * ring.stage_bytes;
      }
      const int at_c = P > 1 ? tid * V : c;  // a piece's channels lie at its stage's start
      if (!ALL && c >= a.H) continue;
      if (has_gh)
        stage_elems<V>(st + ring.at[0] + r_off, at_c, static_cast<const RT*>(nullptr), d[i]);
      if (pre) {
        float gn[V];
        stage_elems<V>(st + ring.at[1] + r_off, at_c, static_cast<const RT*>(nullptr), h[i]);
        stage_elems<V>(st + ring.at[2] + y_off, at_c, static_cast<const YT*>(nullptr), gn);
        float v[V];
        mul_v<kPairs>(v, gn, pw[i]);
        dot_v<kPairs>(sum2[0], v, h[i]);
        fma_v<kPairs>(d[i], rho, v);
        mul_v<kPairs>(gn, rho, gn);
        fma_v<kPairs>(s_pre[i], gn, h[i]);
      }
      if (has_y) {
        stage_elems<V>(st + ring.at[3] + y_off, at_c, static_cast<const YT*>(nullptr), y[i]);
        if (GEL) stage_elems<V>(st + ring.at[4] + y_off, at_c, static_cast<const YT*>(nullptr), g[i]);
        float cy[V];
        mul_v<kPairs>(cy, wg[i], y[i]);
        if (GEL) {
          float gv[V];
#pragma unroll
          for (int q = 0; q < V; ++q) gv[q] = g[i][q];
          gate_values<V>(a, gv);
          mul_v<kPairs>(cy, cy, gv);
        }
        dot_v<kPairs>(sum2[1], cy, d[i]);
        dot_v<kPairs>(sum2[2], cy, h[i]);
      }
    }
    float sums[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) sums[i] = sum2[i][0] + sum2[i][1];
    row_sum<3>(sums, red + buf * 96, wpr, 0);
    // every thread holds its part of the row: the stage is free
    if (wpr == 1) __syncwarp();
    if (P > 1) {
      if (tid == 0 && rs.ok) {
#pragma unroll 1
        for (int i = 0; i < P; ++i) fill_piece(i ? rs.stage : stage0, piece + i + ring.stages);
      }
    } else if (tid == 0 && rs.ok && t + ring.stages * step < a.T)
      ring_fill<V>(rs, ring, ring_smem, rs.stage, src, bytes, t + ring.stages * step, 1, a.T,
                   err);
    rs.next(ring.stages);
    const float m = cubed(rho, sums[0] * inv_h);
    const float dot = a.scale * (sums[1] - m * sums[2]);
    if (gtok && tid == 0) static_cast<float*>(a.grad_gate)[t] = dot * rho_y * gt1[0];
    const float cs = a.scale * gt[0];
    const float my = post ? cubed(rho_y, dot * gt[0] * inv_h) : 0.0f;
    const int64_t at = t * a.H + tid * V;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const bool in = ALL || (i * nt + tid) * V < a.H;
      const int64_t ci = at + i * nt * V;
      fma_v<kPairs>(d[i], -m, h[i]);
      if (in) store_row<V>(static_cast<RT*>(a.grad_residual) + ci, d[i]);
      if (!has_y) continue;
      float gg[V], gy[V], g1[V], yn[V], b[V];
      if (GEL) gate_values<V>(a, g[i], g1);
      mul_v<kPairs>(yn, rho_y, y[i]);
      if (GEL) {
        mul_v<kPairs>(gg, d[i], wg[i]);
        mul_v<kPairs>(gg, gg, yn);
        mul_v<kPairs>(gg, a.scale, gg);  // scale d z
        mul_v<kPairs>(gg, gg, g1);
        mul_v<kPairs>(b, g[i], d[i]);
        mul_v<kPairs>(b, cs, b);
      } else {
        mul_v<kPairs>(b, cs, d[i]);
      }
      fma_v<kPairs>(s_post[i], b, yn);
      mul_v<kPairs>(b, rho_y, b);
      mul_v<kPairs>(gy, -my, y[i]);
      fma_v<kPairs>(gy, b, wg[i]);
      if (!in) continue;
      store_row<V>(static_cast<YT*>(a.grad_y) + ci, gy);
      if (GEL) store_row<V>(static_cast<YT*>(a.grad_gate) + ci, gg);
    }
  }
  const int64_t plane = (int64_t)gridDim.x * a.H;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int c = (i * nt + tid) * V;
    if (c >= a.H) continue;
    float* p = a.partials + (int64_t)blockIdx.x * a.H + c;
    if (post || a.gate_kind == MOE_GATE_CHANNEL) store_elems<V>(p, s_post[i]);
    if (pre) store_elems<V>(p + plane, s_pre[i]);
  }
  rs.drain(ring.stages);
}

cudaError_t launch_partials(const LaunchCtx& c, const NormArgs& a, int blocks) {
  if (!a.grad_post_w && !a.grad_pre_w && a.gate_kind != MOE_GATE_CHANNEL) return cudaSuccess;
  const unsigned cols = (unsigned)((a.H + 31) / 32);
  // a cluster where one CTA's warps would add more than 16 partials each
  if (blocks <= 16 * kSumWarps)
    return launch_pdl(norm_partials_kernel<1>, dim3(cols, 2, 1), 32 * kSumWarps, 0, c.stream, a,
                      blocks);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cols, 2, kSumSplit);
  cfg.blockDim = 32 * kSumWarps;
  cfg.stream = c.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = kSumSplit;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, norm_partials_kernel<kSumSplit>, a, blocks);
}

template <class RT, class YT, int VEC, int NPT>
cudaError_t bwd_t(const LaunchCtx& c, const NormArgs& a) {
  const Shape s = row_shape((a.H + VEC - 1) / VEC, NPT);
  const size_t smem = 192 * sizeof(float) + (s.rows > 1 ? (size_t)s.rows * a.H * sizeof(float) : 0);
  auto* kernel = block_norm_backward_kernel<RT, YT, VEC, NPT>;
  static SmemOptIn opt_in;
  cudaError_t e = opt_in.once(kernel);
  if (e != cudaSuccess) return e;
  // blocks per SM, looked up once for each device and width (1 us a call)
  static Known<std::pair<int, int>, int> known;
  int per_sm = 0;
  if (!known.find({c.device, a.H}, &per_sm)) {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, s.tpr * s.rows, smem);
    if (e != cudaSuccess) return e;
    known.put({c.device, a.H}, per_sm);
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

template <class RT, class YT, bool GEL>
void bwd_bytes(const NormArgs& a, uint32_t (&bytes)[5]) {
  const uint32_t rb = (uint32_t)(a.H * sizeof(RT)), yb = (uint32_t)(a.H * sizeof(YT));
  const uint32_t b[5] = {a.grad_h ? rb : 0u, a.pre_w ? rb : 0u, a.pre_w ? yb : 0u,
                         a.y ? yb : 0u, GEL ? yb : 0u};
  for (int i = 0; i < 5; ++i) bytes[i] = b[i];
}

// The backward through the ring; false if it does not fit.
template <class RT, class YT, bool GEL, int V, int U, int NT, int P, bool ALL>
bool bwd_ring(const LaunchCtx& c, const NormArgs& a, cudaError_t* e) {
  uint32_t bytes[5];
  bwd_bytes<RT, YT, GEL>(a, bytes);
  // of a stage: the first piece is the largest
  const int first = P > 1 ? (a.H + 32 * V * U - 1) / (32 * V * U) * 32 * V : a.H;
  for (int i = 0; i < 5; ++i) bytes[i] = bytes[i] / a.H * first;
  const RingShape s = ring_shape<V, U, NT>(a.H, 1, bytes, P + 1);
  if (!s.ring.stages) return false;
  int blocks = 0;
  *e = ring_launch<norm_backward_ring_kernel<RT, YT, GEL, V, U, NT, P, ALL>>(
      c, a, s, norm_partial_blocks(a.T, a.H), &blocks);
  if (*e == cudaSuccess) *e = launch_partials(c, a, blocks);
  return true;
}

// Units of 8 channels per thread and threads, us, f32 stream and bf16 block / all
// bf16 / the former with an element gate, at 8192 tokens (the last: 4096):
//   H = 256 (32768 tokens), 1024, 2048: one unit by a tenth over two
//   H = 2304: one 63 / 56 / 40, two 58 / 48 / 47     3584: 85 / 68 / 55, 90 / 61 / 64
//   4096: 95 / 74 / 62, 105 / 68 / 83                5120: 117 / 86 / 83, 128 / 108 / 100
//   6144: 147 / 116 / 96, 141 / 114 / 113            7168: 161 / 126 / 113, 166 / 130 / 123
// So one unit, except up to 4096 where an SM holds six rows that way, and around 6144 (768 threads of 80 registers) without an
// element gate.  Only rows that fill the threads have the forms of one unit above
// 2048.
template <class RT, class YT, bool GEL>
bool bwd_ring_8(const LaunchCtx& c, const NormArgs& a, cudaError_t* e) {
  const bool all = a.y && a.pre_w && a.grad_h;
  const bool all1 = all && a.H % 256 == 0, all2 = all && a.H % 512 == 0;
  if (a.H <= 2048)
    return all1 ? bwd_ring<RT, YT, GEL, 8, 1, 0, 1, true>(c, a, e)
                : bwd_ring<RT, YT, GEL, 8, 1, 0, 1, false>(c, a, e);
  if (all1) {
    if (a.H <= 4096) {
      uint32_t bytes[5];
      bwd_bytes<RT, YT, GEL>(a, bytes);
      const RingShape two = ring_shape<8, 2, 0>(a.H, 1, bytes);
      if ((GEL || two.per_sm * two.ring.stages < 6) &&
          bwd_ring<RT, YT, GEL, 8, 1, 512, 1, true>(c, a, e))
        return true;
    } else if (a.H <= 5120) {
      if (bwd_ring<RT, YT, GEL, 8, 1, 640, 1, true>(c, a, e)) return true;
    } else if (a.H <= 6144) {
      if constexpr (GEL)
        if (bwd_ring<RT, YT, GEL, 8, 1, 768, 1, true>(c, a, e)) return true;
    } else if (a.H <= 7168) {
      if (bwd_ring<RT, YT, GEL, 8, 1, 896, 1, true>(c, a, e)) return true;
    }
  }
  if (all2 ? bwd_ring<RT, YT, GEL, 8, 2, 0, 1, true>(c, a, e)
           : bwd_ring<RT, YT, GEL, 8, 2, 0, 1, false>(c, a, e))
    return true;
  // (two rows of the other types fit at any width)
  if constexpr (sizeof(RT) + sizeof(YT) > (GEL ? 4 : 6))
    return all2 ? bwd_ring<RT, YT, GEL, 8, 2, 0, 2, true>(c, a, e)
                : bwd_ring<RT, YT, GEL, 8, 2, 0, 2, false>(c, a, e);
  return false;
}
template <class RT, class YT, bool GEL>
bool bwd_ring_vec(const LaunchCtx& c, const NormArgs& a, int vec, cudaError_t* e) {
  if (vec == 8) return bwd_ring_8<RT, YT, GEL>(c, a, e);
  // the smallest block that holds the row; the next larger one, us at 8192 tokens of
  // f32 streams and bf16 blocks, at an earlier step: H = 250: 32 : 48, 1001: 47 : 58,
  // 2047: 72 : 107
  if (a.H <= 256) return bwd_ring<RT, YT, GEL, 1, 4, 64, 1, false>(c, a, e);
  if (a.H <= 1024) return bwd_ring<RT, YT, GEL, 1, 8, 128, 1, false>(c, a, e);
  if (a.H <= 2048) return bwd_ring<RT, YT, GEL, 1, 8, 256, 1, false>(c, a, e);
  if (a.H <= 4096) return bwd_ring<RT, YT, GEL, 1, 8, 512, 1, false>(c, a, e);
  return bwd_ring<RT, YT, GEL, 1, 16, 512, 1, false>(c, a, e);
}

template <class RT, class YT>
cudaError_t bwd_types(const LaunchCtx& c, const NormArgs& a) {
  const int vec = ring_vec(a);
  if (vec) {
    cudaError_t e;
    if (a.gate_kind == MOE_GATE_ELEMENT ? bwd_ring_vec<RT, YT, true>(c, a, vec, &e)
                                        : bwd_ring_vec<RT, YT, false>(c, a, vec, &e))
      return e;
  }
  if (vec_ok(a)) {
    if (a.H <= 8192) return bwd_t<RT, YT, 8, 1>(c, a);
    return bwd_t<RT, YT, 8, 2>(c, a);
  }
  if (a.H <= 4096) return bwd_t<RT, YT, 1, 4>(c, a);
  return bwd_t<RT, YT, 1, 16>(c, a);
}

}  // namespace

cudaError_t launch_block_norm_backward(const LaunchCtx& c, const NormArgs& a, bool stream_f32,
                                       bool block_f32) {
  if (stream_f32)
    return block_f32 ? bwd_types<float, float>(c, a) : bwd_types<float, Bf16>(c, a);
  return block_f32 ? bwd_types<Bf16, float>(c, a) : bwd_types<Bf16, Bf16>(c, a);
}

}  // namespace moe
