// combine_backward.cu -- gradients of the weighted combine.
//
// With out[t] = sum_j w[t,j] y[pos[t,j]]:
//   grad_y[pos[t,j]] = w[t,j] * grad_out[t]      (f32 product, one rounding to bf16)
//   grad_w[t,j]      = <grad_out[t], y[pos[t,j]]> (f32)
// Every byte moves once: grad_out and y in, grad_y out, so HBM bounds it: 8192
// tokens, H = 7168, k = 8 (2.0 GB) take 297 us, 6.7 TB/s, 99 % of a plain copy.
//
// One CTA per token.  A thread walks the row in 16-byte slices of 8 channels;
// for each slice it holds grad_out in registers and issues the loads of up to
// 8 routed rows before it uses any, so 8 gathers of 16 bytes are in flight per
// thread.  The k dot products stay in registers until the row is done; one
// shuffle and shared-memory reduction in a fixed order then writes them.
#include "block/block_ops.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 8;
constexpr int kZeroRows = 8;  // rows a warp looks at

template <class GT>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(
    const GT* __restrict__ go, const uint16_t* __restrict__ y, const float* __restrict__ w,
    const int32_t* __restrict__ pos, const int32_t* __restrict__ src, int64_t T, int H, int k,
    int64_t R, uint16_t* __restrict__ gy, float* __restrict__ gw, unsigned* err) {
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x;
  if (t >= T) {
    // the CTAs past the tokens zero the rows no copy lands on (whole runs at the
    // ends of the experts' segments: few rows per warp spread a run)
    const int64_t r0 = ((t - T) * kWarps + warp) * kZeroRows;
    const int64_t r = r0 + lane;
    unsigned m = __ballot_sync(0xFFFFFFFFu, lane < kZeroRows && r < R && __ldg(src + r) < 0);
    while (m) {
      const int i = __ffs(m) - 1;
      m &= m - 1;
      uint16_t* q = gy + (r0 + i) * H;
      for (int c = lane * 8; c < H; c += 256) st_stream_v4(q + c, make_uint4(0, 0, 0, 0));
    }
    return;
  }
  __shared__ float part[kWarps][kBatch];
  const GT* grow = go + t * H;
  bool bad = false;
  for (int j0 = 0; j0 < k; j0 += kBatch) {
    int64_t row[kBatch];  // element offset of the routed row, negative: no copy
    float wj[kBatch], dot[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      row[b] = -1;
      wj[b] = 0.0f;
      dot[b] = 0.0f;
      if (j0 + b < k) {
        const int32_t r = __ldg(pos + t * k + j0 + b);
        if (r >= R) bad = true;
        if (r >= 0 && r < R) {
          row[b] = (int64_t)r * H;
          wj[b] = __ldg(w + t * k + j0 + b);
        }
      }
    }
    for (int c = threadIdx.x * 8; c < H; c += kThreads * 8) {
      uint4 v[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (row[b] >= 0) v[b] = ld_stream_v4(y + row[b] + c);
      float g[8];
      load_elems<8>(grow + c, g);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (row[b] < 0) continue;
        float yv[8];
        unpack8(v[b], yv);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot[b] = __fmaf_rn(g[i], yv[i], dot[b]);
        st_stream_v4(gy + row[b] + c,
                     make_uint4(pack_bf16x2_rn(wj[b] * g[0], wj[b] * g[1]),
                                pack_bf16x2_rn(wj[b] * g[2], wj[b] * g[3]),
                                pack_bf16x2_rn(wj[b] * g[4], wj[b] * g[5]),
                                pack_bf16x2_rn(wj[b] * g[6], wj[b] * g[7])));
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const float s = warp_sum(dot[b]);
      if (lane == 0) part[warp][b] = s;
    }
    __syncthreads();
    if (threadIdx.x < kBatch && j0 + (int)threadIdx.x < k) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) s += part[i][threadIdx.x];
      gw[t * k + j0 + threadIdx.x] = s;
    }
    __syncthreads();
  }
  if (bad && threadIdx.x == 0) flag_error(err, MOE_DEVERR_POS_RANGE);
}

template <class GT>
cudaError_t launch_t(const LaunchCtx& c, const void* go, const void* y, const float* w,
                     const int32_t* pos, const int32_t* src, int64_t T, int H, int k, int64_t R,
                     void* gy, float* gw) {
  const int64_t zero = src ? (R + kZeroRows * kWarps - 1) / (kZeroRows * kWarps) : 0;
  const int64_t blocks = T + zero;
  if (blocks == 0) return cudaSuccess;
  if (blocks >= ((int64_t)1 << 31)) return cudaErrorInvalidConfiguration;
  return launch_pdl(combine_backward_kernel<GT>, dim3((unsigned)blocks), kThreads, 0, c.stream,
                    static_cast<const GT*>(go), static_cast<const uint16_t*>(y), w, pos, src, T, H,
                    k, R, static_cast<uint16_t*>(gy), gw, c.err);
}

}  // namespace

cudaError_t launch_combine_backward(const LaunchCtx& c, const void* grad_out, bool grad_f32,
                                    const void* y, const float* w, const int32_t* pos,
                                    const int32_t* src, int64_t T, int H, int k, int64_t R,
                                    void* grad_y, float* grad_w) {
  return grad_f32 ? launch_t<float>(c, grad_out, y, w, pos, src, T, H, k, R, grad_y, grad_w)
                  : launch_t<Bf16>(c, grad_out, y, w, pos, src, T, H, k, R, grad_y, grad_w);
}

}  // namespace moe
