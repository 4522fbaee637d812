// expert_matmul_int8.cu -- products of routed 8-bit rows with their expert's 8-bit
// weights.
//
//   o[r, m] = (sum_c x[src(r), c] * w[e(r), m, c]) * x_sf[src(r)] * w_sf[e(r), m]
//
// The simple form: a warp per run of up to 4 rows of one expert and 4 outputs, each
// lane 16 channels at a time, four products per dp4a.
#include "block/block_ops.cuh"

namespace moe {
namespace {

constexpr int kRows = 4, kOuts = 4, kWarps = 8;

__global__ void __launch_bounds__(kWarps * 32)
    expert_matmul_simple_kernel(const MatmulInt8Args a, unsigned* err) {
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e = blockIdx.y;
  int64_t lo = 0, hi = a.R;
  if (a.offsets != nullptr) {
    lo = a.offsets[e], hi = a.offsets[e + 1];
    if (lo < 0 || hi > a.R) flag_error(err, MOE_DEVERR_POS_RANGE);
    if (lo < 0) lo = 0;
    if (hi > a.R) hi = a.R;
  }
  const int M = a.swiglu ? 2 * a.N : a.N;
  const int per = a.swiglu ? kOuts / 2 : kOuts;
  const int n0 = (blockIdx.x * kWarps + warp) * per;
  if (n0 >= a.N) return;
  int m[kOuts];
#pragma unroll
  for (int j = 0; j < kOuts; ++j) {
    const int n = n0 + (a.swiglu ? j / 2 : j);
    m[j] = (n < a.N ? n : a.N - 1) + (a.swiglu && (j & 1) ? a.N : 0);
  }
  for (int64_t r0 = lo; r0 < hi; r0 += kRows) {
    int64_t s[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      s[i] = -1;
      if (r0 + i >= hi) continue;
      s[i] = r0 + i;
      if (a.src != nullptr) s[i] = a.src[r0 + i] < 0 ? -1 : a.src[r0 + i] / a.k;
      if (s[i] >= a.num_x) {
        flag_error(err, MOE_DEVERR_POS_RANGE);
        s[i] = -1;
      }
    }
    int acc[kRows][kOuts] = {};
    for (int c = lane * 16; c < a.K; c += 512) {
      uint4 xv[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        xv[i] = s[i] >= 0 ? ld_v4(a.x + s[i] * a.K + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < kOuts; ++j) {
        const uint4 wv = ld_v4(a.w + ((int64_t)e * M + m[j]) * a.K + c);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          acc[i][j] = __dp4a((int)wv.x, (int)xv[i].x, acc[i][j]);
          acc[i][j] = __dp4a((int)wv.y, (int)xv[i].y, acc[i][j]);
          acc[i][j] = __dp4a((int)wv.z, (int)xv[i].z, acc[i][j]);
          acc[i][j] = __dp4a((int)wv.w, (int)xv[i].w, acc[i][j]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      float o[kOuts];
#pragma unroll
      for (int j = 0; j < kOuts; ++j) {
        const int sum = (int)__reduce_add_sync(0xFFFFFFFFu, acc[i][j]);
        o[j] = s[i] >= 0 ? (float)sum * a.x_sf[s[i]] * a.w_sf[(int64_t)e * M + m[j]] : 0.0f;
      }
      if (r0 + i >= hi || lane >= per || n0 + lane >= a.N) continue;
      float v = o[0];
#pragma unroll
      for (int j = 0; j < kOuts; ++j)
        if (!a.swiglu && lane == j) v = o[j];
      if (a.swiglu) {
        const float g = lane ? o[2] : o[0], u = lane ? o[3] : o[1];
        v = g / (1.0f + expf(-g)) * u;
      }
      const int64_t at = (r0 + i) * a.N + n0 + lane;
      if (a.out_f32)
        static_cast<float*>(a.out)[at] = v;
      else
        static_cast<uint16_t*>(a.out)[at] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
  }
}

}  // namespace

cudaError_t launch_expert_matmul_int8(const LaunchCtx& c, const MatmulInt8Args& a) {
  const int per = kWarps * (a.swiglu ? kOuts / 2 : kOuts);
  return launch_pdl(expert_matmul_simple_kernel, dim3((unsigned)((a.N + per - 1) / per), a.E),
                    kWarps * 32, 0, c.stream, a, c.err);
}

}  // namespace moe
