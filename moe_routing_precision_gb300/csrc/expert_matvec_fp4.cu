// expert_matvec_fp4.cu -- products of routed rows with their expert's 4-bit
// weights (E2M1 codes, one scale per group of channels), for decode batches.
//
//   o[r, m] = sum_g w_sf[e, m, g] * sum_{c in g} x[src(r), c] * E2M1(w[e, m, c])
//
// With few rows per expert the weights are read once for little arithmetic,
// so HBM bounds it: K/2 bytes of codes and K/group scales per output.
//
// One CTA takes up to kRows rows of one expert (the route map left them
// adjacent) and a tile of outputs; each warp computes one output at a time,
// its lanes walking the weight row 16 bytes (32 codes) apiece.
#include "block_ops.cuh"

#include <cuda_fp16.h>

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 8;
constexpr int kOutPerWarp = 2;

// The two E2M1 codes of byte `i` of w as f16x2, element 0 (the low nibble) in
// the low half: the hardware conversion, exact.
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t w, int i) {
  const uint16_t b = (uint16_t)((w >> (8 * i)) & 0xFFu);
  uint32_t r;
  asm("{\n .reg .b8 t;\n cvt.u8.u16 t, %1;\n cvt.rn.f16x2.e2m1x2 %0, t;\n}" : "=r"(r) : "h"(b));
  return r;
}

// The item-th run of up to kRows rows of one expert, experts ascending; every
// thread of the block calls it.  Empty (n == 0) past the last.
struct Item {
  int e, r0, n;
};
__device__ __forceinline__ Item find_item(const MatvecArgs& a, int item, Item* shared,
                                          unsigned* err) {
  if (a.offsets == nullptr) {
    const int64_t r0 = (int64_t)item * kRows;
    const int64_t left = a.R - r0;
    return Item{0, (int)r0, left < 0 ? 0 : left < kRows ? (int)left : kRows};
  }
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    if (lane == 0) *shared = Item{0, 0, 0};
    __syncwarp();
    int before = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      int lo = 0, hi = 0;
      if (e < a.E) {
        lo = __ldg(a.offsets + e);
        hi = __ldg(a.offsets + e + 1);
        if (lo < 0 || hi > a.R) {
          flag_error(err, MOE_DEVERR_POS_RANGE);
          lo = lo < 0 ? 0 : lo;
          hi = hi > a.R ? (int)a.R : hi;
        }
      }
      const int runs = hi > lo ? (hi - lo + kRows - 1) / kRows : 0;
      int sum = runs;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += v;
      }
      const int first = before + sum - runs;
      if (item >= first && item < first + runs) {
        const int r0 = lo + (item - first) * kRows;
        *shared = Item{e, r0, hi - r0 < kRows ? hi - r0 : kRows};
      }
      before += __shfl_sync(0xFFFFFFFFu, sum, 31);
      if (item < before) break;
    }
  }
  __syncthreads();
  return *shared;
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

__device__ __forceinline__ float scale_at(const MatvecArgs& a, int64_t i) {
  if (a.sf_type == MOE_WSF_F32) return __ldg(static_cast<const float*>(a.sf) + i);
  const uint32_t b = __ldg(static_cast<const uint8_t*>(a.sf) + i);
  // 2^(b - 127): the exponent field itself, and 2^-127 as the denormal it is
  return __uint_as_float(b ? b << 23 : 0x00400000u);
}

__global__ void __launch_bounds__(kThreads)
    expert_matvec_kernel(const MatvecArgs a, unsigned* err) {
  pdl_enter();
  __shared__ Item shared;
  __shared__ int64_t xrow[kRows];
  const Item it = find_item(a, blockIdx.y, &shared, err);
  if (it.n <= 0) return;
  if (threadIdx.x < kRows)
    xrow[threadIdx.x] = (int)threadIdx.x < it.n ? source_row(a, it.r0 + threadIdx.x, err) : -1;
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int M = a.swiglu ? 2 * a.N : a.N, blocks = a.K / 32;
  const uint16_t* x = static_cast<const uint16_t*>(a.x);
  for (int i = 0; i < kOutPerWarp; ++i) {
    const int n = (blockIdx.x * kWarps + warp) * kOutPerWarp + i;
    if (n >= a.N) return;
    float acc[2][kRows];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int r = 0; r < kRows; ++r) acc[h][r] = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1 && !a.swiglu) break;
      const int64_t m = (int64_t)it.e * M + n + h * a.N;
      for (int b = lane; b < blocks; b += 32) {
        const uint4 q = ld_stream_v4(a.w + m * (a.K / 2) + b * 16);
        const uint32_t qw[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int c = b * 32 + half * 16;
          const float s = scale_at(a, m * (a.K / a.group) + c / a.group);
          float w[16];
#pragma unroll
          for (int p = 0; p < 8; ++p) {
            const uint32_t f = e2m1x2_to_f16x2(qw[half * 2 + p / 4], p % 4);
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f));
            w[2 * p] = v.x;
            w[2 * p + 1] = v.y;
          }
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            if (r >= it.n || xrow[r] < 0) continue;
            float v[16];
            const uint16_t* xp = x + xrow[r] * a.K + c;
            unpack16(ld_v4(xp), ld_v4(xp + 8), v);
            float d = 0.0f;
#pragma unroll
            for (int j = 0; j < 16; ++j) d = __fmaf_rn(v[j], w[j], d);
            acc[h][r] = __fmaf_rn(s, d, acc[h][r]);
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (r >= it.n) break;
      float o = warp_sum(acc[0][r]);
      if (a.swiglu) {
        const float up = warp_sum(acc[1][r]);
        o = o / (1.0f + expf(-o)) * up;
      }
      if (lane == 0) {
        const int64_t at = (int64_t)(it.r0 + r) * a.N + n;
        if (a.out_f32)
          static_cast<float*>(a.out)[at] = o;
        else
          static_cast<uint16_t*>(a.out)[at] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
      }
    }
  }
}

}  // namespace

cudaError_t launch_expert_matvec_fp4(const LaunchCtx& c, const MatvecArgs& a) {
  const int per_cta = kWarps * kOutPerWarp;
  // runs of rows: at most one per row, and at most one short run per expert
  int64_t items = a.offsets ? a.E + a.R / kRows : (a.R + kRows - 1) / kRows;
  if (items > a.R) items = a.R;
  if (items > 65535) return cudaErrorInvalidConfiguration;
  return launch_pdl(expert_matvec_kernel,
                    dim3((unsigned)((a.N + per_cta - 1) / per_cta), (unsigned)items), kThreads, 0,
                    c.stream, a, c.err);
}

}  // namespace moe
