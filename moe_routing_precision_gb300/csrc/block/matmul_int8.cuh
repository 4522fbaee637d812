// matmul_int8.cuh -- what the forms of the experts' 8-bit products share: the conversion to
// f16, the list of tiles, the gather and the weights' tensor map.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "tcgen05.cuh"

namespace moe {

// Long runs of rows, by pairs of CTAs (expert_matmul_int8_pair.cu).
cudaError_t launch_expert_matmul_int8_pair(const LaunchCtx& c, const MatmulInt8Args& a);

namespace {

constexpr int kBlockK = 128;  // channels per stage

// Four 8-bit integers to f16, in pairs: u = v + 128 in the low mantissa bits of 1024 is
// 1024 + u, and 1152 off is v, exactly.
__device__ __forceinline__ void int8x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  w ^= 0x80808080u;
  const uint32_t p = __byte_perm(w, 0x64646464u, 0x4140), q = __byte_perm(w, 0x64646464u, 0x4342);
  const __half2 off = __half2half2(__ushort_as_half(0x6480));
  const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&p), off);
  const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&q), off);
  lo = *reinterpret_cast<const uint32_t*>(&a);
  hi = *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ uint4 lds_v4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts_v4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int c, int r,
                                        uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(dst),
      "l"(map), "r"(c), "r"(r), "r"(bar)
      : "memory");
}

// Row r's row of x, or -1 for a row of zeros.
__device__ __forceinline__ int64_t source_row(const MatmulInt8Args& a, int64_t r, unsigned* err) {
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

__device__ __forceinline__ void store_out(const MatmulInt8Args& a, int64_t at, float v) {
  if (a.out_f32)
    static_cast<float*>(a.out)[at] = v;
  else
    static_cast<uint16_t*>(a.out)[at] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// COLS columns of one thread's output channel into rows row + j (j < rows), channel ch.
// Two rows share a conversion, and the address goes from row to row (a product per store
// and a conversion each took the tile of 256 x 256, K = 2048, longer than its products).
template <bool F32, int COLS>
__device__ __forceinline__ void store_column(const MatmulInt8Args& a, const float (&v)[COLS],
                                             int64_t row, int rows, int ch) {
  const int64_t at = row * a.N + ch;
  if constexpr (F32) {
    float* o = static_cast<float*>(a.out) + at;
#pragma unroll
    for (int j = 0; j < COLS; ++j, o += a.N)
      if (j < rows) *o = v[j];
  } else {
    uint16_t* o = static_cast<uint16_t*>(a.out) + at;
#pragma unroll
    for (int j = 0; j < COLS; j += 2) {
      const uint32_t w = pack_bf16x2_rn(v[j], v[j + 1]);
      if (j < rows) *o = (uint16_t)w;
      o += a.N;
      if (j + 1 < rows) *o = (uint16_t)(w >> 16);
      o += a.N;
    }
  }
}
// The scales of 16 rows from shared memory (16-byte aligned).
__device__ __forceinline__ void load_scales16(const float* s, float (&v)[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float4 f = *reinterpret_cast<const float4*>(s + 4 * q);
    v[4 * q] = f.x, v[4 * q + 1] = f.y, v[4 * q + 2] = f.z, v[4 * q + 3] = f.w;
  }
}

// Stage and phase of a ring, step by step.
struct Ring {
  int i = 0;
  uint32_t phase = 0;
  template <int N>
  __device__ __forceinline__ void next(int by = 1) {
    i += by;
    if (i >= N) i -= N, phase ^= 1u;
  }
};

// One item of the work: a tile of an expert's outputs for a run of its rows.
struct Item {
  int e, tile, n;  // n rows from r0
  int64_t r0;
};

// Every expert's rows in equal runs of at most NT, in whole 16 rows.  An expert's runs of
// one tile follow one another, so that its weights are read once from HBM.
struct ItemList {
  int* first;  // [E + 1] in shared memory: runs of the experts before e
  int2* rows;  // [E] first row and end
  int E;

  __device__ __forceinline__ int runs() const { return first[E]; }

  // By all threads of the block; ends in a barrier.
  template <int THREADS, int NT>
  __device__ __forceinline__ void build(const MatmulInt8Args& a, int* totals,
                                        unsigned* err) const {
    constexpr int kPer = (MOE_MAX_EXPERTS + THREADS - 1) / THREADS;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int count[kPer] = {};
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = kPer * tid + i;
      if (e >= E) continue;
      int64_t lo = 0, hi = a.R;
      if (a.offsets != nullptr) {
        lo = __ldg(a.offsets + e);
        hi = __ldg(a.offsets + e + 1);
        if (lo < 0 || hi > a.R) flag_error(err, MOE_DEVERR_POS_RANGE);
        if (lo < 0) lo = 0;
        if (hi > a.R) hi = a.R;
      }
      rows[e] = make_int2((int)lo, (int)hi);
      count[i] = hi > lo ? (int)((hi - lo + NT - 1) / NT) : 0;
      sum += count[i];
    }
    const int own = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) totals[warp] = sum;
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    int before = sum - own;
    for (int w = 0; w < warp; ++w) before += totals[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (kPer * tid + i <= E) first[kPer * tid + i] = before;
      before += count[i];
    }
    __syncthreads();
  }

  __host__ __device__ __forceinline__ Item at(int64_t it, int tiles) const {
    // 32-bit divisions where they do (a 64-bit one takes longer than the search)
    const bool narrow = it < (int64_t)1 << 32;
    const int q = narrow ? (int)((uint32_t)it / (uint32_t)tiles) : (int)(it / tiles);
    int e = 0;  // the last expert with first[e] <= q
    for (int hi = E; hi - e > 1;) {
      const int mid = (e + hi) >> 1;
      if (first[mid] <= q)
        e = mid;
      else
        hi = mid;
    }
    const int n = first[e + 1] - first[e];
    const int64_t local = it - (int64_t)first[e] * tiles;
    Item m;
    m.e = e;
    m.tile = narrow ? (int)((uint32_t)local / (uint32_t)n) : (int)(local / n);
    const int2 span = rows[e];
    const int run = (int)(local - (int64_t)m.tile * n);
    const int per = ((span.y - span.x - 1) / n + 16) / 16 * 16;  // rows up to 2^31 - 1
    m.r0 = span.x + (int64_t)run * per;
    const int64_t left = span.y - m.r0;
    m.n = (int)(left < 0 ? 0 : left < per ? left : per);
    return m;
  }
};

// The weights as a tensor of rows of K bytes, in boxes of `box_rows` rows of 128 bytes.
inline cudaError_t weight_map(const MatmulInt8Args& a, int box_rows, CUtensorMap* map) {
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
  const cuuint64_t dims[2] = {(cuuint64_t)a.K, (cuuint64_t)a.E * a.N * (a.swiglu ? 2 : 1)};
  const cuuint64_t strides[1] = {(cuuint64_t)a.K};
  const cuuint32_t box[2] = {kBlockK, (cuuint32_t)box_rows}, unit[2] = {1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(a.w), dims,
                            strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace
}  // namespace moe
