// cast_int8.cu -- rows to 8-bit integers with one scale per row.
//
//   a = max(max_c |x[t,c]|, 2^-96);  sf = a / 127;  q = rint(x * (127 / a))
//
// Each step is one f32 rounding, so the integers are fixed by the definition.  HBM
// bounds it: a row is read once, kept in registers across the maximum, and written.
#include "block/block_ops.cuh"

namespace moe {
namespace {

constexpr float kFloor = 0x1p-96f;

// rint(x * inv), |x * inv| < 2^22, in the low byte as two's complement: adding
// 1.5 * 2^23 leaves the integer (nearest, ties to even) in the low mantissa bits.
// Two roundings on purpose (the product's, then the integer's): no fused multiply-add.
__device__ __forceinline__ uint32_t round_bits(float x, float inv) {
  return __float_as_uint(__fadd_rn(__fmul_rn(x, inv), 12582912.0f));
}
__device__ __forceinline__ uint32_t pack4(const float* v, float inv) {
  const uint32_t lo = __byte_perm(round_bits(v[0], inv), round_bits(v[1], inv), 0x0040);
  const uint32_t hi = __byte_perm(round_bits(v[2], inv), round_bits(v[3], inv), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

// The block's maximum of m >= 0, for every thread.
template <int THREADS>
__device__ __forceinline__ float block_max(float m, float* part) {
  uint32_t b = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m));
  if constexpr (THREADS > 32) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) part[warp] = __uint_as_float(b);
    __syncthreads();
    b = __reduce_max_sync(0xFFFFFFFFu,
                          lane < THREADS / 32 ? __float_as_uint(part[lane]) : 0u);
  }
  return __uint_as_float(b);
}

// One block per row; a thread holds UNITS units of VEC elements, unit i at
// (i * THREADS + thread) * VEC.  MORE: rows beyond THREADS * UNITS * VEC elements,
// whose rest is read a second time after the maximum.
template <class T, int VEC, int UNITS, int THREADS, bool MORE>
__global__ void __launch_bounds__(THREADS)
    cast_int8_kernel(const T* __restrict__ x, int64_t rows, int H, int8_t* __restrict__ out,
                     float* __restrict__ sf) {
  __shared__ float part[THREADS / 32];
  pdl_enter();
  const int64_t t = blockIdx.x;
  const T* row = x + t * H;
  int8_t* orow = out + t * H;
  float v[UNITS][VEC];
  float m = kFloor;
#pragma unroll
  for (int i = 0; i < UNITS; ++i) {
    const int c = (i * THREADS + (int)threadIdx.x) * VEC;
    if (c < H) {
      load_elems<VEC>(row + c, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < UNITS; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) m = fmaxf(m, fabsf(v[i][j]));
  constexpr int kHeld = UNITS * THREADS * VEC;
  if constexpr (MORE) {
    for (int c = kHeld + (int)threadIdx.x * VEC; c < H; c += THREADS * VEC) {
      float u[VEC];
      load_elems<VEC>(row + c, u);
#pragma unroll
      for (int j = 0; j < VEC; ++j) m = fmaxf(m, fabsf(u[j]));
    }
  }
  m = block_max<THREADS>(m, part);
  const float inv = __fdiv_rn(127.0f, m);
  if (threadIdx.x == 0) sf[t] = __fdiv_rn(m, 127.0f);
  auto store = [&](int c, const float (&u)[VEC]) {
    if constexpr (VEC == 8)
      st_stream_v2(orow + c, make_uint2(pack4(u, inv), pack4(u + 4, inv)));
    else
      orow[c] = (int8_t)(round_bits(u[0], inv) & 0xFFu);
  };
#pragma unroll
  for (int i = 0; i < UNITS; ++i) {
    const int c = (i * THREADS + (int)threadIdx.x) * VEC;
    if (c < H) store(c, v[i]);
  }
  if constexpr (MORE) {
    for (int c = kHeld + (int)threadIdx.x * VEC; c < H; c += THREADS * VEC) {
      float u[VEC];
      load_elems<VEC>(row + c, u);
      store(c, u);
    }
  }
}

template <class T, int VEC, int UNITS, int THREADS, bool MORE>
cudaError_t launch_t(const LaunchCtx& c, const void* x, int64_t T_, int H, int8_t* out,
                     float* sf) {
  return launch_pdl(cast_int8_kernel<T, VEC, UNITS, THREADS, MORE>, dim3((unsigned)T_), THREADS, 0,
                    c.stream, static_cast<const T*>(x), T_, H, out, sf);
}

template <class T>
cudaError_t launch(const LaunchCtx& c, const void* x, int64_t rows, int H, int8_t* out,
                   float* sf) {
  const bool vec = H % 8 == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(out) % 8 == 0;
  if (vec) {
    if (H <= 32 * 8) return launch_t<T, 8, 1, 32, false>(c, x, rows, H, out, sf);
    if (H <= 128 * 8) return launch_t<T, 8, 1, 128, false>(c, x, rows, H, out, sf);
    if (H <= 128 * 32) return launch_t<T, 8, 4, 128, false>(c, x, rows, H, out, sf);
    if (H <= 256 * 32) return launch_t<T, 8, 4, 256, false>(c, x, rows, H, out, sf);
    return launch_t<T, 8, 4, 512, true>(c, x, rows, H, out, sf);
  }
  if (H <= 32 * 4) return launch_t<T, 1, 4, 32, false>(c, x, rows, H, out, sf);
  if (H <= 128 * 16) return launch_t<T, 1, 16, 128, false>(c, x, rows, H, out, sf);
  return launch_t<T, 1, 32, 256, true>(c, x, rows, H, out, sf);
}

}  // namespace

cudaError_t launch_cast_int8(const LaunchCtx& c, const void* x, bool f32, int64_t T, int H,
                             int8_t* out, float* sf) {
  return f32 ? launch<float>(c, x, T, H, out, sf) : launch<Bf16>(c, x, T, H, out, sf);
}

}  // namespace moe
