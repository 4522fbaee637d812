// expert_matmul_int8_pair.cu -- the experts' 8-bit products (expert_matmul_int8.cu) for
// long runs of rows: a pair of CTAs shares one tile.
//
// With one CTA per tile a product of 128 x 128 x 16 takes 64 clocks of the tensor cores
// and as long to read its weights from tensor memory, each converted row of x feeds 256
// outputs, and two threads issue 8 products per wait each: 1.35 PFLOP/s.  Here the weights
// of 256 outputs lie in the two CTAs' tensor memory, 128 each, and up to 256 rows of x in
// their shared memory, half in each: a product is 256 x 256 x 16 in 128 clocks, every
// converted value feeds 256 others, and one thread of the pair issues 8 products per wait.
//
// Measured: 4096 rows, K = N = 7168: 218 us, 1.93 PFLOP/s, as fast as the measured rate of
// a library's f16 product (1.89); 8192 tokens, top 8 of 256, K = 7168, SwiGLU of 2 x 2048:
// 2820 us, 1.36 PFLOP/s, and 2985 us once the power limit is reached (1950 MHz of 2070).  An
// expert's 257 to 400 rows are two runs, each of whose stages takes as long as its weights'
// conversion, 950 clocks, and not the products' 520 to 800.  The down products, K = 2048,
// N = 7168: 1600 us, 1.2 PFLOP/s (also the tile's end: its sums are read before the next
// tile's products may begin).
//
// Warps 0-7 convert the weights (a thread per weight row), 8-15 write finished tiles out,
// 16-23 gather and convert rows; the converting and the gathering warps are two sets of 4
// that take the stages in turn.  24 asks for the weights (TMA), 25 issues the products
// (first CTA).  With SwiGLU a CTA holds 64 gate and the 64 up rows of
// the same channels, in runs of 8 lanes by turns, so that lane l's partner is l ^ 8.
#include "block/matmul_int8.cuh"

namespace moe {
namespace {

constexpr int kConvert = 8, kFinish = 8, kGather = 8;  // warps
constexpr int kWarps = kConvert + kFinish + kGather + 2;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 4;     // of weights (bytes), rows (f16) and weights (f16)
constexpr int kRowsMax = 256;  // rows of a tile
constexpr int kOuts = 128;     // outputs of a CTA
constexpr int kABytes = kOuts * kBlockK;
constexpr int kBHalf = kRowsMax / 2 * 128;  // 64 channels of a CTA's rows
constexpr int kBBytes = 2 * kBHalf;
constexpr int kColA = kRowsMax;  // first column of the weights
static_assert(kColA + kStages * kBlockK / 2 <= 512, "tensor memory has 512 columns");

struct Smem {
  uint32_t a, b, bars, xsf, totals, tmem, first, rows, total;
};
__host__ __device__ inline Smem smem_layout(int E) {
  Smem s;
  s.a = 0;
  s.b = s.a + kStages * kABytes;
  s.bars = s.b + kStages * kBBytes;
  s.xsf = s.bars + (4 * kStages + 4) * 8;  // 16-byte aligned
  s.totals = s.xsf + kRowsMax * 4;
  s.tmem = s.totals + kWarps * 4;
  s.first = s.tmem + 16 - (s.tmem & 7);
  s.rows = s.first + (uint32_t)(E + 2) / 2 * 8;
  s.total = s.rows + (uint32_t)E * 8;
  return s;
}

template <bool SWIGLU, bool F32>
__global__ void __launch_bounds__(kThreads, 1)
    expert_matmul_pair_kernel(const MatmulInt8Args a, const __grid_constant__ CUtensorMap map,
                              unsigned* err) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const Smem L = smem_layout(a.E);
  const uint32_t sbase = (uint32_t)__cvta_generic_to_shared(smem);
  float* s_xsf = reinterpret_cast<float*>(smem + L.xsf);
  const ItemList list = {reinterpret_cast<int*>(smem + L.first),
                         reinterpret_cast<int2*>(smem + L.rows), a.E};
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  const int rank = (int)cluster_rank();
  // barriers, by stage: weights in / out of shared memory; both operands in place (of both
  // CTAs, in the first); products done (in both).  Then: sums full (both) / free (first)
  const uint32_t a_full = sbase + L.bars, a_free = a_full + kStages * 8;
  const uint32_t full = a_free + kStages * 8, done = full + kStages * 8;
  const uint32_t c_full = done + kStages * 8, c_free = c_full + 8, drain = c_free + 8;

  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map) : "memory");
    for (int i = 0; i < kStages; ++i) {
      mbar_init_n(a_full + i * 8, 1);
      mbar_init_n(a_free + i * 8, 4);
      mbar_init_n(full + i * 8, 2 * (4 + 4));  // a set of converting and one of gathering warps
      mbar_init_n(done + i * 8, 1);
    }
    mbar_init_n(c_full, 1);
    mbar_init_n(c_free, 2 * kFinish);
    mbar_init_n(drain, 1);
    mbar_init_done();
  }
  __syncwarp();
  if (warp == kWarps - 1) tmem2_alloc(sbase + L.tmem);
  __syncwarp();
  cluster_sync();  // the barriers, before the peer arrives at one
  pdl_enter();
  list.build<kThreads, kRowsMax>(a, reinterpret_cast<int*>(smem + L.totals), err);
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L.tmem);
  const int M = SWIGLU ? 2 * a.N : a.N;
  const int per_tile = SWIGLU ? kOuts : 2 * kOuts;  // of the pair
  const int tiles = (a.N + per_tile - 1) / per_tile;
  const int nblk = (a.K + kBlockK - 1) / kBlockK;
  const int64_t items = (int64_t)list.runs() * tiles;
  const int64_t item0 = blockIdx.x / 2, item_step = gridDim.x / 2;
  // rows of a tile in each CTA: the products take multiples of 32 in all
  auto half_rows = [](int n) { return (n + 31) / 32 * 16; };

  bool ok = true;  // no wait ran out
  auto failed = [&]() {
    ok = false;
    flag_error(err, MOE_DEVERR_TIMEOUT);
  };
  auto wait = [&](uint32_t bar, uint32_t phase) {
    if (ok && !mbar_wait(bar, phase, a.wait_ns)) failed();
    return ok;
  };
  auto wait_warp = [&](uint32_t bar, uint32_t phase) {
    return ok = __all_sync(0xFFFFFFFFu, wait(bar, phase));
  };

  if (warp < kConvert) {
    const int l = (warp & 3) * 32 + lane, set = warp >> 2;
    const uint32_t lanes = tmem + (uint32_t)((warp & 3) * 32) * kTmemLane;
    const int src = SWIGLU ? (l & 8) * 8 + (l >> 4) * 8 + (l & 7) : l;  // weight row in a stage
    const uint32_t a_at = sbase + L.a + (uint32_t)(src * 128 + ((src & 7) << 4));
    Ring ra;
    ra.next<kStages>(set);
    // every other stage, of all items
    const int64_t stages = item0 < items ? ((items - 1 - item0) / item_step + 1) * nblk : 0;
    for (int64_t s = set; s < stages; s += 2) {
      if (!wait_warp(a_full + ra.i * 8, ra.phase)) break;
      const uint32_t at = a_at + (uint32_t)(ra.i * kABytes);
      const uint32_t to = lanes + (uint32_t)(kColA + ra.i * (kBlockK / 2));
      uint32_t f[32];
      // 64 channels; of the second 64 the two 8s of each 16 exchanged, as the rows' are
      auto convert = [&](auto second) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          constexpr int first = second ? 4 : 0;
          const uint4 v = lds_v4(at ^ (uint32_t)((first + c) << 4));
          uint32_t *p = f + c * 8 + first, *q = f + c * 8 + 4 - first;
          int8x4_to_f16(v.x, p[0], p[1]);
          int8x4_to_f16(v.y, p[2], p[3]);
          int8x4_to_f16(v.z, q[0], q[1]);
          int8x4_to_f16(v.w, q[2], q[3]);
        }
      };
      convert(std::integral_constant<bool, false>());
      if (!wait_warp(done + ra.i * 8, ra.phase ^ 1u)) break;
      tc_after_sync();
      tmem_store32(to, f);
      convert(std::integral_constant<bool, true>());
      tmem_store32(to + 32, f);
      tmem_store_wait();
      tc_before_sync();
      __syncwarp();
      // the weights' place is free only now: an arrival beside the loads was moved before
      // them, and the next weights overtook the second half
      if (lane == 0) {
        pair_arrive(cluster_map(full + ra.i * 8, 0));
        mbar_arrive(a_free + ra.i * 8);
      }
      ra.next<kStages>(2);
    }
  } else if (warp < kConvert + kFinish) {
    // ---- the tiles' outputs: a warp's lanes, every other 16 of the columns
    const int l = (warp & 3) * 32 + lane, turn = (warp >> 2) & 1, t = tid - kConvert * 32;
    const uint32_t lanes = tmem + (uint32_t)((warp & 3) * 32) * kTmemLane;
    const bool up = SWIGLU && (l & 8);
    uint32_t c_phase = 0;
    for (int64_t it = item0; it < items && ok; it += item_step) {
      const Item m = list.at(it, tiles);
      float my_xsf = 0.0f;
      if (t < m.n) {
        const int64_t s = source_row(a, m.r0 + t, err);
        if (s >= 0) my_xsf = __ldg(a.x_sf + s);
      }
      const int n0 = m.tile * per_tile + rank * (per_tile / 2) +
                     (SWIGLU ? (l >> 4) * 8 + (l & 7) : l);
      const float* wsf = a.w_sf + (int64_t)m.e * M;
      const float w0 = n0 < a.N ? __ldg(wsf + n0) : 0.0f;
      const float w1 = SWIGLU && n0 < a.N ? __ldg(wsf + a.N + n0) : 0.0f;
      s_xsf[t] = my_xsf;
      ok = named_and(1, kFinish * 32, ok);
      if (ok && wait_warp(c_full, c_phase)) {
        tc_after_sync();
        for (int c = turn * 16; c < m.n; c += 32) {
          float x[16];
          __syncwarp();
          tmem_load16(lanes + c, x);
          if (c + 32 >= m.n) {  // the last of them: the next tile's products may begin
            tc_before_sync();
            __syncwarp();
            if (lane == 0) pair_arrive(cluster_map(c_free, 0));
          }
          const int rows = m.n - c < 16 ? m.n - c : 16;
          float xs[16];
          load_scales16(s_xsf + c, xs);
          if constexpr (SWIGLU) {
            // of two columns the gate's lane finishes the first, the up lane the second
            float v[16];
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const float got = __shfl_xor_sync(0xFFFFFFFFu, up ? x[j] : x[j + 1], 8);
              const float s = up ? xs[j + 1] : xs[j];
              const float g = (up ? got : x[j]) * s * w0, u = (up ? x[j + 1] : got) * s * w1;
              v[j / 2] = g * sigmoid_f32(g) * u;
            }
            if (n0 < a.N) {
              const int64_t at = (m.r0 + c + (up ? 1 : 0)) * a.N + n0;
              const int mine = up ? rows - 1 : rows;  // columns j = 0, 2, .. below it
#pragma unroll
              for (int j = 0; j < 8; j += 2) {
                if constexpr (F32) {
                  float* o = static_cast<float*>(a.out) + at + 2 * j * (int64_t)a.N;
                  if (2 * j < mine) *o = v[j];
                  if (2 * j + 2 < mine) o[2 * (int64_t)a.N] = v[j + 1];
                } else {
                  uint16_t* o = static_cast<uint16_t*>(a.out) + at + 2 * j * (int64_t)a.N;
                  const uint32_t w = pack_bf16x2_rn(v[j], v[j + 1]);
                  if (2 * j < mine) *o = (uint16_t)w;
                  if (2 * j + 2 < mine) o[2 * (int64_t)a.N] = (uint16_t)(w >> 16);
                }
              }
            }
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = x[j] * xs[j] * w0;
            if (n0 < a.N) store_column<F32, 16>(a, x, m.r0 + c, rows, n0);
          }
        }
        if (turn * 16 >= m.n) {  // no column here
          __syncwarp();
          if (lane == 0) pair_arrive(cluster_map(c_free, 0));
        }
      }
      c_phase ^= 1u;
      // the scales may be written over; the finishing warps leave together
      ok = named_and(1, kFinish * 32, ok);
    }
  } else if (warp < kConvert + kFinish + kGather) {
    // as in the one-CTA form: 4 rows x 8 units of 16 channels per warp, every 16th row
    constexpr int kStep = kGather / 2 * 4, kUnits = kRowsMax / 2 / kStep;
    const int set = (warp >> 2) & 1, c = lane & 7, r0 = (warp & 3) * 4 + (lane >> 3);
    const uint32_t to0 = sbase + L.b + (uint32_t)((c >> 2) * kBHalf + r0 * 128 +
                                                  ((((c & 3) * 2 + (c >> 2)) ^ (r0 & 7)) << 4));
    const uint32_t to1 = to0 ^ 16u;
    Ring rb;
    rb.next<kStages>(set);
    int turn = set;
    for (int64_t it = item0; it < items && ok; it += item_step) {
      const Item m = list.at(it, tiles);
      const int half = half_rows(m.n);
      const int8_t* from[kUnits];
      uint32_t rows = 0;  // units that have a row; the others stay zero
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const int r = r0 + kStep * u, rr = rank * half + r;
        const int64_t s = r < half && rr < m.n ? source_row(a, m.r0 + rr, err) : -1;
        if (s >= 0) rows |= 1u << u;
        from[u] = a.x + (s >= 0 ? s : 0) * a.K + c * 16 + turn * kBlockK;
      }
      uint4 v[kUnits];
#pragma unroll
      for (int u = 0; u < kUnits; ++u) v[u] = make_uint4(0, 0, 0, 0);
      auto fetch = [&](int kb) {  // block kb, where `from` is
        if (kb >= nblk) return;
        if ((kb + 1) * kBlockK <= a.K) {
#pragma unroll
          for (int u = 0; u < kUnits; ++u)
            if ((rows >> u) & 1u) v[u] = ld_v4(from[u]);
        } else {
          const bool in = kb * kBlockK + c * 16 < a.K;
#pragma unroll
          for (int u = 0; u < kUnits; ++u)
            v[u] = in && ((rows >> u) & 1u) ? ld_v4(from[u]) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < kUnits; ++u) from[u] += 2 * kBlockK;
      };
      int kb = turn;
      fetch(kb);
      for (; kb < nblk; kb += 2) {
        if (!wait_warp(done + rb.i * 8, rb.phase ^ 1u)) break;
        const uint32_t blk = (uint32_t)(rb.i * kBBytes);
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
          if (kStep * u + (warp & 3) * 4 >= half) break;  // this warp's rows
          uint32_t f[8];
          int8x4_to_f16(v[u].x, f[0], f[1]);
          int8x4_to_f16(v[u].y, f[2], f[3]);
          int8x4_to_f16(v[u].z, f[4], f[5]);
          int8x4_to_f16(v[u].w, f[6], f[7]);
          sts_v4(to0 + blk + u * (kStep * 128), f[0], f[1], f[2], f[3]);
          sts_v4(to1 + blk + u * (kStep * 128), f[4], f[5], f[6], f[7]);
        }
        fetch(kb + 2);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) pair_arrive(cluster_map(full + rb.i * 8, 0));
        rb.next<kStages>(2);
      }
      turn = kb - nblk;
    }
  } else if (warp == kConvert + kFinish + kGather) {
    if (lane == 0) {
      Ring ra;
      int64_t asked = 0;
      for (int64_t it = item0; it < items && ok && asked < a.stages; it += item_step) {
        const Item m = list.at(it, tiles);
        // rows past the expert's last output are another's, or past the tensor and zero:
        // their products are not stored
        const int r0 = m.e * M + m.tile * per_tile + rank * (per_tile / 2);
        const int r1 = SWIGLU ? r0 + a.N : r0 + kOuts / 2;
        const int end = a.stages - asked < nblk ? (int)(a.stages - asked) : nblk;
        for (int kb = 0; kb < end; ++kb) {
          if (!wait(a_free + ra.i * 8, ra.phase ^ 1u)) break;
          const uint32_t bar = a_full + ra.i * 8, dst = sbase + L.a + (uint32_t)(ra.i * kABytes);
          const bool box_ok = MOE_DBG_OK(dst % 1024 == 0 && dst + kABytes <= sbase + L.b, err);
          mbar_expect(bar, box_ok ? kABytes : 0);
          if (box_ok) {
            tma_box(dst, &map, kb * kBlockK, r0, bar);
            tma_box(dst + kABytes / 2, &map, kb * kBlockK, r1, bar);
          }
          ++asked;
          ra.next<kStages>();
        }
      }
      // what may still be on its way, if another warp gave up: the last stages, each waited
      // for (bounded)
      for (int i = 0; i < kStages && i < asked; ++i) {
        if (ra.i == 0) ra.i = kStages, ra.phase ^= 1u;
        --ra.i;
        (void)mbar_wait(a_full + ra.i * 8, ra.phase);
      }
    }
  } else if (rank == 0) {
    if (lane == 0) {
      Ring rb;
      uint32_t c_phase = 0;
      bool any = false;
      for (int64_t it = item0; it < items && ok; it += item_step) {
        const Item m = list.at(it, tiles);
        const uint32_t idesc = tc_idesc_f16(2 * kOuts, 2 * half_rows(m.n));
        if (!wait(c_free, c_phase ^ 1u)) break;
        for (int kb = 0; kb < nblk; ++kb) {
          if (!wait(full + rb.i * 8, rb.phase)) break;
          tc_after_sync();
          const uint64_t b0 = tc_desc_sw128(sbase + L.b + (uint32_t)(rb.i * kBBytes));
#pragma unroll
          for (int s = 0; s < kBlockK / 16; ++s)
            tc2_mma_f16(tmem, tmem + (uint32_t)(kColA + rb.i * (kBlockK / 2) + s * 8),
                        b0 + (uint64_t)((s >> 2) * kBHalf >> 4) + (uint64_t)((s & 3) * 2), idesc,
                        kb > 0 || s > 0);
          any = true;
          tc2_commit(done + rb.i * 8);
          rb.next<kStages>();
        }
        if (!ok) break;
        tc2_commit(c_full);
        c_phase ^= 1u;
      }
      if (any) {  // the products in flight end before either CTA gives its memory back
        tc2_commit_here(drain);
        (void)mbar_wait(drain, 0);
      }
    }
  }
  __syncwarp();
  tc_before_sync();
  __syncthreads();
  cluster_sync();  // no peer arrives here, and no product reads this CTA, any more
  if (warp == kWarps - 1) {
    tc_after_sync();
    tmem2_free(tmem);
  }
}

template <bool SWIGLU, bool F32>
cudaError_t launch_t(const LaunchCtx& c, const MatmulInt8Args& a) {
  auto* kernel = expert_matmul_pair_kernel<SWIGLU, F32>;
  static SmemOptIn opt_in;
  cudaError_t e = opt_in.once(kernel);
  if (e != cudaSuccess) return e;
  CUtensorMap map;
  e = weight_map(a, kOuts / 2, &map);
  if (e != cudaSuccess) return e;
  const int per_tile = SWIGLU ? kOuts : 2 * kOuts;
  int64_t runs = (a.offsets ? a.E : 1) + (a.R + kRowsMax - 1) / kRowsMax - 1;
  if (runs > a.R) runs = a.R;
  const int64_t items = runs * ((a.N + per_tile - 1) / per_tile), pairs = c.num_sms / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * (items < pairs ? items : pairs)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_layout(a.E).total;
  cfg.stream = c.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, kernel, a, map, c.err);
}

}  // namespace

cudaError_t launch_expert_matmul_int8_pair(const LaunchCtx& c, const MatmulInt8Args& a) {
  if (a.swiglu) return a.out_f32 ? launch_t<true, true>(c, a) : launch_t<true, false>(c, a);
  return a.out_f32 ? launch_t<false, true>(c, a) : launch_t<false, false>(c, a);
}

}  // namespace moe
