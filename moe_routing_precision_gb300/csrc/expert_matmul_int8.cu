// expert_matmul_int8.cu -- products of routed 8-bit rows with their expert's 8-bit
// weights.
//
//   o[r, m] = (sum_c x[src(r), c] * w[e(r), m, c]) * x_sf[src(r)] * w_sf[e(r), m]
//
// sm_103a's tensor cores take no 8-bit integers (tcgen05.mma kind::i8 exists on other
// parts only), and mma.sync's are far slower.  8-bit integers are exact in f16, and their
// products and any sum below 2^24 in f32, so the products go to tcgen05.mma kind::f16:
// the weights are the M operand, converted from shared into tensor memory on their way,
// the rows of x the N operand, converted from global into shared memory.  Both are read
// as bytes, which is what counts for few rows, where HBM bounds it.
//
// A tile is 2 x 128 outputs (two accumulators in the same lanes; with SwiGLU the gate's
// and the up outputs of 128 channels, which one thread then holds) by up to NT rows.
// One CTA per SM, its warps in roles joined by barriers:
//   0-7    convert a stage of weights (a thread per weight row) into tensor memory, and
//          write the finished tiles out; 4 warps per half
//   8-15   gather, convert and store the rows of x
//   16     asks for the weights (TMA, 128-byte swizzle)
//   17-18  issue the products of one half each: a product takes at least the 61 clocks
//          that its weights take out of tensor memory, and what one issuer waits for does
//          not keep the tensor cores from the other's (one issuer: 620 : 496 us, 64 tokens,
//          top 8 of 256, K = 2048, N = 7168)
// Measured: 64 tokens, top 8 of 256, K = 7168, SwiGLU of 2 x 2048 (6.5 GB): 939 us, 6.9
// TB/s, and K = 2048, N = 7168 (3.3 GB) 510 us: HBM bounds them.  One token: 49 us for 235
// MB, which a kernel that only reads them takes 45 us for (5.3 TB/s; the rate for so few bytes
// bounds it, then the 5 us until the first weights are there and their conversion); smaller
// tiles, one for each of 152 SMs, or six stages of weights were no faster.  16 converting warps in two sets were
// slower for long runs (308 : 336 us), as were tiles of 32, 64 or 96 rows (no faster for few
// rows).  Long runs: expert_matmul_int8_pair.cu.
#include "block/matmul_int8.cuh"

namespace moe {

std::atomic<int64_t> g_matmul_int8_stages{INT64_MAX};

namespace {

constexpr int kWarps = 19;
constexpr int kThreads = kWarps * 32;
constexpr int kConvert = 8;          // warps 0 .. 7
constexpr int kGather = 8;           // warps 8 .. 15
constexpr int kHalf = 128;           // outputs of one accumulator
constexpr int kABytes = 2 * kHalf * kBlockK;

// NT rows per tile; SA stages of weights (bytes) and SB of rows (f16) in shared memory,
// ST of weights (f16) in tensor memory, behind the two accumulators.  SPLIT: the CTAs of
// a cluster take equal parts of K of one tile and add their sums up.
template <int NT_, int SA_, int SB_, int ST_, bool SPLIT_>
struct Shape {
  static constexpr int NT = NT_, SA = SA_, SB = SB_, ST = ST_;
  static constexpr bool SPLIT = SPLIT_;
  static constexpr int kPartBytes = SPLIT ? 2 * NT * kHalf * 4 : 0;
  static constexpr int kBBytes = NT * kBlockK * 2;
  static constexpr int kColA = 2 * NT;  // first column of the weights
  static_assert(kColA + ST * 128 <= 512, "tensor memory has 512 columns");
};

struct Smem {
  uint32_t a, b, part, bars, xsf, totals, tmem, first, rows, total;
};
template <class S>
__host__ __device__ inline Smem smem_layout(int E) {
  Smem s;
  s.a = 0;
  s.b = s.a + S::SA * kABytes;
  s.part = s.b + S::SB * S::kBBytes;
  s.bars = s.part + S::kPartBytes;
  s.xsf = s.bars + (2 * S::SA + 2 * S::SB + 4 * S::ST + 6) * 8;  // 16-byte aligned
  s.totals = s.xsf + S::NT * 4;
  s.tmem = s.totals + kWarps * 4;
  s.first = s.tmem + 16 - (s.tmem & 7);
  s.rows = s.first + (uint32_t)(E + 2) / 2 * 8;
  s.total = s.rows + (uint32_t)E * 8;
  return s;
}

template <class S, bool F32>
__global__ void __launch_bounds__(kThreads, 1)
    expert_matmul_kernel(const MatmulInt8Args a, const __grid_constant__ CUtensorMap map,
                         unsigned* err) {
  constexpr int NT = S::NT;
  extern __shared__ __align__(1024) uint8_t smem[];
  const Smem L = smem_layout<S>(a.E);
  const uint32_t sbase = (uint32_t)__cvta_generic_to_shared(smem);
  float* s_xsf = reinterpret_cast<float*>(smem + L.xsf);
  int* first = reinterpret_cast<int*>(smem + L.first);
  int2* rows_of = reinterpret_cast<int2*>(smem + L.rows);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);
  // barriers: weights in / out of a shared stage, rows in / out, a half's weights in / out
  // of a tensor-memory stage, accumulators full / free, and two to drain the products
  const uint32_t a_full = sbase + L.bars, a_free = a_full + S::SA * 8;
  const uint32_t b_full = a_free + S::SA * 8, b_free = b_full + S::SB * 8;
  const uint32_t t_full = b_free + S::SB * 8, t_free = t_full + 2 * S::ST * 8;
  const uint32_t c_full = t_free + 2 * S::ST * 8, c_free = c_full + 8, drain = c_free + 8;
  const uint32_t p_full = drain + 16, p_free = p_full + 8;  // SPLIT: sums written, read

  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map) : "memory");
    for (int i = 0; i < S::SA; ++i) mbar_init_n(a_full + i * 8, 1), mbar_init_n(a_free + i * 8, kConvert);
    for (int i = 0; i < S::SB; ++i) mbar_init_n(b_full + i * 8, kGather), mbar_init_n(b_free + i * 8, 2);
    for (int i = 0; i < 2 * S::ST; ++i) mbar_init_n(t_full + i * 8, kConvert / 2), mbar_init_n(t_free + i * 8, 1);
    mbar_init_n(c_full, 2);
    mbar_init_n(c_free, kConvert);
    mbar_init_n(drain, 1);
    mbar_init_n(drain + 8, 1);
    if (S::SPLIT) {
      mbar_init_n(p_full, kConvert * (int)cluster_size());
      mbar_init_n(p_free, kConvert * (int)cluster_size());
    }
    mbar_init_done();
  }
  if (warp == kWarps - 1) tmem_alloc(sbase + L.tmem);
  __syncwarp();
  if (S::SPLIT) cluster_sync();  // the barriers, before a peer arrives at one
  pdl_enter();

  const ItemList list = {first, rows_of, a.E};
  list.build<kThreads, NT>(a, reinterpret_cast<int*>(smem + L.totals), err);
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L.tmem);
  const int M = a.swiglu ? 2 * a.N : a.N;
  const int per_tile = a.swiglu ? kHalf : 2 * kHalf;
  const int tiles = (a.N + per_tile - 1) / per_tile;
  const int nblk = (a.K + kBlockK - 1) / kBlockK;
  const int64_t items = (int64_t)list.runs() * tiles;
  // this CTA's items, and its part of their channels
  const int ctas = S::SPLIT ? (int)cluster_size() : 1, rank = S::SPLIT ? (int)cluster_rank() : 0;
  const int64_t item0 = blockIdx.x / ctas, item_step = gridDim.x / ctas;
  const int kb0 = nblk * rank / ctas, kb1 = nblk * (rank + 1) / ctas;

  auto item_at = [&](int64_t it) { return list.at(it, tiles); };
  bool ok = true;  // no wait ran out
  auto wait = [&](uint32_t bar, uint32_t phase) {
    if (ok && !mbar_wait(bar, phase, a.wait_ns)) {
      ok = false;
      flag_error(err, MOE_DEVERR_TIMEOUT);
    }
    return ok;
  };
  // the same for a whole warp, with one answer
  auto wait_warp = [&](uint32_t bar, uint32_t phase) {
    return ok = __all_sync(0xFFFFFFFFu, wait(bar, phase));
  };

  if (warp < kConvert) {
    const int half = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + (uint32_t)((warp & 3) * 32) * kTmemLane;
    // this thread's row in a stage, at the first 16 bytes' place under the swizzle
    const uint32_t a_at = sbase + L.a + (uint32_t)(half * (kABytes / 2) + row * 128 + ((row & 7) << 4));
    Ring ra, rt;
    uint32_t c_phase = 0;
    for (int64_t it = item0; it < items && ok; it += item_step) {
      const Item m = item_at(it);
      // the scales of the run's rows, asked for early
      float my_xsf = 0.0f;
      if (tid < m.n) {
        const int64_t s = source_row(a, m.r0 + tid, err);
        if (s >= 0) my_xsf = __ldg(a.x_sf + s);
      }
      const int n0 = m.tile * per_tile + row, n1 = n0 + kHalf;  // n1 without SwiGLU
      const float* wsf = a.w_sf + (int64_t)m.e * M;
      const float w0 = n0 < a.N ? __ldg(wsf + n0) : 0.0f;
      const float w1 = a.swiglu ? (n0 < a.N ? __ldg(wsf + a.N + n0) : 0.0f)
                                : (n1 < a.N ? __ldg(wsf + n1) : 0.0f);
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!wait_warp(a_full + ra.i * 8, ra.phase)) break;
        const uint32_t at = a_at + (uint32_t)(ra.i * kABytes);
        uint4 v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = lds_v4(at ^ (uint32_t)(c << 4));
        uint32_t f[32];
        auto convert = [&](int c0) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            // units 4 to 7 with their two groups exchanged, as the rows' are
            uint32_t* o = f + c * 8;
            uint32_t *p = c0 ? o + 4 : o, *q = c0 ? o : o + 4;
            int8x4_to_f16(v[c0 + c].x, p[0], p[1]);
            int8x4_to_f16(v[c0 + c].y, p[2], p[3]);
            int8x4_to_f16(v[c0 + c].z, q[0], q[1]);
            int8x4_to_f16(v[c0 + c].w, q[2], q[3]);
          }
        };
        convert(0);
        if (!wait_warp(t_free + (half * S::ST + rt.i) * 8, rt.phase ^ 1u)) break;
        tc_after_sync();
        const uint32_t to = lanes + (uint32_t)(S::kColA + rt.i * 128 + half * 64);
        tmem_store32(to, f);
        convert(4);
        tmem_store32(to + 32, f);
        tmem_store_wait();
        tc_before_sync();
        __syncwarp();
        // the weights' place is free only now, when the stores have taken what was loaded: an
        // arrival beside the loads may be moved before them
        if (lane == 0) {
          mbar_arrive(t_full + (half * S::ST + rt.i) * 8);
          mbar_arrive(a_free + ra.i * 8);
        }
        ra.next<S::SA>();
        rt.next<S::ST>();
      }
      // ---- the tile's outputs: this warp's lanes, half of its columns
      if (tid < NT) s_xsf[tid] = my_xsf;
      ok = named_and(1, kConvert * 32, ok);
      auto finish = [&](float p, float q, float xs, float u0, float u1, int64_t at, int n) {
        // p and q: the sums of output n and, behind it, of its partner
        p = p * xs * u0, q = q * xs * u1;
        if (a.swiglu) {
          if (n < a.N) store_out(a, at + n, p * sigmoid_f32(p) * q);
        } else {
          if (n < a.N) store_out(a, at + n, p);
          if (n + kHalf < a.N) store_out(a, at + n + kHalf, q);
        }
      };
      if (S::SPLIT && ok) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_cluster(p_free, c_phase ^ 1u, a.wait_ns));
        if (!ok) flag_error(err, MOE_DEVERR_TIMEOUT);
      }
      if (ok && wait_warp(c_full, c_phase)) {
        tc_after_sync();
        float* part = reinterpret_cast<float*>(smem + L.part);
        for (int c = half * (NT / 2); c < (half + 1) * (NT / 2) && c < m.n; c += 16) {
          float x[16], y[16];
          __syncwarp();
          tmem_load16x2(lanes + c, lanes + NT + c, x, y);
          const int rows = m.n - c < 16 ? m.n - c : 16;
          if constexpr (S::SPLIT) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              if (j >= rows) break;
              part[(c + j) * kHalf + row] = x[j];
              part[(NT + c + j) * kHalf + row] = y[j];
            }
          } else {
            // 4 columns at a time: a run may have few rows
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              if (j >= rows) break;
              const float4 xs = *reinterpret_cast<const float4*>(s_xsf + c + j);
              const float s[4] = {xs.x, xs.y, xs.z, xs.w};
              float p[4], q[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                p[i] = x[j + i] * s[i] * w0, q[i] = y[j + i] * s[i] * w1;
                if (a.swiglu) p[i] = p[i] * sigmoid_f32(p[i]) * q[i];
              }
              if (n0 < a.N) store_column<F32, 4>(a, p, m.r0 + c + j, rows - j, n0);
              if (!a.swiglu && n1 < a.N) store_column<F32, 4>(a, q, m.r0 + c + j, rows - j, n1);
            }
          }
        }
        tc_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(c_free);
        if constexpr (S::SPLIT) {
          if (lane < ctas) cluster_arrive(cluster_map(p_full, lane));
          ok = __all_sync(0xFFFFFFFFu, mbar_wait_cluster(p_full, c_phase, a.wait_ns));
          if (!ok) flag_error(err, MOE_DEVERR_TIMEOUT);
          if (ok) {
            // this CTA's share of the tile: pairs of sums, added in the CTAs' order
            const int pairs = m.n * kHalf;
            const int p0 = pairs * rank / ctas, p1 = pairs * (rank + 1) / ctas;
            const int l = (p0 + tid) & (kHalf - 1), n = m.tile * per_tile + l;
            const float u0 = n < a.N ? __ldg(wsf + n) : 0.0f;
            const int partner = a.swiglu ? a.N + n : n + kHalf;
            const float u1 = partner < M ? __ldg(wsf + partner) : 0.0f;
            const uint32_t at = sbase + L.part;
            for (int p = p0 + tid; p < p1; p += kConvert * 32) {
              float x = 0.0f, y = 0.0f;
              for (int r = 0; r < ctas; ++r) {
                const uint32_t from = cluster_map(at + (uint32_t)p * 4, r);
                x += cluster_load(from);
                y += cluster_load(from + NT * kHalf * 4);
              }
              const int c = p / kHalf;
              finish(x, y, s_xsf[c], u0, u1, (m.r0 + c) * a.N, n);
            }
          }
          __syncwarp();
          if (lane < ctas) cluster_arrive(cluster_map(p_free, lane));
        }
      }
      c_phase ^= 1u;
      // the scales may be written over; the converting warps leave together
      ok = named_and(1, kConvert * 32, ok);
    }
  } else if (warp < kConvert + kGather) {
    // A warp takes 4 rows x 8 units of 16 channels of a stage (8 lanes per row: whole lines
    // asked for at once, half lines took twice as long), and every 32nd row after them.
    // A unit becomes two 16-byte groups of f16; units 4 to 7 lie in a second block of rows,
    // with their groups exchanged, so that the 8 lanes of a store meet 8 different groups
    // of banks.  The weights' channels are exchanged in the same way: a sum has no order.
    constexpr int kStep = kGather * 4, kUnits = NT > kStep ? NT / kStep : 1;
    const int c = lane & 7, r0 = (warp - kConvert) * 4 + (lane >> 3);
    const uint32_t to0 = sbase + L.b + (uint32_t)((c >> 2) * (NT * 128) + r0 * 128 +
                                                  ((((c & 3) * 2 + (c >> 2)) ^ (r0 & 7)) << 4));
    const uint32_t to1 = to0 ^ 16u;
    Ring rb;
    for (int64_t it = item0; it < items && ok; it += item_step) {
      const Item m = item_at(it);
      const int8_t* from[kUnits];
      uint32_t rows = 0;  // units that have a row; the others stay zero
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        const int r = r0 + kStep * u;
        const int64_t s = r < m.n ? source_row(a, m.r0 + r, err) : -1;
        if (s >= 0) rows |= 1u << u;
        from[u] = a.x + (s >= 0 ? s : 0) * a.K + c * 16 + (int64_t)kb0 * kBlockK;
      }
      uint4 v0[kUnits], v1[kUnits];
#pragma unroll
      for (int u = 0; u < kUnits; ++u) v0[u] = v1[u] = make_uint4(0, 0, 0, 0);
      // asks for block kb; `from` is at block kb - ahead
      auto fetch = [&](uint4 (&v)[kUnits], int kb, int ahead) {
        if (kb >= kb1) return;
        if ((kb + 1) * kBlockK <= a.K) {
#pragma unroll
          for (int u = 0; u < kUnits; ++u)
            if ((rows >> u) & 1u) v[u] = ld_v4(from[u] + ahead * kBlockK);
        } else {
          const bool in = kb * kBlockK + c * 16 < a.K;
#pragma unroll
          for (int u = 0; u < kUnits; ++u)
            v[u] = in && ((rows >> u) & 1u) ? ld_v4(from[u] + ahead * kBlockK)
                                            : make_uint4(0, 0, 0, 0);
        }
      };
      // one stage from registers that were asked for two stages before
      auto stage = [&](uint4 (&v)[kUnits], int kb) {
        if (!wait_warp(b_free + rb.i * 8, rb.phase ^ 1u)) return;
        const uint32_t blk = (uint32_t)(rb.i * S::kBBytes);
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
          if (kStep * u + (warp - kConvert) * 4 >= m.n) break;  // this warp's rows
          uint32_t f[8];
          int8x4_to_f16(v[u].x, f[0], f[1]);
          int8x4_to_f16(v[u].y, f[2], f[3]);
          int8x4_to_f16(v[u].z, f[4], f[5]);
          int8x4_to_f16(v[u].w, f[6], f[7]);
          sts_v4(to0 + blk + u * (kStep * 128), f[0], f[1], f[2], f[3]);
          sts_v4(to1 + blk + u * (kStep * 128), f[4], f[5], f[6], f[7]);
          from[u] += kBlockK;
        }
        fetch(v, kb + 2, 1);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_full + rb.i * 8);
        rb.next<S::SB>();
      };
      fetch(v0, kb0, 0);
      fetch(v1, kb0 + 1, 1);
      for (int kb = kb0; kb < kb1 && ok; kb += 2) {
        stage(v0, kb);
        if (kb + 1 < kb1 && ok) stage(v1, kb + 1);
      }
    }
  } else if (warp == kConvert + kGather) {
    if (lane == 0) {
      Ring ra;
      int64_t asked = 0;
      for (int64_t it = item0; it < items && ok && asked < a.stages; it += item_step) {
        const Item m = item_at(it);
        // rows past the expert's last output are another's, or past the tensor and zero:
        // their products are not stored
        const int r0 = m.e * M + m.tile * per_tile;
        const int r1 = a.swiglu ? r0 + a.N : r0 + kHalf;
        const int end = a.stages - asked < kb1 - kb0 ? kb0 + (int)(a.stages - asked) : kb1;
        for (int kb = kb0; kb < end; ++kb) {
          if (!wait(a_free + ra.i * 8, ra.phase ^ 1u)) break;
          const uint32_t bar = a_full + ra.i * 8, dst = sbase + L.a + (uint32_t)(ra.i * kABytes);
          const bool box_ok = MOE_DBG_OK(dst % 1024 == 0 && dst + kABytes <= sbase + L.b, err);
          mbar_expect(bar, box_ok ? kABytes : 0);
          if (box_ok) {
            tma_box(dst, &map, kb * kBlockK, r0, bar);
            tma_box(dst + kABytes / 2, &map, kb * kBlockK, r1, bar);
          }
          ++asked;
          ra.next<S::SA>();
        }
      }
      // what may still be on its way, if another warp gave up: the last SA stages, each waited
      // for (bounded)
      for (int i = 0; i < S::SA && i < asked; ++i) {
        if (ra.i == 0) ra.i = S::SA, ra.phase ^= 1u;
        --ra.i;
        (void)mbar_wait(a_full + ra.i * 8, ra.phase);
      }
    }
  } else {
    if (lane == 0) {
      const int h = warp - (kWarps - 2);
      const uint32_t th_full = t_full + h * S::ST * 8, th_free = t_free + h * S::ST * 8;
      Ring rb, rt;
      uint32_t c_phase = 0;
      bool any = false;
      for (int64_t it = item0; it < items && ok; it += item_step) {
        const Item m = item_at(it);
        const uint32_t idesc = tc_idesc_f16(kHalf, (m.n + 15) / 16 * 16);
        if (!wait(c_free, c_phase ^ 1u)) break;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait(b_full + rb.i * 8, rb.phase)) break;
          if (!wait(th_full + rt.i * 8, rt.phase)) break;
          tc_after_sync();
          const uint64_t b0 = tc_desc_sw128(sbase + L.b + (uint32_t)(rb.i * S::kBBytes));
#pragma unroll
          for (int s = 0; s < kBlockK / 16; ++s)
            tc_mma_f16(tmem + (uint32_t)(h * NT),
                       tmem + (uint32_t)(S::kColA + rt.i * 128 + h * 64 + s * 8),
                       b0 + (uint64_t)((s >> 2) * (NT * 128) >> 4) + (uint64_t)((s & 3) * 2),
                       idesc, kb > kb0 || s > 0);
          any = true;
          tc_commit(b_free + rb.i * 8);
          tc_commit(th_free + rt.i * 8);
          rb.next<S::SB>();
          rt.next<S::ST>();
        }
        if (!ok) break;
        tc_commit(c_full);
        c_phase ^= 1u;
      }
      if (any) {  // the products in flight end before tensor memory is given back
        tc_commit(drain + h * 8);
        (void)mbar_wait(drain + h * 8, 0);
      }
    }
  }
  __syncwarp();
  tc_before_sync();
  __syncthreads();
  if (S::SPLIT) cluster_sync();  // no peer reads or arrives here any more
  if (warp == kWarps - 1) {
    tc_after_sync();
    tmem_free(tmem);
  }
}

// A launch of `blocks` CTAs in clusters of `ctas`.
template <class S>
struct Config {
  cudaLaunchConfig_t c = {};
  cudaLaunchAttribute attr[2];
  Config(int E, int64_t blocks, int ctas) {
    c.gridDim = dim3((unsigned)blocks);
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = smem_layout<S>(E).total;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    c.attrs = attr;
    c.numAttrs = S::SPLIT ? 2 : 1;
  }
};

// How many clusters of 2, 4 or 8 CTAs the device runs at once: one CTA per SM, and fewer
// SMs than a die's that a cluster can share.  Asked once per process and size.
template <class S>
cudaError_t clusters_at_once(const LaunchCtx& c, int ctas, int* n) {
  static std::atomic<int> known[4];
  std::atomic<int>& slot = known[ctas == 2 ? 1 : ctas == 4 ? 2 : 3];
  *n = slot.load(std::memory_order_relaxed);
  if (*n > 0) return cudaSuccess;
  auto* kernel = expert_matmul_kernel<S, false>;
  cudaError_t e = allow_max_dynamic_smem(kernel);
  if (e != cudaSuccess) return e;
  Config<S> cfg(MOE_MAX_EXPERTS, (int64_t)c.num_sms / ctas * ctas, ctas);
  // the query takes no launch attribute but the cluster's
  cfg.attr[0] = cfg.attr[1];
  cfg.c.numAttrs = 1;
  e = cudaOccupancyMaxActiveClusters(n, kernel, &cfg.c);
  if (e == cudaSuccess) slot.store(*n, std::memory_order_relaxed);
  return e;
}

// `ctas` CTAs per item (a cluster, if more than one).
template <class S, bool F32>
cudaError_t launch_f(const LaunchCtx& c, const MatmulInt8Args& a, int64_t groups, int ctas) {
  auto* kernel = expert_matmul_kernel<S, F32>;
  static SmemOptIn opt_in;
  cudaError_t e = opt_in.once(kernel);
  if (e != cudaSuccess) return e;
  CUtensorMap map;
  e = weight_map(a, kHalf, &map);
  if (e != cudaSuccess) return e;
  Config<S> cfg(a.E, groups * ctas, ctas);
  cfg.c.stream = c.stream;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg.c, kernel, a, map, c.err);
}
template <class S>
cudaError_t launch_t(const LaunchCtx& c, const MatmulInt8Args& a, int64_t groups, int ctas) {
  return a.out_f32 ? launch_f<S, true>(c, a, groups, ctas) : launch_f<S, false>(c, a, groups, ctas);
}

using Whole = Shape<128, 4, 2, 2, false>;
using Split = Shape<32, 4, 4, 3, true>;

// Tiles times runs of at most nt rows, at most.
int64_t items_at_most(const MatmulInt8Args& a, int nt) {
  const int per_tile = a.swiglu ? kHalf : 2 * kHalf;
  int64_t runs = (a.offsets ? a.E : 1) + (a.R + nt - 1) / nt - 1;
  if (runs > a.R) runs = a.R;
  return runs * ((a.N + per_tile - 1) / per_tile);
}

}  // namespace

cudaError_t expert_matmul_int8_form(const LaunchCtx& c, const MatmulInt8Args& a, int* form,
                                    int* ctas) {
  // Few tiles: a cluster shares each one's channels, as long as all clusters run at once
  // (E = 1, one row, us, 1 : 2 : 4 : 8 CTAs per tile: K = N = 4096 28 : 18 : 12.4 : two
  // rounds 18; K = 7168, N = 256 46 : 27 : 16.6 : 11.7.  With tiles for 128 CTAs, 1 token
  // of 8 experts: 49 : two rounds 56 : 94 : 130).
  const int nblk = (a.K + kBlockK - 1) / kBlockK;
  const int64_t split = items_at_most(a, Split::NT);
  *ctas = 1;
  for (int s = 2; s <= 8 && s <= nblk; s *= 2) {
    if (split * s > c.num_sms) break;
    int fit = 0;
    const cudaError_t e = clusters_at_once<Split>(c, s, &fit);
    if (e != cudaSuccess) return e;
    if (split <= fit) *ctas = s;
  }
  // Long runs of rows: a pair of CTAs per tile (us, one CTA : a pair; 256 experts, K = 7168,
  // SwiGLU of 2 x 2048: 64 rows per expert on average 1532 : 1720, 80 1621 : 1772, 128 2086 :
  // 1963, 256 3507 : 2850; one expert, K = N = 4096: 128 rows 22 : 22, 256 35 : 27; 16 experts
  // of 1024 rows, K = N = 256: 17 : 19, its start counts).  The host knows the rows of out
  // alone: rows that no expert has (a padded layout, a worst-case buffer) count as its rows.
  *form = *ctas > 1                                ? MOE_MATMUL_INT8_CLUSTER
          : a.R > 104 * (int64_t)a.E && a.K > 512 ? MOE_MATMUL_INT8_PAIR
                                                   : MOE_MATMUL_INT8_CTA;
  return cudaSuccess;
}

cudaError_t launch_expert_matmul_int8(const LaunchCtx& c, const MatmulInt8Args& a) {
  int form = 0, ctas = 1;
  const cudaError_t e = expert_matmul_int8_form(c, a, &form, &ctas);
  if (e != cudaSuccess) return e;
  if (form == MOE_MATMUL_INT8_CLUSTER)
    return launch_t<Split>(c, a, items_at_most(a, Split::NT), ctas);
  if (form == MOE_MATMUL_INT8_PAIR) return launch_expert_matmul_int8_pair(c, a);
  const int64_t whole = items_at_most(a, Whole::NT);
  return launch_t<Whole>(c, a, whole < c.num_sms ? whole : c.num_sms, 1);
}

}  // namespace moe
