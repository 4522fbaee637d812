// balance_loss.cu -- per-expert counts, the balance loss and the z-loss of a
// router over packed sequences, and the router's score gradient.
//
// Forward.  Tokens are cut into chunks of equal length, one CTA each; a chunk
// meets one or more sequences.  Walking the chunk and sequence boundaries in
// order, every step enters the next chunk or the next sequence (or both), so
// the sums of (chunk b, sequence i) can live in row b + i of a table of
// chunks + sequences rows without any prefix sum over the sequences.  A
// second launch adds each sequence's rows in ascending order.  No float is
// added atomically: the same inputs give the same bits.
//
// A group of L lanes holds one token's scores in registers (W consecutive
// experts per access); the row's maximum, exponentials and sums come from
// those registers, so the scores are read once, which bounds both passes.
#include "block_ops.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Chunks of consecutive tokens: about kBalanceChunks of them, each a multiple
// of kWarps tokens.
constexpr int64_t kBalanceChunks = 304;
__host__ __device__ inline int64_t chunk_tokens(int64_t T) {
  const int64_t c = (T + kBalanceChunks - 1) / kBalanceChunks;
  return (c + kWarps - 1) / kWarps * kWarps;
}
inline int64_t num_chunks(int64_t T) {
  if (T <= 0) return 0;
  const int64_t c = chunk_tokens(T);
  return (T + c - 1) / c;
}
inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Workspace: [slots][E] f32 sums of p, [slots][E] i32 counts, [slots] f32 sums
// of lse^2, [slots] i32 tokens, [S][tiles] f32 partial losses, [S] u32 arrivals.
struct Work {
  float* p;
  int32_t* cnt;
  float* z;
  int32_t* n;
  float* part;
  unsigned* arrived;
  size_t bytes;
};
constexpr int kTile = 32;  // experts per CTA of the second launch
__host__ inline Work work_layout(void* ws, int64_t T, int E, int S) {
  const size_t slots = (size_t)num_chunks(T) + S;
  const size_t tiles = (size_t)(E + kTile - 1) / kTile;
  char* b = static_cast<char*>(ws);
  size_t at = 0;
  Work w;
  auto take = [&](size_t n) {
    char* q = b + at;
    at += round256(n);
    return q;
  };
  w.p = reinterpret_cast<float*>(take(slots * E * 4));
  w.cnt = reinterpret_cast<int32_t*>(take(slots * E * 4));
  w.z = reinterpret_cast<float*>(take(slots * 4));
  w.n = reinterpret_cast<int32_t*>(take(slots * 4));
  w.part = reinterpret_cast<float*>(take(S * tiles * 4));
  w.arrived = reinterpret_cast<unsigned*>(take((size_t)S * 4));
  w.bytes = at;
  return w;
}

// Sequence boundaries, kept inside [0, T] whatever the data says.
__device__ __forceinline__ int64_t seq_at(const BalanceArgs& a, int i) {
  if (a.seq == nullptr) return i == 0 ? 0 : a.T;
  const int64_t v = __ldg(a.seq + i);
  return v < 0 ? 0 : (v > a.T ? a.T : v);
}
// The first sequence that ends after token t (S if none).
__device__ __forceinline__ int first_seq(const BalanceArgs& a, int64_t t) {
  int lo = 0, hi = a.S;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (seq_at(a, mid + 1) <= t)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}

template <int L>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

constexpr float kNegInf = -INFINITY;

// Lane layout: value (v, i) of a lane is expert (v L + lane) W + i.
template <int L, int W, int NV>
struct Row {
  float x[NV * W];
  __device__ __forceinline__ static int expert(int sub, int v) { return (v * L + sub) * W; }
  // Scores of token t; -inf past E and for a token that is not wanted.
  __device__ __forceinline__ void load(const float* scores, int64_t t, int E, int sub, bool want) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = expert(sub, v);
      if constexpr (W == 4) {
        uint4 q = make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
        if (want && e < E) q = ld_stream_v4(scores + t * E + e);
        x[4 * v] = __uint_as_float(q.x);
        x[4 * v + 1] = __uint_as_float(q.y);
        x[4 * v + 2] = __uint_as_float(q.z);
        x[4 * v + 3] = __uint_as_float(q.w);
      } else {
        x[v] = want && e < E ? __ldg(scores + t * E + e) : kNegInf;
      }
    }
  }
};

// From a row's scores x: the maximum m (-inf: the token does not count), the
// log of the summed exponentials, and p in place of nothing else than `p`.
// SIG: p = sigmoid(x) / sum sigmoid.  sigmoid(x) = e^min(x,0) / (1 + e^-|x|);
// the numerators are taken relative to e^min(m,0), so a row of very negative
// scores keeps its proportions instead of underflowing.
template <int L, int N, bool SIG>
__device__ __forceinline__ void row_probs(const float (&x)[N], float (&p)[N], float (&q)[N],
                                          float* lse, bool* counts) {
  float m = kNegInf;
#pragma unroll
  for (int i = 0; i < N; ++i) m = fmaxf(m, x[i]);
  m = group_max<L>(m);
  const bool ok = m > kNegInf;
  const float mm = ok ? m : 0.0f;
  float tot = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    q[i] = expf(x[i] - mm);
    tot += q[i];
  }
  tot = group_sum<L>(tot);
  const float inv = ok ? 1.0f / tot : 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) q[i] *= inv;
  *lse = ok ? mm + logf(tot) : 0.0f;
  *counts = ok;
  if (SIG) {
    const float m0 = fminf(mm, 0.0f);
    tot = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      p[i] = expf(fminf(x[i], 0.0f) - m0) / (1.0f + expf(-fabsf(x[i])));
      tot += p[i];
    }
    tot = group_sum<L>(tot);
    const float pin = ok ? 1.0f / tot : 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] *= pin;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = q[i];
  }
}

template <int L, int W, int NV, bool SIG>
__global__ void __launch_bounds__(kThreads)
    balance_chunk_kernel(const BalanceArgs a, const Work ws, int64_t chunk, unsigned* err) {
  pdl_enter();
  extern __shared__ float smem[];  // [kWarps][E] sums of p, [E] counts, then per-warp n and z
  constexpr int N = NV * W, TPW = 32 / L;
  const int E = a.E, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % L, grp = lane / L;
  float* psum = smem;
  int* cnt = reinterpret_cast<int*>(smem + kWarps * E);
  float* wz = reinterpret_cast<float*>(cnt + E);
  int* wn = reinterpret_cast<int*>(wz + kWarps);

  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.S; i += kThreads) ws.arrived[i] = 0u;
  for (int e = threadIdx.x; e < E; e += kThreads) cnt[e] = 0;
  __syncthreads();

  const int64_t b0 = (int64_t)blockIdx.x * chunk;
  const int64_t b1 = b0 + chunk < a.T ? b0 + chunk : a.T;
  bool bad = false;
  for (int s = first_seq(a, b0); s < a.S; ++s) {
    const int64_t s0 = seq_at(a, s), s1 = seq_at(a, s + 1);
    if (s0 >= b1) break;
    const int64_t lo = s0 > b0 ? s0 : b0, hi = s1 < b1 ? s1 : b1;
    if (lo >= hi) continue;
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.0f;
    float zsum = 0.0f;
    int n = 0;
    for (int64_t t0 = lo + warp * TPW; t0 < hi; t0 += kWarps * TPW) {
      const int64_t t = t0 + grp;
      const bool want = t < hi && (a.mask == nullptr || __ldg(a.mask + t) != 0);
      Row<L, W, NV> row;
      row.load(a.scores, t, E, sub, want);
      float p[N], q[N], lse;
      bool counts;
      row_probs<L, N, SIG>(row.x, p, q, &lse, &counts);
      if (!counts) continue;  // uniform in the group; no shuffle follows
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] += p[i];
      if (sub == 0) {
        zsum = __fmaf_rn(lse, lse, zsum);
        n += 1;
      }
      for (int j = sub; j < a.k; j += L) {
        const int e = __ldg(a.idx + t * a.k + j);
        if (e >= 0 && e < E)
          atomicAdd(cnt + e, 1);
        else
          bad = true;
      }
    }
    // the warp's groups, then the block's warps, in a fixed order
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int o = 16; o >= L; o >>= 1) acc[i] += __shfl_xor_sync(0xFFFFFFFFu, acc[i], o);
    zsum = warp_sum(zsum);
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    if (grp == 0) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const int e = Row<L, W, NV>::expert(sub, v) + i;
          if (e < E) psum[warp * E + e] = acc[v * W + i];
        }
    }
    if (lane == 0) {
      wz[warp] = zsum;
      wn[warp] = n;
    }
    __syncthreads();
    const int64_t slot = (int64_t)blockIdx.x + s;
    for (int e = threadIdx.x; e < E; e += kThreads) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += psum[w * E + e];
      ws.p[slot * E + e] = v;
      ws.cnt[slot * E + e] = cnt[e];
      cnt[e] = 0;
    }
    if (threadIdx.x == 0) {
      float v = 0.0f;
      int m = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += wz[w], m += wn[w];
      ws.z[slot] = v;
      ws.n[slot] = m;
    }
    __syncthreads();
  }
  if (bad) flag_error(err, MOE_DEVERR_EXPERT_RANGE);
}

// One CTA per (sequence, 32 experts): warp w adds the sequence's table rows w,
// w + kSumWarps, ...; the CTA that arrives last at a sequence adds the tiles'
// losses in order.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(32 * kSumWarps)
    balance_sum_kernel(const BalanceArgs a, const Work ws, int64_t chunk) {
  pdl_enter();
  __shared__ float sp[kSumWarps][33];
  __shared__ int sc[kSumWarps][33];
  __shared__ float sz[kSumWarps];
  __shared__ int sn[kSumWarps];
  __shared__ int last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s = blockIdx.y, tile = blockIdx.x, e = tile * kTile + lane;
  const int64_t s0 = seq_at(a, s), s1 = seq_at(a, s + 1);
  float p = 0.0f, z = 0.0f;
  int c = 0, n = 0;
  if (s0 < s1) {
    const int64_t r0 = s0 / chunk + s, r1 = (s1 - 1) / chunk + s;
#pragma unroll 4
    for (int64_t r = r0 + warp; r <= r1; r += kSumWarps) {
      if (e < a.E) {
        p += ws.p[r * a.E + e];
        c += ws.cnt[r * a.E + e];
      }
    }
    for (int64_t r = r0 + threadIdx.x; r <= r1; r += 32 * kSumWarps) {
      z += ws.z[r];
      n += ws.n[r];
    }
  }
  z = warp_sum(z);
  n = __reduce_add_sync(0xFFFFFFFFu, n);
  sp[warp][lane] = p;
  sc[warp][lane] = c;
  if (lane == 0) {
    sz[warp] = z;
    sn[warp] = n;
  }
  __syncthreads();
  if (warp != 0) return;
  p = 0.0f, c = 0, z = 0.0f, n = 0;
#pragma unroll
  for (int w = 0; w < kSumWarps; ++w) {
    p += sp[w][lane];
    c += sc[w][lane];
    z += sz[w];
    n += sn[w];
  }
  const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
  float f = 0.0f;
  if (e < a.E) {
    const float mean = n > 0 ? p / (float)n : 0.0f;
    a.probs[(int64_t)s * a.E + e] = mean;
    a.counts[(int64_t)s * a.E + e] = c;
    f = (float)c * inv * mean;
  }
  f = warp_sum(f);
  if (lane == 0) {
    ws.part[(int64_t)s * gridDim.x + tile] = f;
    __threadfence();
    last = atomicAdd(ws.arrived + s, 1u) == gridDim.x - 1;
  }
  __syncwarp();
  if (!last) return;
  __threadfence();
  f = 0.0f;
  for (int i = lane; i < (int)gridDim.x; i += 32)
    f += *const_cast<volatile float*>(ws.part + (int64_t)s * gridDim.x + i);
  f = warp_sum(f);
  if (lane == 0) {
    a.balance[s] = f * ((float)a.E / (float)a.k);
    a.z[s] = n > 0 ? z / (float)n : 0.0f;
    a.tokens[s] = n;
  }
}

template <int L, int W, int NV, bool SIG>
__global__ void __launch_bounds__(kThreads)
    balance_backward_kernel(const BalanceArgs a, int64_t chunk, unsigned* err) {
  pdl_enter();
  extern __shared__ float smem[];  // per group: [E] gradients of the selected scores
  constexpr int N = NV * W, TPW = 32 / L;
  const int E = a.E, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % L, grp = lane / L;
  const bool sel = a.grad_w != nullptr;
  float* mine = smem + (warp * TPW + grp) * E;
  if (sel)
    for (int e = sub; e < E; e += L) mine[e] = 0.0f;
  __syncwarp();

  const int64_t b0 = (int64_t)blockIdx.x * chunk;
  const int64_t b1 = b0 + chunk < a.T ? b0 + chunk : a.T;
  bool bad = false;
  int64_t done = b0;  // tokens below it are written
  for (int s = first_seq(a, b0); done < b1; ++s) {
    // the run [done, hi) of tokens in sequence s, or in none (gaps, and the rest)
    int64_t s0 = a.T, s1 = a.T;
    if (s < a.S) s0 = seq_at(a, s), s1 = seq_at(a, s + 1);
    for (int part = 0; part < 2; ++part) {
      const bool in_seq = part == 1;
      const int64_t lo = done;
      int64_t hi = in_seq ? s1 : s0;
      if (hi > b1) hi = b1;
      if (hi <= lo) continue;
      done = hi;
      float coef[N], zc = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) coef[i] = 0.0f;
      if (in_seq) {
        const int n = __ldg(a.tokens + s);
        if (n > 0) {
          const float inv = 1.0f / (float)n;
          if (a.grad_z) zc = 2.0f * __ldg(a.grad_z + s) * inv;
          if (a.grad_balance) {
            const float gb =
                __ldg(a.grad_balance + s) * inv * inv * ((float)E / (float)a.k);
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
              for (int i = 0; i < W; ++i) {
                const int e = Row<L, W, NV>::expert(sub, v) + i;
                if (e < E) coef[v * W + i] = gb * (float)__ldg(a.counts + (int64_t)s * E + e);
              }
          }
        }
      }
      for (int64_t t0 = lo + warp * TPW; t0 < hi; t0 += kWarps * TPW) {
        const int64_t t = t0 + grp;
        const bool mine_t = t < hi;
        const bool want = in_seq && mine_t && (a.mask == nullptr || __ldg(a.mask + t) != 0);
        Row<L, W, NV> row;
        row.load(a.scores, t, E, sub, want);
        float p[N], q[N], lse;
        bool counts;
        row_probs<L, N, SIG>(row.x, p, q, &lse, &counts);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) dot = __fmaf_rn(p[i], coef[i], dot);
        dot = group_sum<L>(dot);
        float d[N];
        const float zl = zc * lse;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          float v = p[i] * (coef[i] - dot);
          if (SIG) v *= 1.0f / (1.0f + expf(row.x[i]));
          d[i] = counts ? __fmaf_rn(zl, q[i], v) : 0.0f;
        }
        if (sel) {
          float wg = 0.0f;
          for (int j = sub; j < a.k; j += L)
            if (counts) wg = __fmaf_rn(__ldg(a.w + t * a.k + j), __ldg(a.grad_w + t * a.k + j), wg);
          wg = group_sum<L>(wg);
          for (int j = sub; j < a.k; j += L) {
            if (!counts) break;
            const int e = __ldg(a.idx + t * a.k + j);
            if (e >= 0 && e < E)
              mine[e] = __ldg(a.w + t * a.k + j) * (__ldg(a.grad_w + t * a.k + j) - wg);
            else
              bad = true;
          }
          __syncwarp();
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < W; ++i) {
              const int e = Row<L, W, NV>::expert(sub, v) + i;
              if (e < E) d[v * W + i] += mine[e];
            }
          __syncwarp();
          for (int j = sub; j < a.k; j += L) {
            if (!counts) break;
            const int e = __ldg(a.idx + t * a.k + j);
            if (e >= 0 && e < E) mine[e] = 0.0f;
          }
          __syncwarp();
        }
        if (mine_t) {
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            const int e = Row<L, W, NV>::expert(sub, v);
            if (e >= E) continue;
            if constexpr (W == 4)
              st_stream_v4(a.grad_scores + t * E + e,
                           make_uint4(__float_as_uint(d[4 * v]), __float_as_uint(d[4 * v + 1]),
                                      __float_as_uint(d[4 * v + 2]),
                                      __float_as_uint(d[4 * v + 3])));
            else
              st_stream_f32(a.grad_scores + t * E + e, d[v]);
          }
        }
      }
    }
  }
  if (bad) flag_error(err, MOE_DEVERR_EXPERT_RANGE);
}

template <int L, int W, int NV, bool SIG>
cudaError_t forward_t(const LaunchCtx& c, const BalanceArgs& a) {
  const int64_t chunk = chunk_tokens(a.T), chunks = num_chunks(a.T);
  const Work ws = work_layout(a.ws, a.T, a.E, a.S);
  const size_t smem = (size_t)(kWarps + 1) * a.E * 4 + kWarps * 8;
  cudaError_t e = launch_pdl(balance_chunk_kernel<L, W, NV, SIG>, dim3((unsigned)chunks), kThreads,
                             smem, c.stream, a, ws, chunk, c.err);
  if (e != cudaSuccess) return e;
  return launch_pdl(balance_sum_kernel, dim3((unsigned)((a.E + kTile - 1) / kTile), (unsigned)a.S),
                    32 * kSumWarps, 0, c.stream, a, ws, chunk);
}

template <int L, int W, int NV, bool SIG>
cudaError_t backward_t(const LaunchCtx& c, const BalanceArgs& a) {
  const int64_t chunk = chunk_tokens(a.T), chunks = num_chunks(a.T);
  const size_t smem = a.grad_w ? (size_t)kWarps * (32 / L) * a.E * 4 : 0;
  return launch_pdl(balance_backward_kernel<L, W, NV, SIG>, dim3((unsigned)chunks), kThreads, smem,
                    c.stream, a, chunk, c.err);
}

template <int L, int W, int NV>
cudaError_t dispatch_func(const LaunchCtx& c, const BalanceArgs& a, bool backward) {
  if (a.func == MOE_SCORE_SIGMOID)
    return backward ? backward_t<L, W, NV, true>(c, a) : forward_t<L, W, NV, true>(c, a);
  return backward ? backward_t<L, W, NV, false>(c, a) : forward_t<L, W, NV, false>(c, a);
}

// Lanes per token and accesses per lane from E: 16-byte accesses where the
// rows are 16-byte aligned; a token takes only as many lanes as its scores need.
cudaError_t dispatch(const LaunchCtx& c, const BalanceArgs& a, bool backward) {
  const uintptr_t bits =
      reinterpret_cast<uintptr_t>(a.scores) | reinterpret_cast<uintptr_t>(a.grad_scores);
  const int E = a.E;
  if (E % 4 == 0 && (bits & 15u) == 0) {
    if (E <= 16) return dispatch_func<4, 4, 1>(c, a, backward);
    if (E <= 32) return dispatch_func<8, 4, 1>(c, a, backward);
    if (E <= 64) return dispatch_func<16, 4, 1>(c, a, backward);
    if (E <= 128) return dispatch_func<32, 4, 1>(c, a, backward);
    if (E <= 256) return dispatch_func<32, 4, 2>(c, a, backward);
    if (E <= 512) return dispatch_func<32, 4, 4>(c, a, backward);
    return dispatch_func<32, 4, 8>(c, a, backward);
  }
  if (E <= 8) return dispatch_func<8, 1, 1>(c, a, backward);
  if (E <= 32) return dispatch_func<32, 1, 1>(c, a, backward);
  if (E <= 128) return dispatch_func<32, 1, 4>(c, a, backward);
  if (E <= 512) return dispatch_func<32, 1, 16>(c, a, backward);
  return dispatch_func<32, 1, 32>(c, a, backward);
}

}  // namespace

size_t balance_workspace_bytes(int64_t T, int E, int S) {
  return work_layout(nullptr, T, E, S).bytes;
}

cudaError_t launch_balance_loss(const LaunchCtx& c, const BalanceArgs& a) {
  return dispatch(c, a, false);
}

cudaError_t launch_balance_loss_backward(const LaunchCtx& c, const BalanceArgs& a) {
  return dispatch(c, a, true);
}

}  // namespace moe
