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
// A small problem (see kBlockScores) is one launch of a block per sequence,
// without the table (162 tokens of 64 experts in 52 sequences: 3.4 us; 89 us with
// one block for all sequences).  The gradient's warps have a run of tokens each
// (244 tokens of 16 experts in 63 sequences: 13.7 us; 26 us with a run per block).
//
// A group of L lanes holds one token's scores in registers (W consecutive
// experts per access), and loads the next token's while it works; the
// exponentials and sums come from those registers, so the scores are read once,
// which bounds both passes.  Rows whose largest score lies in [-20, 80] (any
// router's, whatever its masked scores) need no maximum taken off: e^x, its sums
// and their inverses, and the sigmoids e^x / (1 + e^x) stay in f32's range, and what
// underflows is below 1e-29 of the row.  Other rows take the shifted form.
//
// At 65536 tokens of 256 experts (67 MB of scores) instruction issue bounds both
// passes, not HBM: 260 warp instructions per token forward (26 us, 2.7 TB/s; sigmoid 29
// us) and 463 for the sigmoid gradient with the top-k weights (36 us, 3.9 TB/s; softmax
// 32 us), about half of them on the exponentials, sums and scaling, the rest on the
// row's form (maximum, votes), its walk and its selections.  Rows all in the shifted
// form: 29 and 40 us forward, 36 and 49 us backward.  The rows' next scores are in
// flight meanwhile; without them the forward waited on its loads (43 us).
#include "block/block_ops.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512;  // forward
constexpr int kWarps = kThreads / 32;
constexpr int kBwdThreads = 256;
constexpr int kBwdWarps = kBwdThreads / 32;

// Chunks of consecutive tokens: about kBalanceChunks of them (two blocks per
// SM), each a multiple of kWarps tokens.
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
// Lanes that hold a token's scores: as many as they need, four scores each where
// the rows are 16-byte aligned (vec), else one.
inline int token_lanes(int E, bool vec) {
  if (vec) return E <= 16 ? 4 : E <= 32 ? 8 : E <= 64 ? 16 : 32;
  return E <= 8 ? 8 : 32;
}
// A block per sequence up to this many scores, and up to eight passes of a block's
// warps over all tokens for each of the first four sequences (the longest is not
// known here).  That against the table and its second launch, us:
//   one sequence, passes: E = 17, 33, 100: 4 (64 tokens) 4.0, 4.4, 4.5 : 6.4; 8 6.0,
//   6.6, 6.7 : 6.4; 16 (256 tokens) 9.8, 11 : 6.4; 61 (E = 17, 963 tokens) 31 : 7.5
//   E = 16, 12, 8: 4 4.3 : 6.6; 8 6.4 : 7.0      E = 4: 4 5.8 : 7.4; 8 9.9 : 7.9
//   E = 1: 1 2.8 : 6.4, 4 4.9 : 6.4; 8 7.8 : 6.6; 256 173 : 11.5
//   E = 256: 4 (64 tokens) 5.1 : 6.7             E = 1024: 1 (16 tokens) 5.5 : 9.4
//   four sequences of equal length: E = 33: 31 passes 6.9 : 8.5; E = 4: 16 6.7 : 8.1, 32
//   10.1 : 9.5; E = 17: 61 10.0 : 8.5; E = 3: 86 15.8 : 9.4
constexpr int64_t kBlockScores = 16384, kBlockPasses = 8, kBlockSeqs = 4;
inline bool block_per_seq(int64_t T, int E, int S, bool vec) {
  const int64_t pass = kWarps * (32 / token_lanes(E, vec));
  const int64_t most = kBlockPasses * (S < kBlockSeqs ? S : kBlockSeqs);
  return T * E <= kBlockScores && (T + pass - 1) / pass <= most;
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
// Below so many table rows per sequence the second launch takes 4 warps per CTA
// instead of 16, us at 65536 tokens, 256 experts: 1000 sequences 48 : 74, 256:
// 31 : 39, 64 (five rows each): 28.4 : 27.9, 8: 32 : 26.
constexpr int64_t kFewRows = 4;
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
// The first sequence that ends after token t (S if none).  A whole warp calls
// it: 32 boundaries are looked at per step (one load deep instead of five).
__device__ __forceinline__ int first_seq(const BalanceArgs& a, int64_t t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = a.S;  // the answer lies in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32, p = lo + lane * step;
    const int n = __popc(__ballot_sync(0xFFFFFFFFu, p < hi && seq_at(a, p + 1) <= t));
    if (n == 0) return lo;
    const int last = lo + (n - 1) * step;  // the last probe that ends by t
    if (last + step < hi) hi = last + step;
    lo = last + 1;
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

// Lane layout: value (v, i) of a lane is expert (v L + lane) W + i.  FULL: E = L W NV,
// so every lane's experts exist.
template <int L, int W, int NV, bool FULL>
struct Row {
  float x[NV * W];
  __device__ __forceinline__ static int expert(int sub, int v) { return (v * L + sub) * W; }
  // A token's scores, p its first one of this lane; -inf past E and for a token
  // that is not wanted.
  __device__ __forceinline__ void load(const float* p, int E, int sub, bool want) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const bool in = want && (FULL || expert(sub, v) < E);
      if constexpr (W == 4) {
        uint4 q = make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
        if (in) q = ld_stream_v4(p + v * L * W);
        x[4 * v] = __uint_as_float(q.x);
        x[4 * v + 1] = __uint_as_float(q.y);
        x[4 * v + 2] = __uint_as_float(q.z);
        x[4 * v + 3] = __uint_as_float(q.w);
      } else {
        x[v] = in ? __ldg(p + v * L) : kNegInf;
      }
    }
  }
  // The same, value i alone.
  __device__ __forceinline__ static float fetch(const float* p, int E, int sub, bool want, int i) {
    const int v = i / W;
    return want && (FULL || expert(sub, v) < E) ? __ldg(p + v * L * W + i % W) : kNegInf;
  }
};

// The tokens first, first + stride, ... below hi of one group of lanes, by
// offsets that move along (index products in 64 bits cost a fifth of the
// instructions).
struct Walk {
  int64_t e_at, k_at;  // this lane's first score, and its first of the k selections
  const uint8_t* mask;
  int left;  // tokens from the current one to hi
  __device__ __forceinline__ Walk(const BalanceArgs& a, int64_t first, int64_t hi, int sub, int w)
      : e_at(first * a.E + sub * w),
        k_at(first * a.k + sub),
        mask(a.mask == nullptr ? nullptr : a.mask + first),
        left(hi > first ? (int)(hi - first) : 0) {}
  __device__ __forceinline__ bool want() const {
    return left > 0 && (mask == nullptr || __ldg(mask) != 0);
  }
  __device__ __forceinline__ void step(const BalanceArgs& a, int stride) {
    e_at += (int64_t)stride * a.E;
    k_at += stride * a.k;
    if (mask != nullptr) mask += stride;
    left -= stride;
  }
};

// Whether any group of this warp (L lanes a row, N values per lane) needs the
// shifted form: its largest score is above 80, or finite and below -20.
template <int L, int N>
__device__ __forceinline__ bool far_row(const float (&x)[N], float* top_out) {
  float top = kNegInf;
#pragma unroll
  for (int i = 0; i < N; ++i) top = fmaxf(top, x[i]);
  *top_out = top;
  // groups with a finite score, and with one that is at least -20, one bit each
  unsigned some = __ballot_sync(0xFFFFFFFFu, top > kNegInf);
  unsigned near = __ballot_sync(0xFFFFFFFFu, top >= -20.0f);
  if (L == 32) {
    some = some != 0, near = near != 0;
  } else {
#pragma unroll
    for (int o = 1; o < L; o <<= 1) some |= some >> o, near |= near >> o;
  }
  constexpr unsigned kFirst = L == 4 ? 0x11111111u : L == 8 ? 0x01010101u : L == 16 ? 0x00010001u : 1u;
  return (some & ~near & kFirst) != 0 || __any_sync(0xFFFFFFFFu, top > 80.0f);
}

// The shifted form: e^(x - max), and sigmoids relative to e^min(max, 0) with
// n = 1 - sigmoid(x); the sums over the row.
template <int L, int N, bool SIG>
__device__ __forceinline__ void far_sums(const float (&x)[N], float top, float (&p)[N],
                                         float (&q)[N], float (&n)[N], float* m_out, float* tot,
                                         float* stot) {
  top = group_max<L>(top);
  const float m = top > kNegInf ? top : 0.0f, m0 = fminf(m, 0.0f);
  *m_out = top;
  float t = 0.0f, st = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    q[i] = expf(x[i] - m);
    t += q[i];
    if (SIG) {
      const float e = expf(-fabsf(x[i])), r = rcp_f32(1.0f + e);
      p[i] = expf(fminf(x[i], 0.0f) - m0) * r;
      n[i] = x[i] < 0.0f ? r : e * r;
      st += p[i];
    }
  }
  *tot = group_sum<L>(t);
  *stot = SIG ? group_sum<L>(st) : 0.0f;
}

// The log of a near row's summed exponentials `tot`.  Where tot lies near one its
// own rounding is all of the log's digits (one open expert of score 1e-3: the log
// is 1e-3, tot 1.001 to 2^-24), so there the lane's scores, score(0) to score(N - 1),
// are fetched again (kept, they would cost the registers of every row) and the log
// is taken as max + log sum e^(x - max), which is the score itself where one expert
// is open.  Outside [0.5, 2] the fast logarithm is within 3 ulp.
template <int L, int N, class Score>
__device__ __forceinline__ float near_log(float tot, Score&& score) {
  float lse = __logf(tot);
  const bool one = tot >= 0.5f && tot <= 2.0f;
  if (__any_sync(0xFFFFFFFFu, one)) {
    float top = kNegInf, t = 0.0f;
#pragma unroll 1
    for (int i = 0; i < N; ++i) top = fmaxf(top, score(i));
    top = group_max<L>(top);
#pragma unroll 1
    for (int i = 0; i < N; ++i) t += expf(score(i) - top);
    t = group_sum<L>(t);
    if (one) lse = top + logf(t);
  }
  return lse;
}

// A row's probabilities, the log of its summed exponentials, and whether the
// token counts: a score above -inf and no NaN, for which either form's sum of
// exponentials is above zero.
template <int L, int N, bool SIG, class Score>
__device__ __forceinline__ void row_probs(const float (&x)[N], float (&p)[N], float* lse,
                                          bool* counts, Score&& score) {
  float top, tot = 0.0f, stot = 0.0f;
  if (far_row<L, N>(x, &top)) {
    float q[N], n[N], m;
    far_sums<L, N, SIG>(x, top, p, q, n, &m, &tot, &stot);
    *counts = tot > 0.0f;
    *lse = *counts ? m + logf(tot) : 0.0f;
    const float inv = *counts ? 1.0f / (SIG ? stot : tot) : 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = (SIG ? p[i] : q[i]) * inv;
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    p[i] = expf(x[i]);
    tot += p[i];
    if (SIG) {
      p[i] *= rcp_f32(1.0f + p[i]);
      stot += p[i];
    }
  }
  tot = group_sum<L>(tot);
  if (SIG) stot = group_sum<L>(stot);
  *counts = tot > 0.0f;
  *lse = near_log<L, N>(tot, score);
  const float inv = *counts ? rcp_f32(SIG ? stot : tot) : 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) p[i] *= inv;
}

// A row's score gradient p (a - sum p a) [(1 - sigmoid)] + zc lse q, of no meaning
// for a token that does not count.  Near rows keep u = e^x and n = 1 - sigmoid alone:
// p = u / sum u or u n / sum (u n).  u meets its sum before it meets a coefficient:
// a may be anything finite (small losses over many tokens, a loss scale), and
// a / sum u or u a would leave f32's range.  That takes two dependent reductions;
// two values per instruction make up for it (36.2 us; 37.7 one by one).
template <int L, int N, bool SIG, class Score>
__device__ __forceinline__ void row_grad(const float (&x)[N], const float (&a)[N], float zc,
                                         float (&d)[N], bool* counts, Score&& score) {
  float top, tot = 0.0f, stot = 0.0f, n[N];
  if (far_row<L, N>(x, &top)) {
    float p[N], m, dot = 0.0f;
    far_sums<L, N, SIG>(x, top, p, d, n, &m, &tot, &stot);
    *counts = tot > 0.0f;
    const float inv = *counts ? 1.0f / tot : 0.0f, sinv = SIG && *counts ? 1.0f / stot : 0.0f;
    const float z = *counts ? zc * (m + logf(tot)) * inv : 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      p[i] = SIG ? p[i] * sinv : d[i] * inv;
      dot = __fmaf_rn(p[i], a[i], dot);
    }
    dot = group_sum<L>(dot);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float v = p[i] * (a[i] - dot);
      d[i] = __fmaf_rn(z, d[i], SIG ? v * n[i] : v);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    d[i] = expf(x[i]);
    tot += d[i];
    if (SIG) {
      n[i] = rcp_f32(1.0f + d[i]);
      stot = __fmaf_rn(d[i], n[i], stot);
    }
  }
  tot = group_sum<L>(tot);
  if (SIG) stot = group_sum<L>(stot);
  *counts = tot > 0.0f;
  const float inv = *counts ? rcp_f32(tot) : 0.0f;
  const float pinv = SIG ? (*counts ? rcp_f32(stot) : 0.0f) : inv;
  const float z = zc * near_log<L, N>(tot, score);
  float dot2[2] = {}, p[N], t[N];
  if (SIG) {
    // (e^x n lies in [0, 1]; n^2 alone underflows from x = 44 on)
    mul_v<true>(p, d, n);
    mul_v<true>(p, pinv, p);
    dot_v<true>(dot2, p, a);
    add_v<true>(t, a, -group_sum<L>(dot2[0] + dot2[1]));
    mul_v<true>(p, p, t);
    mul_v<true>(t, p, n);
    mul_v<true>(d, inv, d);
    fma_v<true>(t, z, d);
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = t[i];
  } else {
    mul_v<true>(d, inv, d);
    dot_v<true>(dot2, d, a);
    add_v<true>(t, a, z - group_sum<L>(dot2[0] + dot2[1]));
    mul_v<true>(d, d, t);
  }
}

// one: a block is a sequence, and writes its results itself.
template <int L, int W, int NV, bool SIG, bool FULL>
__global__ void __launch_bounds__(kThreads, NV * W <= 8 ? 2 : 1)
    balance_chunk_kernel(const BalanceArgs a, const Work ws, int64_t chunk, bool one,
                         unsigned* err) {
  pdl_enter();
  extern __shared__ float smem[];  // [kWarps][E] sums of p, [E] counts, then per-warp n and z
  constexpr int N = NV * W, TPW = 32 / L;
  const int E = a.E, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % L, grp = lane / L;
  float* psum = smem;
  int* cnt = reinterpret_cast<int*>(smem + kWarps * E);
  float* wz = reinterpret_cast<float*>(cnt + E);
  int* wn = reinterpret_cast<int*>(wz + kWarps);
  float* wf = reinterpret_cast<float*>(wn + kWarps);

  if (blockIdx.x == 0 && !one)
    for (int i = threadIdx.x; i < a.S; i += kThreads) ws.arrived[i] = 0u;
  for (int e = threadIdx.x; e < E; e += kThreads) cnt[e] = 0;
  __syncthreads();

  const int64_t b0 = one ? 0 : (int64_t)blockIdx.x * chunk;
  const int64_t b1 = b0 + chunk < a.T ? b0 + chunk : a.T;
  const int s_end = one ? blockIdx.x + 1 : a.S;
  bool bad = false;
  for (int s = one ? (int)blockIdx.x : first_seq(a, b0); s < s_end; ++s) {
    const int64_t s0 = seq_at(a, s), s1 = seq_at(a, s + 1);
    if (s0 >= b1 && !one) break;
    const int64_t lo = s0 > b0 ? s0 : b0, hi = s1 < b1 ? s1 : b1;
    if (lo >= hi) {
      if (one) {
        for (int e = threadIdx.x; e < E; e += kThreads) {
          a.probs[(int64_t)s * E + e] = 0.0f;
          a.counts[(int64_t)s * E + e] = 0;
        }
        if (threadIdx.x == 0) a.balance[s] = 0.0f, a.z[s] = 0.0f, a.tokens[s] = 0;
      }
      continue;
    }
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.0f;
    float zsum = 0.0f;
    int n = 0;
    Row<L, W, NV, FULL> next;
    int32_t next_e = 0;  // this lane's first index of the next token
    constexpr int kStride = kWarps * TPW;
    Walk walk(a, lo + warp * TPW + grp, hi, sub, W);
    bool now = false;  // whether the next token is wanted
    auto fetch = [&]() {
      now = walk.want();
      next.load(a.scores + walk.e_at, E, sub, now);
      if (now && sub < a.k) next_e = __ldg(a.idx + walk.k_at);
    };
    fetch();
    const int64_t mine = hi - lo - warp * TPW;
    for (int64_t done = 0; done < mine; done += kStride) {
      const Row<L, W, NV, FULL> row = next;
      const int32_t e0 = next_e;
      const int64_t k_at = walk.k_at;
      const bool want = now;
      walk.step(a, kStride);
      fetch();
      if (L == 32 && !want) continue;  // the warp's only row
      float p[N], lse;
      bool counts;
      row_probs<L, N, SIG>(row.x, p, &lse, &counts, [&](int i) {
        return row.fetch(a.scores + walk.e_at - (int64_t)kStride * E, E, sub, want, i);
      });
      if (!counts) continue;  // uniform in the group; the next shuffle waits for all groups
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] += p[i];
      if (sub == 0) {
        zsum = __fmaf_rn(lse, lse, zsum);
        n += 1;
      }
      for (int j = sub; j < a.k; j += L) {
        const int e = j == sub ? e0 : __ldg(a.idx + k_at + j - sub);
        if (e >= 0 && e < E)
          atomicAdd(cnt + e, 1);
        else
          bad = true;
      }
    }
    __syncwarp();
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
          const int e = Row<L, W, NV, FULL>::expert(sub, v) + i;
          if (FULL || e < E) psum[warp * E + e] = acc[v * W + i];
        }
    }
    if (lane == 0) {
      wz[warp] = zsum;
      wn[warp] = n;
    }
    __syncthreads();
    float z = 0.0f;
    n = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) z += wz[w], n += wn[w];
    const int64_t slot = (int64_t)blockIdx.x + s;
    float f = 0.0f;
    for (int e = threadIdx.x; e < E; e += kThreads) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += psum[w * E + e];
      const int c = cnt[e];
      cnt[e] = 0;
      if (one) {
        v = n > 0 ? v / (float)n : 0.0f;
        a.probs[(int64_t)s * E + e] = v;
        a.counts[(int64_t)s * E + e] = c;
        f = __fmaf_rn((float)c, v, f);
      } else {
        ws.p[slot * E + e] = v;
        ws.cnt[slot * E + e] = c;
      }
    }
    if (one) {
      f = warp_sum(f);
      if (lane == 0) wf[warp] = f;
      __syncthreads();
      if (threadIdx.x == 0) {
        f = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) f += wf[w];
        const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
        a.balance[s] = f * inv * ((float)E / (float)a.k);
        a.z[s] = z * inv;
        a.tokens[s] = n;
      }
    } else if (threadIdx.x == 0) {
      ws.z[slot] = z;
      ws.n[slot] = n;
    }
    __syncthreads();
  }
  if (bad) flag_error(err, MOE_DEVERR_EXPERT_RANGE);
}

// One CTA per (sequence, 32 experts): warp w of SW adds the sequence's table rows
// w, w + SW, ...; the CTA that arrives last at a sequence adds the tiles'
// losses in order.
template <int SW>
__global__ void __launch_bounds__(32 * SW)
    balance_sum_kernel(const BalanceArgs a, const Work ws, int64_t chunk) {
  pdl_enter();
  __shared__ float sp[SW][33];
  __shared__ int sc[SW][33];
  __shared__ float sz[SW];
  __shared__ int sn[SW];
  __shared__ int last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s = blockIdx.y, tile = blockIdx.x, e = tile * kTile + lane;
  const int64_t s0 = seq_at(a, s), s1 = seq_at(a, s + 1);
  float p = 0.0f, z = 0.0f;
  int c = 0, n = 0;
  if (s0 < s1) {
    const int64_t r0 = s0 / chunk + s, r1 = (s1 - 1) / chunk + s;
#pragma unroll 4
    for (int64_t r = r0 + warp; r <= r1; r += SW) {
      if (e < a.E) {
        p += ws.p[r * a.E + e];
        c += ws.cnt[r * a.E + e];
      }
    }
    for (int64_t r = r0 + threadIdx.x; r <= r1; r += 32 * SW) {
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
  for (int w = 0; w < SW; ++w) {
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

template <int L, int W, int NV, bool SIG, bool FULL>
__global__ void __launch_bounds__(kBwdThreads, NV * W <= 8 ? 3 : 1)
    balance_backward_kernel(const BalanceArgs a, int64_t run, unsigned* err) {
  pdl_enter();
  extern __shared__ __align__(16) float smem[];  // per group: [E] gradients of the selected scores
  constexpr int N = NV * W, TPW = 32 / L;
  const int E = a.E, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % L, grp = lane / L;
  const bool sel = a.grad_w != nullptr;
  float* mine = smem + (warp * TPW + grp) * E;
  if (sel)
    for (int e = sub; e < E; e += L) mine[e] = 0.0f;
  __syncwarp();

  // each warp has its own run of tokens, so that it meets few short sequences
  const int64_t b0 = ((int64_t)blockIdx.x * kBwdWarps + warp) * run;
  const int64_t b1 = b0 + run < a.T ? b0 + run : a.T;
  if (b0 >= b1) return;
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
      // the next token's scores, and this lane's first selection of it
      Row<L, W, NV, FULL> next;
      int32_t next_e = 0;
      float next_w = 0.0f, next_g = 0.0f;
      Walk walk(a, lo + grp, hi, sub, W);
      bool now = false;  // whether the next token is wanted
      auto fetch = [&]() {
        now = in_seq && walk.want();
        next.load(a.scores + walk.e_at, E, sub, now);
        if (sel && now && sub < a.k) {
          next_e = __ldg(a.idx + walk.k_at);
          next_w = __ldg(a.w + walk.k_at);
          next_g = __ldg(a.grad_w + walk.k_at);
        }
      };
      fetch();
      float coef[N], zc = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) coef[i] = 0.0f;
      if (in_seq) {
        const int n = __ldg(a.tokens + s);
        if (n > 0) {
          const float inv = 1.0f / (float)n;
          if (a.grad_z) zc = 2.0f * __ldg(a.grad_z + s) * inv;
          if (a.grad_balance) {
            const float gb = __ldg(a.grad_balance + s) * inv * ((float)E / (float)a.k);
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
              for (int i = 0; i < W; ++i) {
                const int e = Row<L, W, NV, FULL>::expert(sub, v) + i;
                if (FULL || e < E)
                  coef[v * W + i] = gb * ((float)__ldg(a.counts + (int64_t)s * E + e) * inv);
              }
          }
        }
      }
      for (int64_t at = lo; at < hi; at += TPW) {
        const bool live = walk.left > 0, want = now;
        const Row<L, W, NV, FULL> row = next;
        const int32_t e0 = next_e;
        const float w0 = next_w, g0 = next_g;
        const int64_t k_at = walk.k_at;
        float* out = a.grad_scores + walk.e_at;
        walk.step(a, TPW);
        fetch();
        float d[N];
        bool counts;
        row_grad<L, N, SIG>(row.x, coef, zc, d, &counts, [&](int i) {
          return row.fetch(a.scores + (out - a.grad_scores), E, sub, want, i);
        });
        if (!counts) {  // (a NaN is no zero times the row's inverse sum)
#pragma unroll
          for (int i = 0; i < N; ++i) d[i] = 0.0f;
        }
        if (sel) {
          // this lane's selections sub, sub + L, ...: the first is at hand
          float wg = counts && sub < a.k ? w0 * g0 : 0.0f;
          if (a.k > L && counts)
            for (int j = sub + L; j < a.k; j += L)
              wg = __fmaf_rn(__ldg(a.w + k_at + j - sub), __ldg(a.grad_w + k_at + j - sub), wg);
          wg = group_sum<L>(wg);
          if (counts) {
            if (sub < a.k) {
              if (e0 >= 0 && e0 < E)
                mine[e0] = w0 * (g0 - wg);
              else
                bad = true;
            }
            if (a.k > L)
              for (int j = sub + L; j < a.k; j += L) {
                const int e = __ldg(a.idx + k_at + j - sub);
                if (e >= 0 && e < E)
                  mine[e] = __ldg(a.w + k_at + j - sub) * (__ldg(a.grad_w + k_at + j - sub) - wg);
                else
                  bad = true;
              }
          }
          __syncwarp();
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int e = Row<L, W, NV, FULL>::expert(sub, v);
          if (!FULL && e >= E) continue;
          if constexpr (W == 4) {
            if (sel) {
              const float4 m = *reinterpret_cast<const float4*>(mine + e);
              d[4 * v] += m.x, d[4 * v + 1] += m.y, d[4 * v + 2] += m.z, d[4 * v + 3] += m.w;
            }
            if (live)
              st_stream_v4(out + v * L * W,
                           make_uint4(__float_as_uint(d[4 * v]), __float_as_uint(d[4 * v + 1]),
                                      __float_as_uint(d[4 * v + 2]),
                                      __float_as_uint(d[4 * v + 3])));
          } else {
            if (sel) d[v] += mine[e];
            if (live) st_stream_f32(out + v * L, d[v]);
          }
        }
        if (sel) {
          __syncwarp();
          if (counts) {
            if (sub < a.k && e0 >= 0 && e0 < E) mine[e0] = 0.0f;
            if (a.k > L)
              for (int j = sub + L; j < a.k; j += L) {
                const int e = __ldg(a.idx + k_at + j - sub);
                if (e >= 0 && e < E) mine[e] = 0.0f;
              }
          }
          __syncwarp();
        }
      }
    }
  }
  if (bad) flag_error(err, MOE_DEVERR_EXPERT_RANGE);
}

// Whether the rows take 16-byte accesses.
inline bool rows_vec(const BalanceArgs& a, bool backward) {
  uintptr_t bits = reinterpret_cast<uintptr_t>(a.scores);
  if (backward) bits |= reinterpret_cast<uintptr_t>(a.grad_scores);
  return a.E % 4 == 0 && (bits & 15u) == 0;
}

template <int L, int W, int NV, bool SIG, bool FULL>
cudaError_t forward_t(const LaunchCtx& c, const BalanceArgs& a) {
  const bool one = block_per_seq(a.T, a.E, a.S, rows_vec(a, false));
  const int64_t chunk = one ? a.T : chunk_tokens(a.T), chunks = one ? a.S : num_chunks(a.T);
  const Work ws = work_layout(a.ws, a.T, a.E, a.S);
  const size_t smem = (size_t)(kWarps + 1) * a.E * 4 + kWarps * 12;
  auto* kernel = balance_chunk_kernel<L, W, NV, SIG, FULL>;
  static SmemOptIn opt_in;
  cudaError_t e = smem > 48 * 1024 ? opt_in.once(kernel) : cudaSuccess;
  if (e != cudaSuccess) return e;
  e = launch_pdl(kernel, dim3((unsigned)chunks), kThreads, smem, c.stream, a, ws, chunk, one,
                 c.err);
  if (e != cudaSuccess || one) return e;
  const dim3 grid((unsigned)((a.E + kTile - 1) / kTile), (unsigned)a.S);
  if (chunks / a.S < kFewRows)
    return launch_pdl(balance_sum_kernel<4>, grid, 128, 0, c.stream, a, ws, chunk);
  return launch_pdl(balance_sum_kernel<16>, grid, 512, 0, c.stream, a, ws, chunk);
}

template <int L, int W, int NV, bool SIG, bool FULL>
cudaError_t backward_t(const LaunchCtx& c, const BalanceArgs& a) {
  // eight blocks' worth of tokens per SM, at least one pass of a block's warps
  constexpr int kPass = kBwdWarps * (32 / L);
  int64_t chunk = (a.T + 8 * c.num_sms - 1) / (8 * c.num_sms);
  chunk = (chunk + kPass - 1) / kPass * kPass;
  const int64_t chunks = (a.T + chunk - 1) / chunk;
  const size_t smem = a.grad_w ? (size_t)kPass * a.E * 4 : 0;
  return launch_pdl(balance_backward_kernel<L, W, NV, SIG, FULL>, dim3((unsigned)chunks), kBwdThreads,
                    smem, c.stream, a, chunk / kBwdWarps, c.err);
}

template <int L, int W, int NV, bool FULL>
cudaError_t dispatch_func(const LaunchCtx& c, const BalanceArgs& a, bool backward) {
  if (a.func == MOE_SCORE_SIGMOID)
    return backward ? backward_t<L, W, NV, true, FULL>(c, a)
                    : forward_t<L, W, NV, true, FULL>(c, a);
  return backward ? backward_t<L, W, NV, false, FULL>(c, a)
                  : forward_t<L, W, NV, false, FULL>(c, a);
}
template <int L, int W, int NV>
cudaError_t dispatch_full(const LaunchCtx& c, const BalanceArgs& a, bool backward) {
  return a.E == L * W * NV ? dispatch_func<L, W, NV, true>(c, a, backward)
                           : dispatch_func<L, W, NV, false>(c, a, backward);
}

// Lanes per token (token_lanes) and accesses per lane.
cudaError_t dispatch(const LaunchCtx& c, const BalanceArgs& a, bool backward) {
  const int E = a.E;
  if (rows_vec(a, backward)) {
    if (E <= 16) return dispatch_full<4, 4, 1>(c, a, backward);
    if (E <= 32) return dispatch_full<8, 4, 1>(c, a, backward);
    if (E <= 64) return dispatch_full<16, 4, 1>(c, a, backward);
    if (E <= 128) return dispatch_full<32, 4, 1>(c, a, backward);
    if (E <= 256) return dispatch_full<32, 4, 2>(c, a, backward);
    if (E <= 512) return dispatch_full<32, 4, 4>(c, a, backward);
    return dispatch_full<32, 4, 8>(c, a, backward);
  }
  if (E <= 8) return dispatch_func<8, 1, 1, false>(c, a, backward);
  if (E <= 32) return dispatch_func<32, 1, 1, false>(c, a, backward);
  if (E <= 128) return dispatch_func<32, 1, 4, false>(c, a, backward);
  if (E <= 256) return dispatch_func<32, 1, 8, false>(c, a, backward);
  if (E <= 512) return dispatch_func<32, 1, 16, false>(c, a, backward);
  return dispatch_func<32, 1, 32, false>(c, a, backward);
}

}  // namespace

size_t balance_workspace_bytes(int64_t T, int E, int S, bool aligned) {
  if (block_per_seq(T, E, S, aligned && E % 4 == 0)) return 0;
  return work_layout(nullptr, T, E, S).bytes;
}

cudaError_t launch_balance_loss(const LaunchCtx& c, const BalanceArgs& a) {
  return dispatch(c, a, false);
}

cudaError_t launch_balance_loss_backward(const LaunchCtx& c, const BalanceArgs& a) {
  return dispatch(c, a, true);
}

}  // namespace moe
