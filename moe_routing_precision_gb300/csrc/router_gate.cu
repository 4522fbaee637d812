// router_gate.cu -- the router with a bias for balance and groups of experts, and
// the gradient of its weights.
//
//   s = softmax(x) or sigmoid(x);  c = s + bias, -inf where x is -inf
//   the g groups with the largest max, or sum of the two largest, of c; among their
//   experts the k with the largest c; ties to the lower group and expert
//   w_j = scale s_j / sum s, or scale s_j
//
// The selection is that of the real numbers.  Without a bias c orders the experts as
// x does, and they are compared by x, exactly.  Otherwise c is taken in f32 with a
// bounded error (score_err); where two values at a border of the selection lie closer
// than that, the token is decided again in f64, one value per candidate, which is rare:
// about one token in a thousand for 8 of 256 experts.
//
// A token has a warp, or 4 to 16 lanes of one, lane l holding the V consecutive experts
// l V .. l V + V - 1, so that a group is a run of lanes.  The selection is topk_warp.cuh's:
// a lower bound of the k-th value from the lanes' two largest leaves a few candidates,
// ranked against one another.
#include <type_traits>

#include "block/block_ops.cuh"
#include "topk_warp.cuh"

namespace moe {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kWarps = 8;
// Several tokens per warp: tokens per SM from which on, warps of a block, blocks per SM.
constexpr int kLanesFrom = 12, kLaneWarps = 4, kLaneBlocks = 4;
constexpr float kInf = __builtin_huge_valf();
constexpr float kLog2e = 1.4426950408889634f;

// A difference of two f32 c is off by at most 2 score_err + 2^-23 (|c| + |c'|).  Both forms
// take 2^y and 1 / y from the hardware estimates (2 ulp and 1 ulp).
// Sigmoid: e = 2^(-x log2 e) is off by (3 |x| + 4) 2^-24 e, which moves s by less than
// s (1 - s) times that, under 2^-23; the sum and the estimate of its inverse add 3 * 2^-24.
// Softmax: e = 2^((x - max) log2 e) in the same way, |x - max| e^(x - max) < 0.37: within
// 5.1 * 2^-24 of the largest score for each.  The sum of 1024 terms (at most 36 roundings in
// sequence), the terms' own errors and the inverse put all scores of a row off by one factor,
// within 43 * 2^-24, and so the difference of two by that part of the largest: 54 * 2^-24 in
// all, against 64 * 2^-24.
__device__ __forceinline__ float score_err(int func, float top) {
  return func == MOE_SCORE_SIGMOID ? 0x1p-21f : 0x1p-19f * top;
}
__device__ __forceinline__ float exp2_est(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_est(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The largest and the second of a group.
struct Top2 {
  float a, b;
};
__device__ __forceinline__ void merge(Top2& t, float v) {
  t.b = fmaxf(t.b, fminf(t.a, v));
  t.a = fmaxf(t.a, v);
}
__device__ __forceinline__ void merge(Top2& t, Top2 o) {
  t.b = fmaxf(fminf(t.a, o.a), fmaxf(t.b, o.b));
  t.a = fmaxf(t.a, o.a);
}
__device__ __forceinline__ bool both_count(const Top2& t, int kind) {
  return kind == MOE_GROUP_TOP2 && t.b > -kInf;
}
__device__ __forceinline__ float group_value(const Top2& t, int kind) {
  return both_count(t, kind) ? t.a + t.b : t.a;
}
// How far group_value may be off, err being score_err: by the errors of its one or two
// values, which their sum does not show where they cancel (biases of both signs).  3 * 2^-24
// of each covers the rounding of s + bias, of the sum, and of the sum plus or minus this.
__device__ __forceinline__ float group_err(const Top2& t, int kind, float err) {
  const float size = fabsf(t.a) + (both_count(t, kind) ? fabsf(t.b) : 0.0f);
  return t.a > -kInf ? __fmaf_rn(0x1p-22f, size, 2.0f * err) : 0.0f;
}
// The value from which on an expert of a group at the border may be one of those that count:
// the second (the first, where only that counts) less what the errors of two values may hide.
__device__ __forceinline__ float group_edge(const Top2& t, int kind, float err) {
  const float v = both_count(t, kind) ? t.b : t.a;
  return v - __fmaf_rn(0x1p-21f, fabsf(v), 2.0f * err);
}

__device__ __forceinline__ float warp_max(float v) {
  return key_score(__reduce_max_sync(kAll, score_key(v)));
}
__device__ __forceinline__ float warp_min(float v) {
  return key_score(__reduce_min_sync(kAll, score_key(v)));
}

// ------------------------------------------------ what f32 cannot tell, in f64

__device__ __forceinline__ double sigmoid64(double x) {
  const double e = exp(-fabs(x));
  return x < 0.0 ? e / (1.0 + e) : 1.0 / (1.0 + e);
}
// c of an expert with score x; m and z: the softmax's largest x and sum of exp(x - m).
__device__ __forceinline__ double choice64(int func, float x, const float* bias, int e, float m,
                                           double z) {
  if (x == -kInf) return -__builtin_huge_val();
  const double s =
      func == MOE_SCORE_SIGMOID ? sigmoid64((double)x) : exp((double)x - (double)m) / z;
  return bias ? s + (double)__ldg(bias + e) : s;
}
__device__ __forceinline__ double sum64(const float* row, int E, float m, int lane) {
  double z = 0.0;
  for (int e = lane; e < E; e += 32) z += exp((double)__ldg(row + e) - (double)m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kAll, z, o);
  return z;
}

// An order-preserving integer of a non-NaN value; 0 is below all of them.
__device__ __forceinline__ unsigned long long order64(double d) {
  const long long b = __double_as_longlong(d + 0.0);  // -0 + 0 = +0
  return (unsigned long long)b ^ ((unsigned long long)(b >> 63) | (1ull << 63));
}

// The groups at the border decided again.  Lane i < G is group i: `sure` those that stay
// whatever the errors, `near` those that may; lane j < C holds expert e of a near group,
// all that may be among its group's two largest.  s_v, s_e: scratch of 32.
__device__ __noinline__ uint32_t groups64(const float* row, const float* bias, int func, float m,
                                          int E, int n, int g, int kind, uint32_t sure,
                                          uint32_t near, int C, int e, int lane, double* s_v,
                                          int* s_e) {
  const double z = func == MOE_SCORE_SOFTMAX ? sum64(row, E, m, lane) : 1.0;
  const double none = -__builtin_huge_val();
  if (lane < C) {
    s_v[lane] = choice64(func, __ldg(row + e), bias, e, m, z);
    s_e[lane] = e / n;
  }
  __syncwarp();
  unsigned long long key = 0ull;
  if ((near >> lane) & 1u) {
    double a = none, b = none;
    for (int j = 0; j < C; ++j) {
      if (s_e[j] != lane) continue;
      const double c = s_v[j];
      if (c > a) {
        b = a, a = c;
      } else if (c > b) {
        b = c;
      }
    }
    key = order64(kind == MOE_GROUP_TOP2 && b > none ? a + b : a);
  }
  int rank = __popc(sure);
  for (uint32_t left = near; left; left &= left - 1) {
    const int i = __ffs(left) - 1;
    const unsigned long long o = __shfl_sync(kAll, key, i);
    rank += o > key || (o == key && i < lane) ? 1 : 0;
  }
  return sure | __ballot_sync(kAll, ((near >> lane) & 1u) && rank < g);
}

// The same for all groups from scratch.
__device__ __noinline__ uint32_t all_groups64(const float* row, const float* bias, int func,
                                              float m, int E, int G, int g, int kind, int lane) {
  const double z = func == MOE_SCORE_SOFTMAX ? sum64(row, E, m, lane) : 1.0;
  const double none = -__builtin_huge_val();
  const int n = E / G;
  unsigned long long key = 0ull;
  for (int i = 0; i < G; ++i) {  // each group in turn by the whole warp
    double a = none, b = none;
    for (int e = i * n + lane; e < (i + 1) * n; e += 32) {
      const double c = choice64(func, __ldg(row + e), bias, e, m, z);
      b = fmax(b, fmin(a, c));
      a = fmax(a, c);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double oa = __shfl_xor_sync(kAll, a, o), ob = __shfl_xor_sync(kAll, b, o);
      b = fmax(fmin(a, oa), fmax(b, ob));
      a = fmax(a, oa);
    }
    if (lane == i) key = order64(kind == MOE_GROUP_TOP2 && b > none ? a + b : a);
  }
  int rank = 0;
  for (int i = 0; i < G; ++i) {
    const unsigned long long o = __shfl_sync(kAll, key, i);
    rank += o > key || (o == key && i < lane) ? 1 : 0;
  }
  return __ballot_sync(kAll, lane < G && rank < g);
}

// Whether all scores of a row are one value, and all biases: then ties are exact.
__device__ __noinline__ bool one_value(const float* row, const float* bias, int E, int lane) {
  float xl = kInf, xh = -kInf, bl = kInf, bh = -kInf;
  for (int e = lane; e < E; e += 32) {
    const float x = __ldg(row + e), b = bias ? __ldg(bias + e) : 0.0f;
    xl = fminf(xl, x), xh = fmaxf(xh, x), bl = fminf(bl, b), bh = fmaxf(bh, b);
  }
  return warp_min(xl) == warp_max(xh) && warp_min(bl) == warp_max(bh);
}

// Ranks of C candidates, expert e in lane < C: by x (exact), or by c in f64.
__device__ __noinline__ int rank64(const float* row, const float* bias, int func, float m, int E,
                                   bool by_x, int e, int C, int lane) {
  const double z = !by_x && func == MOE_SCORE_SOFTMAX ? sum64(row, E, m, lane) : 1.0;
  unsigned long long d = 0ull;
  if (lane < C) {
    const float x = __ldg(row + e);
    d = by_x ? score_key(x) : order64(choice64(func, x, bias, e, m, z));
  }
  int rank = 0;
  for (int j = 0; j < C; ++j) {
    const unsigned long long od = __shfl_sync(kAll, d, j);
    const int oe = __shfl_sync(kAll, e, j);
    rank += od > d || (od == d && oe < e) ? 1 : 0;
  }
  return rank;
}

// The k winners of the open groups one after the other, the r-th in lane r, where there
// are more candidates than lanes.  list: [E], order-preserving integers.
__device__ __noinline__ int select64(const float* row, const float* bias, int func, float m,
                                     int E, int n, uint32_t open, int k, int lane,
                                     unsigned long long* list) {
  const double z = func == MOE_SCORE_SOFTMAX ? sum64(row, E, m, lane) : 1.0;
  for (int e = lane; e < E; e += 32) {
    unsigned long long key = 0ull;
    if ((open >> (e / n)) & 1u)
      key = order64(choice64(func, __ldg(row + e), bias, e, m, z));
    list[e] = key;
  }
  __syncwarp();
  int mine = 0;
  for (int r = 0; r < k; ++r) {
    unsigned long long best = 0ull;
    int at = E;
    for (int e = lane; e < E; e += 32)
      if (list[e] > best) best = list[e], at = e;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long ob = __shfl_xor_sync(kAll, best, o);
      const int oa = __shfl_xor_sync(kAll, at, o);
      if (ob > best || (ob == best && oa < at)) best = ob, at = oa;
    }
    if (lane == r) mine = at;
    if (lane == 0 && at < E) list[at] = 0ull;
    __syncwarp();
  }
  return mine;
}

// ------------------------------------------------------------------- weights

// The scores of the selected experts (one per lane, have: this lane's is one) for the
// weights: s itself, or with `ratio` s times a factor that all of them share.
__device__ __forceinline__ float weight_score(int func, bool ratio, float x, bool have, float m,
                                              float z_inv) {
  if (func == MOE_SCORE_SOFTMAX) {
    const float top = ratio ? warp_max(have ? x : -kInf) : m;
    return have && x > -kInf ? expf(x - top) * (ratio ? 1.0f : z_inv) : 0.0f;
  }
  // s = e^min(x,0) / (1 + e^-|x|): with the largest min(x, 0) taken off, the ratio of
  // scores far below f32's range keeps its digits
  const float lo = fminf(x, 0.0f);
  const float top = ratio ? warp_max(have ? lo : -kInf) : 0.0f;
  return have && x > -kInf ? expf(lo - top) * rcp_f32(1.0f + expf(-fabsf(x))) : 0.0f;
}

// ------------------------------------------------------------------- forward

struct WarpScratch {
  float c[36];  // the candidates' c, then -inf up to a multiple of four
  float by_rank[36];
  double v64[32];
  int e[32];
};

// f32 c of one expert, as the kernel takes it; -inf where x is -inf (for the sigmoid by a
// bound that no other x brings below 2^126).
__device__ __forceinline__ float choice32(int func, float x, float b, float m, float z_inv) {
  return func == MOE_SCORE_SIGMOID
             ? fminf(rcp_est(1.0f + exp2_est(x * -kLog2e)) + b, __fmaf_rn(x, 0x1p-60f, 0x1p127f))
             : (x > -kInf ? __fmaf_rn(exp2_est((x - m) * kLog2e), z_inv, b) : -kInf);
}

// One token with every border looked at, by one warp: where f32 cannot tell, in f64.
// list: [E] words of scratch.
__device__ __noinline__ void careful_token(const RouterArgs& a, int64_t t, int lane,
                                           WarpScratch& ws, unsigned long long* list) {
  const int E = a.E, k = a.k, n = E / a.G;
  const float* row = a.scores + t * E;
  float* c = reinterpret_cast<float*>(list);
  const bool by_x = a.bias == nullptr;  // c orders the experts as x does
  const bool grouped = a.g < a.G;
  const bool need_c = !by_x || (grouped && a.group_score == MOE_GROUP_TOP2);
  float m = 0.0f, z_inv = 0.0f, err = 0.0f;
  __syncwarp();
  if (a.func == MOE_SCORE_SOFTMAX) {
    m = -kInf;
    for (int e = lane; e < E; e += 32) m = fmaxf(m, __ldg(row + e));
    m = warp_max(m);
    if (m == -kInf) m = 0.0f;
    float z = 0.0f;
    for (int e = lane; e < E; e += 32) z += exp2_est((__ldg(row + e) - m) * kLog2e);
    z = warp_sum(z);
    z_inv = z > 0.0f ? rcp_f32(z) : 0.0f;
  }
  for (int e = lane; e < E; e += 32) {
    const float x = __ldg(row + e);
    c[e] = need_c ? choice32(a.func, x, by_x ? 0.0f : __ldg(a.bias + e), m, z_inv) : x;
  }
  if (need_c) err = score_err(a.func, a.func == MOE_SCORE_SIGMOID ? 1.0f : z_inv);
  __syncwarp();

  // ---- groups, one per lane
  uint32_t open = kAll >> (32 - a.G);
  if (grouped) {
    Top2 g2 = {-kInf, -kInf};
    if (lane < a.G)
      for (int e = 0; e < n; ++e) merge(g2, c[lane * n + e]);
    const float gv = group_value(g2, a.group_score);
    int rank = 0;
    for (int i = 0; i < a.G; ++i) {
      const float o = __shfl_sync(kAll, gv, i);
      rank += o > gv || (o == gv && i < lane) ? 1 : 0;
    }
    open = __ballot_sync(kAll, lane < a.G && rank < a.g);
    // the least that a group inside may be against the most that one outside may be
    const bool in = rank < a.g;
    const float spread = group_err(g2, a.group_score, err);
    const float low = warp_min(lane < a.G && in ? gv - spread : kInf);
    const float high = warp_max(lane < a.G && !in ? gv + spread : -kInf);
    // unless the whole row is one value: those ties are exact
    if (need_c && high > -kInf && low <= high && !one_value(row, a.bias, E, lane)) {
      const uint32_t near = __ballot_sync(
          kAll, lane < a.G && (in ? gv - spread <= high : gv + spread >= low));
      // the near groups' experts that may be among the two largest
      const float edge = group_edge(g2, a.group_score, err);
      int C = 0;
      for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + lane, gi = e / n;
        const float from = __shfl_sync(kAll, edge, gi & 31);
        const bool take = e < E && (near >> (gi & 31) & 1u) && c[e] >= from;
        const uint32_t b = __ballot_sync(kAll, take);
        const int at = C + __popc(b & ((1u << lane) - 1u));
        if (take && at < 32) ws.e[at] = e;
        C += __popc(b);
      }
      __syncwarp();
      const int e = lane < C ? ws.e[lane] : 0;
      __syncwarp();
      if (C <= 32)
        open = groups64(row, a.bias, a.func, m, E, n, a.g, a.group_score, open & ~near, near, C, e,
                        lane, ws.v64, ws.e);
      else  // a bundle of equal experts: each group in turn
        open = all_groups64(row, a.bias, a.func, m, E, a.G, a.g, a.group_score, lane);
    }
  }

  // ---- the experts of open groups, round by round: the k largest, one more for the
  // border, and as many more as lie too close to it
  const float none = __int_as_float(0x7FFFFFFF), twice = 2.0f * err;
  __syncwarp();
  for (int e = lane; e < E; e += 32)
    c[e] = !((open >> (e / n)) & 1u) ? none : by_x ? __ldg(row + e) : c[e];
  __syncwarp();
  bool again = false, more = false;
  float last = 0.0f, edge = 0.0f;
  int sel = 0, slot = k, r = 0;
  for (;; ++r) {
    uint32_t best = 0;
    int at = 0;
    for (int e = lane; e < E; e += 32) {
      const float v = c[e];
      const uint32_t key = v == v ? score_key(v) : 0u;
      if (key > best) best = key, at = e;
    }
    const uint32_t win = __reduce_max_sync(kAll, best);
    if (win == 0u) break;
    const float v = key_score(win);
    const bool near = r > 0 && !by_x && v > -kInf &&
                      last - v <= twice + 0x1p-22f * fmaxf(fabsf(last), fabsf(v));
    if (r <= k) again = again || near;
    if (r == k - 1) edge = v;
    // past the k-th: only those that may change places with it
    if (r >= k && (!again || edge - v > twice + 0x1p-22f * fmaxf(fabsf(edge), fabsf(v)))) break;
    more = r == 32;  // no lane left
    if (more) break;
    last = v;
    const int e = (int)__reduce_min_sync(kAll, best == win ? (uint32_t)at : ~0u);
    if (lane == r) sel = e, slot = r;
    if (lane == 0) c[e] = none;
    __syncwarp();
  }
  if (again && more) {
    // the border hides more experts than there are lanes
    sel = select64(row, a.bias, a.func, m, E, n, open, k, lane, list);
    slot = lane;
  } else if (again) {
    const int rank = rank64(row, a.bias, a.func, m, E, by_x, sel, r, lane);
    slot = lane < r ? rank : k;
  }

  // ---- weights
  const bool have = slot < k;
  const float xs = have ? __ldg(row + sel) : -kInf;
  float w = weight_score(a.func, a.renorm, xs, have, m, z_inv);
  if (a.renorm) {
    const float sum = warp_sum(w);
    w = sum > 0.0f ? w * rcp_f32(sum) : 0.0f;
  }
  if (have) {
    a.idx[t * k + slot] = sel;
    a.w[t * k + slot] = w * a.scale;
  }
  __syncwarp();
}

// How the experts are compared: by x; by c of a sigmoid; by c of a softmax.
constexpr int kByX = 0, kSigmoid = 1, kSoftmax = 2;

// One warp per token.  V experts per lane; VEC: E = 32 V, V % 4 == 0 and 16-byte aligned
// rows; KFIX > 0: k.  A token with more unsettled experts than a warp has lanes is noted
// and done again at the end (careful_token, 10 us), which keeps that work's registers out
// of the loop.
//
// For few tokens, for selections by x, and for numbers of experts and groups that
// router_gate_lanes_kernel does not divide.  65536 tokens, 8 of 256 experts (67 MB; us):
// by x alone 26; sigmoid and bias 42; with 8 groups 50 (640 instructions per token, 70 % of
// the issue slots; the rest waits in one token's chain of reductions).  k = 32: 373, for k
// rounds of reductions, and as many again where there are more than 32 candidates.  A
// border decided in f64 costs its warp 1.2 us for experts and 3 us for groups.  Asking for a
// row ahead was slower.
template <int V, bool VEC, int KFIX, int MODE>
__global__ void __launch_bounds__(kWarps * 32, V <= 8 ? 4 : V <= 16 ? 2 : 1)
    router_gate_kernel(const RouterArgs a) {
  __shared__ __align__(16) WarpScratch s_scratch[kWarps];
  extern __shared__ unsigned long long s_list[];  // [kWarps][E]
  pdl_enter();
  const int lane = threadIdx.x & 31, wib = threadIdx.x >> 5;
  WarpScratch& ws = s_scratch[wib];
  const int E = VEC ? 32 * V : a.E;
  const int k = KFIX > 0 ? KFIX : a.k, n = E / a.G;
  unsigned long long* list = s_list + (size_t)wib * E;
  float* s_c = reinterpret_cast<float*>(list);
  const int warps = (int)((gridDim.x * blockDim.x) >> 5);
  // groups that are a power of two of whole lanes are merged by shuffles; others
  // through shared memory by L lanes each
  const int run = n % V == 0 ? n / V : 0;
  const bool runs = run > 0 && (run & (run - 1)) == 0;
  int L = 32;
  while (L > 1 && L * a.G > 32) L >>= 1;
  const int width = runs ? run : L;  // lanes of a group
  const int my_group = lane / width, from_lane = (lane * width) & 31;
  const uint32_t inv_n = ((1u << 21) + n - 1) / n;  // e / n = e inv_n >> 21 for e < 1024
  const int present = VEC ? V : (E - lane * V < 0 ? 0 : E - lane * V > V ? V : E - lane * V);
  const bool by_x = MODE == kByX || a.bias == nullptr;
  const bool grouped = a.g < a.G;
  float bias[V];
  if constexpr (MODE != kByX) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      bias[i] = !by_x && i < present ? __ldg(a.bias + lane * V + i) : 0.0f;
  }
  const float none = __int_as_float(0x7FFFFFFF);  // NaN: a slot that is no candidate
  uint32_t careful = 0;                           // tokens to be done again

  const int64_t t0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  int64_t t = t0;
  for (int turn = 0; t < a.T; t += warps, ++turn) {
    const float* row = a.scores + t * E;
    float c[V];
    auto load_x = [&]() {
      if constexpr (VEC) {
#pragma unroll
        for (int h = 0; h < V / 4; ++h) {
          const float4 f = __ldg(reinterpret_cast<const float4*>(row + lane * V + 4 * h));
          c[4 * h] = f.x, c[4 * h + 1] = f.y, c[4 * h + 2] = f.z, c[4 * h + 3] = f.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = i < present ? __ldg(row + lane * V + i) : -kInf;
      }
    };
    load_x();
    // ---- c, and the softmax's largest x and inverse sum
    float m = 0.0f, z_inv = 0.0f, err = 0.0f;
    if (MODE == kSoftmax || (MODE == kByX && a.func == MOE_SCORE_SOFTMAX && !a.renorm)) {
      m = c[0];
#pragma unroll
      for (int i = 1; i < V; ++i) m = fmaxf(m, c[i]);
      m = warp_max(m);
      if (m == -kInf) m = 0.0f;
      float z = 0.0f, ex[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        ex[i] = exp2_est((c[i] - m) * kLog2e);
        z += ex[i];
      }
      z = warp_sum(z);
      z_inv = z > 0.0f ? rcp_f32(z) : 0.0f;
      if constexpr (MODE == kSoftmax) {
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = c[i] > -kInf ? __fmaf_rn(ex[i], z_inv, bias[i]) : -kInf;
        err = score_err(MOE_SCORE_SOFTMAX, z_inv);
      }
    } else if constexpr (MODE == kSigmoid) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        c[i] = choice32(MOE_SCORE_SIGMOID, c[i], bias[i], 0.0f, 0.0f);
      err = score_err(MOE_SCORE_SIGMOID, 1.0f);
    }

    // ---- the lane's two largest, and the groups
    Top2 l2 = {c[0], -kInf};
#pragma unroll
    for (int i = 1; i < V; ++i) merge(l2, c[i]);
    uint32_t open = kAll;
    bool settled = true;  // f32 tells
    if (grouped) {
      Top2 g2 = l2;
      if (!runs) {
        g2 = Top2{-kInf, -kInf};
        __syncwarp();
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i < present) s_c[lane * V + i] = c[i];
        __syncwarp();
        if (my_group < a.G)
          for (int e = lane % L; e < n; e += L) merge(g2, s_c[my_group * n + e]);
      }
      for (int o = 1; o < width; o <<= 1)
        merge(g2, Top2{__shfl_xor_sync(kAll, g2.a, o), __shfl_xor_sync(kAll, g2.b, o)});
      const float gv = __shfl_sync(kAll, group_value(g2, a.group_score), from_lane);
      // the groups of the g largest distinct values; more than g of them: ties
      [[maybe_unused]] const float spread =
          MODE == kByX ? 0.0f
                       : __shfl_sync(kAll, group_err(g2, a.group_score, err), from_lane);
      const uint32_t gkey = lane < a.G ? score_key(gv) : 0u;
      uint32_t edge_in = 0, left = gkey;
      for (int r = 0; r < a.g; ++r) {
        edge_in = __reduce_max_sync(kAll, left);
        if (left == edge_in) left = 0u;
      }
      open = __ballot_sync(kAll, gkey >= edge_in && gkey > 0u);
      const bool ties = __popc(open) != a.g;
      if (MODE != kByX && ties) {  // the g-th largest value, each group counted
        left = gkey;
        for (int count = 0; count < a.g;) {
          edge_in = __reduce_max_sync(kAll, left);
          count += __popc(__ballot_sync(kAll, left == edge_in));
          if (left == edge_in) left = 0u;
        }
      }
      if constexpr (MODE == kByX) {
        if (ties) {  // of the last value that has a place, the first groups
          uint32_t all = kAll >> (32 - a.G);
          open = 0u;
          for (int r = 0; r < a.g; ++r) {
            const uint32_t best =
                __reduce_max_sync(kAll, (all >> lane & 1u) ? gkey : 0u);
            const uint32_t who = __ballot_sync(kAll, gkey == best) & all;
            open |= who & (0u - who);
            all &= ~(who & (0u - who));
          }
        }
      } else {
        // the least that a group inside may be against the most that one outside may be;
        // of ties at the border each group is on both sides
        const bool inside = lane < a.G && gkey >= edge_in;
        const bool outside = lane < a.G && (ties ? gkey <= edge_in : gkey < edge_in);
        const float low = warp_min(inside ? gv - spread : kInf);
        const float high = warp_max(outside ? gv + spread : -kInf);
        if (ties || (high > -kInf && low <= high)) {
          // the near groups' experts that may be among the two largest
          const uint32_t near = __ballot_sync(
              kAll, (inside && gv - spread <= high) || (outside && gv + spread >= low));
          const float edge = __shfl_sync(kAll, group_edge(g2, a.group_score, err), from_lane);
          uint32_t take = 0;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const int gi = (int)((uint32_t)(lane * V + i) * inv_n >> 21) & 31;
            const float from = __shfl_sync(kAll, edge, gi);
            if (i < present && (near >> gi & 1u) && c[i] >= from) take |= 1u << i;
          }
          int C = 0;
          for (uint32_t more = take;;) {
            const uint32_t b = __ballot_sync(kAll, more != 0u);
            if (b == 0u) break;
            const int at = C + __popc(b & ((1u << lane) - 1u));
            if (more != 0u && at < 32) ws.e[at] = lane * V + __ffs(more) - 1;
            more &= more - 1;
            C += __popc(b);
          }
          __syncwarp();
          const int e = lane < C ? ws.e[lane] : 0;
          __syncwarp();
          settled = C <= 32 && low > -kInf;
          if (settled) {
            const uint32_t sure = __ballot_sync(kAll, inside) & ~near;
            open = groups64(row, by_x ? nullptr : a.bias, a.func, m, E, n, a.g, a.group_score,
                            sure, near, C, e, lane, ws.v64, ws.e);
          }
        }
      }
    }

    // ---- candidates: from here on c is what the experts are compared by, NaN where no
    // expert can be selected
    if (MODE != kByX && by_x) {
      load_x();
      l2 = Top2{c[0], -kInf};
#pragma unroll
      for (int i = 1; i < V; ++i) merge(l2, c[i]);
    }
    bool in = present > 0;  // this lane has any
    if (grouped && runs) {
      in = in && ((open >> my_group) & 1u);
    } else if (grouped) {
      in = false;
      l2 = Top2{-kInf, -kInf};
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const bool yes =
            i < present && (open >> ((uint32_t)(lane * V + i) * inv_n >> 21)) & 1u;
        if (yes) merge(l2, c[i]);
        c[i] = yes ? c[i] : none;
        in = in || yes;
      }
    } else if (!VEC) {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = i < present ? c[i] : none;
    }
    // the k-th largest distinct value among the lanes' two largest: k experts reach it
    uint32_t head = in ? score_key(l2.a) : 0u, next = in && l2.b > -kInf ? score_key(l2.b) : 0u;
    uint32_t theta = 0;
#pragma unroll
    for (int r = 0; r < (KFIX > 0 ? KFIX : 1); ++r) {
      theta = __reduce_max_sync(kAll, head);
      if (head == theta) head = next, next = 0u;
    }
    if constexpr (KFIX == 0) {
      for (int r = 1; r < k; ++r) {
        theta = __reduce_max_sync(kAll, head);
        if (head == theta) head = next, next = 0u;
      }
    }
    // less what the errors of two values may hide
    float from = theta ? key_score(theta) : -kInf;
    if (!by_x && from > -kInf) from -= 2.0f * err + 0x1p-22f * fabsf(from);
    if (!in) from = none;
    uint32_t cmask = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) cmask |= c[i] >= from ? 1u << i : 0u;
    // the candidates' experts, one after the other
    int C = 0;
    for (uint32_t left = cmask;;) {
      const uint32_t b = __ballot_sync(kAll, left != 0u);
      if (b == 0u) break;
      const int at = C + __popc(b & ((1u << lane) - 1u));
      if (left != 0u && at < 32) ws.e[at] = lane * V + __ffs(left) - 1;
      left &= left - 1;
      C += __popc(b);
    }
    __syncwarp();
    int sel = 0;
    float xs = -kInf, v = -kInf;  // the candidate's x and what it is compared by
    if (lane < C) {
      sel = ws.e[lane];
      xs = v = __ldg(row + sel);
      if (!by_x)
        v = choice32(MODE == kSigmoid ? MOE_SCORE_SIGMOID : MOE_SCORE_SOFTMAX, xs,
                     __ldg(a.bias + sel), m, z_inv);
    }
    ws.c[lane] = v;
    ws.by_rank[lane] = none;
    __syncwarp();
    int rank = 0;
    const int held = C <= 32 ? C : 0;  // candidates one per lane
    for (int j = 0; j < held; j += 4) {
      const float4 o = *reinterpret_cast<const float4*>(ws.c + j);
      rank += (o.x > v ? 1 : 0) + (o.y > v ? 1 : 0) + (o.z > v ? 1 : 0) + (o.w > v ? 1 : 0);
    }
    if (lane < held) ws.by_rank[rank] = v;
    __syncwarp();
    // an empty rank follows equal values; and neighbours that are too close
    bool bad = false;
    if (lane < k && lane + 1 < held) {
      const float p = ws.by_rank[lane], q = ws.by_rank[lane + 1];
      bad = q != q || (!by_x && q > -kInf &&
                       p - q <= 2.0f * err + 0x1p-22f * fmaxf(fabsf(p), fabsf(q)));
    }
    if (C > 32) {
      // many equal values, or k near the number of lanes: round by round, and one more
      // for the border
      float last = 0.0f;
      for (int r = 0; r <= k; ++r) {
        float best = -kInf;
        int at = V;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (c[i] >= from && (at == V || c[i] > best)) best = c[i], at = i;
        const uint32_t key = at < V ? score_key(best) : 0u;
        const uint32_t win = __reduce_max_sync(kAll, key);
        if (win == 0u) break;
        const float top = key_score(win);
        if (r > 0 && !by_x && top > -kInf &&
            last - top <= 2.0f * err + 0x1p-22f * fmaxf(fabsf(last), fabsf(top)))
          settled = false;
        last = top;
        const int e = (int)__reduce_min_sync(kAll, key == win ? (uint32_t)(lane * V + at) : ~0u);
        if (lane == r) sel = e, xs = __ldg(row + e);
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (lane * V + i == e) c[i] = none;
      }
      rank = lane;
    } else if (__any_sync(kAll, bad) && settled) {
      rank = rank64(row, a.bias, a.func, m, E, by_x, sel, C, lane);
    }
    if (!settled) {
      careful |= 1u << turn;
      continue;
    }

    // ---- weights
    const bool have = lane < C && rank < k;  // C > 32: lane r has the r-th
    float w = weight_score(a.func, a.renorm, xs, have, m, z_inv);
    if (a.renorm) {
      // the largest score's factor is in [1/2, 1]
      const float sum = warp_sum(w);
      w = sum > 0.0f ? w * rcp_f32(sum) : 0.0f;
    }
    if (have) {
      a.idx[t * k + rank] = sel;
      a.w[t * k + rank] = w * a.scale;
    }
  }
  for (; careful; careful &= careful - 1)
    careful_token(a, t0 + (int64_t)(__ffs(careful) - 1) * warps, lane, ws, list);
}

// ------------------------------------------- forward, several tokens per warp

template <int L, class F>
__device__ __forceinline__ float lanes_reduce(float v, F f) {
#pragma unroll
  for (int o = 1; o < L; o <<= 1) v = f(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// One token's candidates, and its winners in their order.
struct TokenScratch {
  float v[32];        // what they are compared by
  uint32_t at[32];    // expert | place in the warp's rows << 16
  float by_rank[20];  // the values of the first L + 1
  float x[16];
  int e[16];
};

// E = L V experts by L lanes per token, 32 / L tokens per warp, each lane V consecutive
// experts and S candidates; groups are runs of whole lanes (L % G == 0); k <= L; a bias, or
// groups by the sum of two.  What a token takes beyond its scores, the groups' ranks, the
// bound of the k-th value, the candidates' ranks and the weights, serves all tokens of the
// warp.  Rows come by coalesced asynchronous
// copies into shared memory, each lane's run padded so that reading 16 bytes per lane
// meets no bank twice, and the next rows are asked for once the candidates' x is taken.
//
// 65536 tokens, 8 of 256 experts, sigmoid and bias: 8 groups 30 us (router_gate_kernel:
// 50), one group 26 (42); 322 instructions per token against 640, 60 % of the issue slots:
// 18 us of issue, and latency that 16 warps per SM do not cover.  80 registers and 24 warps
// were slower (34: spills).  Below about 12 tokens per SM a token per warp is as fast or
// faster (1024 tokens 4.3 against 5.1 us, 4096 9.9 against 8.2).  Nearly equal borders, one token in a thousand, are decided in
// f64 by the whole warp where they are met.
template <int L, int V, int MODE>
__global__ void __launch_bounds__(kLaneWarps * 32, kLaneBlocks)
    router_gate_lanes_kernel(const RouterArgs a) {
  constexpr int Q = 32 / L, E = L * V, S = (E < 32 ? E : 32) / L, kStride = (V / 4) % 2 ? V : V + 4;
  struct Warp {
    float x[32 * kStride];
    TokenScratch q[Q];
  };
  __shared__ __align__(16) float s_bias[L * kStride];
  __shared__ __align__(16) Warp s_warp[kLaneWarps];
  static_assert(sizeof(s_warp[0].x) >= E * 8 && sizeof(s_warp[0].q) >= sizeof(WarpScratch),
                "careful_token's scratch");
  pdl_enter();
  const int lane = threadIdx.x & 31, q = lane / L, j = lane % L;
  Warp& ws = s_warp[threadIdx.x >> 5];
  TokenScratch& tok = ws.q[q];
  const int k = a.k, width = L / a.G;
  const bool grouped = a.g < a.G;
  const int warps = (int)((gridDim.x * blockDim.x) >> 5);
  const int64_t b0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int64_t batches = (a.T + Q - 1) / Q;
  const uint32_t x_to = (uint32_t)__cvta_generic_to_shared(ws.x);
  auto ask = [&](int64_t b) {  // the rows of a batch; past the last token the last row again
    if (b < batches) {
#pragma unroll
      for (int i = 0; i < Q * E / 128; ++i) {
        const int c = i * 32 + lane, row = c / (E / 4), at = c % (E / 4);
        const int64_t t = b * Q + row < a.T ? b * Q + row : a.T - 1;
        cp_async16(x_to + (uint32_t)((row * L + at / (V / 4)) * kStride + at % (V / 4) * 4) * 4,
                   a.scores + t * E + at * 4);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  ask(b0);
  for (int e = threadIdx.x; e < E; e += blockDim.x)
    s_bias[e / V * kStride + e % V] = a.bias ? __ldg(a.bias + e) : 0.0f;
  __syncthreads();
  uint32_t careful = 0;  // tokens to be done again

  int64_t b = b0;
  for (int turn = 0; b < batches; b += warps, ++turn) {
    const int64_t t = b * Q + q;
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
    // ---- c
    const float4* my_x = reinterpret_cast<const float4*>(ws.x + lane * kStride);
    const float4* my_b = reinterpret_cast<const float4*>(s_bias + j * kStride);
    float c[V];
    float m = 0.0f, z_inv = 0.0f, err, x_min = kInf;
#pragma unroll
    for (int h = 0; h < V / 4; ++h) {
      const float4 f = my_x[h];
      c[4 * h] = f.x, c[4 * h + 1] = f.y, c[4 * h + 2] = f.z, c[4 * h + 3] = f.w;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) x_min = fminf(x_min, c[i]);
    if constexpr (MODE == kSoftmax) {
      m = c[0];
#pragma unroll
      for (int i = 1; i < V; ++i) m = fmaxf(m, c[i]);
      m = lanes_reduce<L>(m, [](float u, float w) { return fmaxf(u, w); });
      if (m == -kInf) m = 0.0f;
      float z = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        c[i] = exp2_est((c[i] - m) * kLog2e);
        z += c[i];
      }
      z = lanes_reduce<L>(z, [](float u, float w) { return u + w; });
      z_inv = z > 0.0f ? rcp_f32(z) : 0.0f;
      err = score_err(MOE_SCORE_SOFTMAX, z_inv);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = rcp_est(1.0f + exp2_est(c[i] * -kLog2e));
      err = score_err(MOE_SCORE_SIGMOID, 1.0f);
    }
#pragma unroll
    for (int h = 0; h < V / 4; ++h) {
      const float4 f = my_b[h];
      const float bias[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c[4 * h + i] = MODE == kSoftmax ? __fmaf_rn(c[4 * h + i], z_inv, bias[i])
                                        : c[4 * h + i] + bias[i];
    }
    if (__any_sync(kAll, x_min == -kInf)) {
#pragma unroll
      for (int h = 0; h < V / 4; ++h) {
        const float4 f = my_x[h];
        c[4 * h] = f.x == -kInf ? -kInf : c[4 * h];
        c[4 * h + 1] = f.y == -kInf ? -kInf : c[4 * h + 1];
        c[4 * h + 2] = f.z == -kInf ? -kInf : c[4 * h + 2];
        c[4 * h + 3] = f.w == -kInf ? -kInf : c[4 * h + 3];
      }
    }
    // ---- the lane's two largest, and the groups
    Top2 l2 = {fmaxf(c[0], c[1]), fminf(c[0], c[1])};
#pragma unroll
    for (int i = 2; i < V; i += 2) {
      const float hi = fmaxf(c[i], c[i + 1]), lo = fminf(c[i], c[i + 1]);
      l2.b = fmaxf(fmaxf(l2.b, lo), fminf(l2.a, hi));
      l2.a = fmaxf(l2.a, hi);
    }
    bool in = true;
    if (grouped) {
      Top2 g2 = l2;
      for (int o = 1; o < width; o <<= 1)
        merge(g2, Top2{__shfl_xor_sync(kAll, g2.a, o), __shfl_xor_sync(kAll, g2.b, o)});
      const float gv = group_value(g2, a.group_score);
      int rank = 0;
      for (int o = width; o < L; o += width) {
        const float other = __shfl_xor_sync(kAll, gv, o);
        rank += other > gv || (other == gv && (lane ^ o) < lane) ? 1 : 0;
      }
      in = rank < a.g;
      // the least that a group inside may be against the most that one outside may be
      const float spread = group_err(g2, a.group_score, err);
      const float low = lanes_reduce<L>(in ? gv - spread : kInf,
                                        [](float u, float w) { return fminf(u, w); });
      const float high = lanes_reduce<L>(in ? -kInf : gv + spread,
                                         [](float u, float w) { return fmaxf(u, w); });
      uint32_t near = __ballot_sync(kAll, high > -kInf && low <= high);
      while (near) {  // rare
        const int w = (__ffs(near) - 1) / L;
        near &= ~((kAll >> (32 - L)) << (w * L));
        const int64_t tw = b * Q + w < a.T ? b * Q + w : a.T - 1;
        const float* row = a.scores + tw * E;
        const float mw = __shfl_sync(kAll, m, w * L);
        // the near groups' experts that may be among the two largest
        const bool close = q == w && (in ? gv - spread <= high : gv + spread >= low);
        const float edge = group_edge(g2, a.group_score, err);
        uint32_t take = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) take |= close && c[i] >= edge ? 1u << i : 0u;
        int n = 0;
        for (;;) {
          const uint32_t some = __ballot_sync(kAll, take != 0u);
          if (some == 0u) break;
          const int at = n + __popc(some & ((1u << lane) - 1u));
          if (take != 0u && at < 32) ws.q[w].at[at] = (uint32_t)(j * V + __ffs(take) - 1);
          take &= take - 1;
          n += __popc(some);
        }
        uint32_t maybe = 0, sure = 0;  // a bit per group
        for (int i = 0; i < a.G; ++i) {
          const int of = w * L + i * width;
          maybe |= __shfl_sync(kAll, close ? 1u : 0u, of) << i;
          sure |= __shfl_sync(kAll, in && !close ? 1u : 0u, of) << i;
        }
        __syncwarp();
        const int e = lane < n ? (int)ws.q[w].at[lane] : 0;
        __syncwarp();
        uint32_t open = 0;
        bool known = true;
        if (n <= 32)
          open = groups64(row, a.bias, a.func, mw, E, E / a.G, a.g, a.group_score, sure, maybe, n,
                          e, lane, reinterpret_cast<double*>(ws.q[w].v),
                          reinterpret_cast<int*>(ws.q[w].by_rank));
        else if (!one_value(row, a.bias, E, lane))  // else these ties are exact
          open = all_groups64(row, a.bias, a.func, mw, E, a.G, a.g, a.group_score, lane);
        else
          known = false;
        if (q == w && known) in = (open >> (j / width)) & 1u;
        __syncwarp();
      }
    }
    // ---- candidates: the k-th largest among the lanes' two largest is reached by k experts
    if (!in) l2 = Top2{-kInf, -kInf};
    int rank_a = 0, rank_b = 1;
#pragma unroll
    for (int o = 1; o < L; ++o) {
      const float oa = __shfl_xor_sync(kAll, l2.a, o), ob = __shfl_xor_sync(kAll, l2.b, o);
      rank_a += (oa > l2.a ? 1 : 0) + (ob > l2.a ? 1 : 0);
      rank_b += (oa > l2.b ? 1 : 0) + (ob > l2.b ? 1 : 0);
    }
    auto larger = [](float u, float w) { return fmaxf(u, w); };
    float theta = lanes_reduce<L>(rank_b < k ? l2.b : rank_a < k ? l2.a : kInf,
                                  [](float u, float w) { return fminf(u, w); });
    // fewer than k finite values: settled with care
    const bool lost = !(theta > -kInf && theta < kInf);
    uint32_t mine;
    int upto, C;
    float from;
    auto collect = [&]() {
      // less what the errors of two values may hide
      from = theta - (2.0f * err + 0x1p-22f * fabsf(theta));
      if (!in || lost) from = __int_as_float(0x7FFFFFFF);
      mine = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) mine |= c[i] >= from ? 1u << i : 0u;
      upto = __popc(mine);
#pragma unroll
      for (int o = 1; o < L; o <<= 1) {
        const int v = __shfl_up_sync(kAll, upto, o, L);
        if (j >= o) upto += v;
      }
      C = __shfl_sync(kAll, upto, L - 1, L);
    };
    collect();
    // one token in a hundred has more than the scratch holds: the bound by bisection
    bool again = false;
    if (__any_sync(kAll, C > 32)) {
      float lo = theta, hi = lanes_reduce<L>(l2.a, larger);
      for (int i = 0; i < 12 && __any_sync(kAll, C > 32 || C < k); ++i) {
        if (C > 32) lo = theta;
        if (C < k) hi = theta;
        if (C > 32 || C < k) theta = 0.5f * (lo + hi);
        collect();
      }
      int reach = 0;  // the bound itself: k experts reach it, not the margin alone
#pragma unroll
      for (int i = 0; i < V; ++i) reach += in && c[i] >= theta ? 1 : 0;
#pragma unroll
      for (int o = 1; o < L; o <<= 1) reach += __shfl_xor_sync(kAll, reach, o);
      again = reach < k;
    }
    again = again || C > 32 || C < k;
    if (again) C = 0, mine = 0u;
    int put = upto - __popc(mine);
    while (mine) {
      const int i = __ffs(mine) - 1;
      mine &= mine - 1;
      tok.at[put++] = (uint32_t)(j * V + i) | (uint32_t)(lane * kStride + i) << 16;
    }
    for (int r = j; r <= k; r += L) tok.by_rank[r] = __int_as_float(0x7FFFFFFF);
    const int most = (int)__reduce_max_sync(kAll, (uint32_t)C);
    __syncwarp();
    float xs[S], v[S];
    int e[S], rank[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
      xs[s] = v[s] = -kInf;
      e[s] = 0, rank[s] = 32;
      if (s * L < most) {
        const int r = s * L + j;
        if (r < C) {
          const uint32_t at = tok.at[r];
          e[s] = (int)(at & 0xFFFFu);
          xs[s] = ws.x[at >> 16];
          v[s] = choice32(MODE == kSigmoid ? MOE_SCORE_SIGMOID : MOE_SCORE_SOFTMAX, xs[s],
                          s_bias[(int)(at >> 16) - q * L * kStride], m, z_inv);
        }
        tok.v[r] = v[s];
      }
    }
    __syncwarp();
    ask(b + warps);
    auto ranks = [&](auto count) {
#pragma unroll
      for (int s = 0; s < count.value; ++s) rank[s] = 0;
      for (int o = 0; o < most; o += 4) {
        const float4 u = *reinterpret_cast<const float4*>(tok.v + o);
#pragma unroll
        for (int s = 0; s < count.value; ++s)
          rank[s] += (u.x > v[s] ? 1 : 0) + (u.y > v[s] ? 1 : 0) + (u.z > v[s] ? 1 : 0) +
                     (u.w > v[s] ? 1 : 0);
      }
    };
    if (S == 2 || most <= 2 * L)
      ranks(std::integral_constant<int, 2>());
    else if (most <= 3 * L)
      ranks(std::integral_constant<int, S < 3 ? S : 3>());
    else
      ranks(std::integral_constant<int, S>());
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if (s * L + j >= C) rank[s] = 32;
      if (rank[s] <= k) tok.by_rank[rank[s]] = v[s];
      if (rank[s] < k) tok.e[rank[s]] = e[s], tok.x[rank[s]] = xs[s];
    }
    __syncwarp();
    // an empty rank follows equal values; and neighbours that are too close
    bool bad = false;
    if (j < k && j + 1 < C) {
      const float p = tok.by_rank[j], n = tok.by_rank[j + 1];
      bad = n != n || (n > -kInf && p - n <= 2.0f * err + 0x1p-22f * fmaxf(fabsf(p), fabsf(n)));
    }
    uint32_t near = __ballot_sync(kAll, bad);
    while (near) {  // one token in a thousand
      const int w = (__ffs(near) - 1) / L;
      near &= ~((kAll >> (32 - L)) << (w * L));
      const int64_t tw = b * Q + w < a.T ? b * Q + w : a.T - 1;
      const int Cw = __shfl_sync(kAll, C, w * L);
      const float* row = a.scores + tw * E;
      const int ew = lane < Cw ? (int)(ws.q[w].at[lane] & 0xFFFFu) : 0;
      const int rw = rank64(row, a.bias, a.func, __shfl_sync(kAll, m, w * L), E,
                            a.bias == nullptr, ew, Cw, lane);
      if (lane < Cw && rw < k) ws.q[w].e[rw] = ew, ws.q[w].x[rw] = __ldg(row + ew);
      __syncwarp();
    }
    // ---- weights, the r-th winner's by lane r
    const bool have = j < k && !again;
    const float x = have ? tok.x[j] : -kInf;
    float w = 0.0f;
    if (MODE == kSoftmax) {
      const float top = a.renorm ? lanes_reduce<L>(x, larger) : m;
      if (x > -kInf) w = expf(x - top) * (a.renorm ? 1.0f : z_inv);
    } else {
      const float lo = fminf(x, 0.0f);
      const float top = a.renorm ? lanes_reduce<L>(lo, larger) : 0.0f;
      if (x > -kInf) w = expf(lo - top) * rcp_f32(1.0f + expf(-fabsf(x)));
    }
    if (a.renorm) {
      const float sum = lanes_reduce<L>(w, [](float u, float y) { return u + y; });
      w = sum > 0.0f ? w * rcp_f32(sum) : 0.0f;
    }
    if (have && t < a.T) {
      a.idx[t * k + j] = tok.e[j];
      a.w[t * k + j] = w * a.scale;
    }
    const uint32_t redo = __ballot_sync(kAll, again && j == 0 && t < a.T);
#pragma unroll
    for (int w2 = 0; w2 < Q; ++w2) careful |= (redo >> (w2 * L) & 1u) << (turn * Q + w2);
    __syncwarp();
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncwarp();
  for (; careful; careful &= careful - 1) {
    const int at = __ffs(careful) - 1;
    careful_token(a, (b0 + (int64_t)(at / Q) * warps) * Q + at % Q, lane,
                  *reinterpret_cast<WarpScratch*>(ws.q),
                  reinterpret_cast<unsigned long long*>(ws.x));
  }
}

template <int L, int V, int MODE>
cudaError_t launch_lanes(const LaunchCtx& c, const RouterArgs& a) {
  constexpr int Q = 32 / L;
  // at most 32 tokens per warp
  const int64_t need = ((a.T + Q - 1) / Q + kLaneWarps - 1) / kLaneWarps;
  int64_t blocks = (int64_t)c.num_sms * kLaneBlocks;
  if (blocks > need) blocks = need;
  if (blocks < (need + L - 1) / L) blocks = (need + L - 1) / L;
  return launch_pdl(router_gate_lanes_kernel<L, V, MODE>, dim3((unsigned)blocks), kLaneWarps * 32,
                    0, c.stream, a);
}
template <int L, int V>
cudaError_t launch_lanes(const LaunchCtx& c, const RouterArgs& a) {
  return a.func == MOE_SCORE_SIGMOID ? launch_lanes<L, V, kSigmoid>(c, a)
                                     : launch_lanes<L, V, kSoftmax>(c, a);
}

template <int V, bool VEC, int KFIX, int MODE>
cudaError_t launch_m(const LaunchCtx& c, const RouterArgs& a) {
  auto* kernel = router_gate_kernel<V, VEC, KFIX, MODE>;
  const size_t smem = (size_t)kWarps * a.E * 8;
  if (smem > 40 * 1024) {
    static SmemOptIn opt_in;
    const cudaError_t e = opt_in.once(kernel);
    if (e != cudaSuccess) return e;
  }
  // two rounds of blocks, and at most 32 tokens per warp
  const int64_t need = (a.T + kWarps - 1) / kWarps;
  int64_t blocks = (int64_t)c.num_sms * 8;
  if (blocks > need) blocks = need;
  if (blocks < (need + 31) / 32) blocks = (need + 31) / 32;
  return launch_pdl(kernel, dim3((unsigned)blocks), kWarps * 32, smem, c.stream, a);
}
template <int V, bool VEC, int KFIX>
cudaError_t launch_k(const LaunchCtx& c, const RouterArgs& a) {
  if (!a.bias && (a.g == a.G || a.group_score == MOE_GROUP_MAX))
    return launch_m<V, VEC, KFIX, kByX>(c, a);
  return a.func == MOE_SCORE_SIGMOID ? launch_m<V, VEC, KFIX, kSigmoid>(c, a)
                                     : launch_m<V, VEC, KFIX, kSoftmax>(c, a);
}
template <int V, bool VEC>
cudaError_t launch_v(const LaunchCtx& c, const RouterArgs& a) {
  if constexpr (V == 8) {
    if (a.k == 8) return launch_k<V, VEC, 8>(c, a);
  }
  return launch_k<V, VEC, 0>(c, a);
}

// ------------------------------------------------------------------ backward

// L >= k lanes per token, 32 / L tokens per warp: what a token takes beyond its row (the
// scores, weights and sums of the selected experts) serves all of them.  A row is copied
// (or zeroed) by the whole warp; the selected entries are then written over by their
// lanes, from add's values read before.  DENSE, the softmax without renormalisation: every
// entry changes; one token per warp.  U > 0: rows of whole, 16-byte aligned fours, at
// most 128 U; they are asked for before the selected experts are known.
//
// 65536 tokens, E = 256, k = 8, added onto another gradient: 27.6 us for 155 MB, counting
// whole sectors of the gathered scores (without add 15.2 us).  One token per warp: 31 us
// (24.6) at 290 instructions per token.
template <int U, int L, bool DENSE>
__global__ void __launch_bounds__(kWarps * 32)
    router_gate_backward_kernel(const RouterArgs a, unsigned* err) {
  constexpr int TOK = DENSE ? 1 : 32 / L;
  static_assert(!DENSE || L == 32, "a whole warp per row");
  pdl_enter();
  const int lane = threadIdx.x & 31, q = lane / L, j = lane % L;
  const int64_t t0 = (((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5) * TOK;
  if (t0 >= a.T) return;
  const int E = a.E, k = a.k;
  const int64_t t = t0 + q;
  const bool slot = t < a.T && j < k;
  const bool copy = DENSE || a.add != a.grad_scores;
  int e = slot ? a.idx[t * k + j] : -1;
  float g = slot ? a.grad_w[t * k + j] : 0.0f;
  float4 v[TOK][U > 0 ? U : 1], y[DENSE && U > 0 ? U : 1];
  if constexpr (U > 0) {
#pragma unroll
    for (int p = 0; p < TOK; ++p)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = u * 128 + lane * 4;
        v[p][u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (a.add && copy && c < E && t0 + p < a.T)
          v[p][u] = *reinterpret_cast<const float4*>(a.add + (t0 + p) * E + c);
      }
    if constexpr (DENSE) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = u * 128 + lane * 4;
        y[u] = make_float4(-kInf, -kInf, -kInf, -kInf);
        if (c < E) y[u] = __ldg(reinterpret_cast<const float4*>(a.scores + t0 * E + c));
      }
    }
  }
  if (slot && (e < 0 || e >= E)) {
    flag_error(err, MOE_DEVERR_EXPERT_RANGE);
    e = -1;
  }
  const bool have = e >= 0;
  const float x = have ? a.scores[t * E + e] : -kInf;
  const float before = have && a.add ? a.add[t * E + e] : 0.0f;
  if (!have) g = 0.0f;
  // an expert that its token names n times: one entry, for the sum of its gradients
  const unsigned same = __match_any_sync(kAll, have ? q * E + e : -1 - lane);
  float g_e = g;
  if (__any_sync(kAll, (same & (same - 1)) != 0)) {
    g_e = 0.0f;
    for (int l = 0; l < 32; ++l) {
      const float o = __shfl_sync(kAll, g, l);
      if (same >> l & 1) g_e += o;
    }
  }
  const float n = DENSE ? 1.0f : (float)__popc(same);
  float m = 0.0f, z_inv = 0.0f;
  if constexpr (DENSE) {
    const float* row = a.scores + t0 * E;
    float z = 0.0f;
    m = -kInf;
    if constexpr (U > 0) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        m = fmaxf(m, fmaxf(fmaxf(y[u].x, y[u].y), fmaxf(y[u].z, y[u].w)));
      m = warp_max(m);
      if (m == -kInf) m = 0.0f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        y[u].x = expf(y[u].x - m), y[u].y = expf(y[u].y - m);
        y[u].z = expf(y[u].z - m), y[u].w = expf(y[u].w - m);
        z += (y[u].x + y[u].y) + (y[u].z + y[u].w);
      }
    } else {
      for (int c = lane; c < E; c += 32) m = fmaxf(m, row[c]);
      m = warp_max(m);
      if (m == -kInf) m = 0.0f;
      for (int c = lane; c < E; c += 32) z += expf(row[c] - m);
    }
    z = warp_sum(z);
    z_inv = z > 0.0f ? __fdiv_rn(1.0f, z) : 0.0f;
  }
  // the selected scores as in weight_score, by their token's lanes
  auto larger = [](float u, float w) { return fmaxf(u, w); };
  auto plus = [](float u, float w) { return u + w; };
  float w = 0.0f;
  if (a.func == MOE_SCORE_SOFTMAX) {
    const float top = DENSE ? m : lanes_reduce<L>(x, larger);
    if (have && x > -kInf) w = expf(x - top) * (DENSE ? z_inv : 1.0f);
  } else {
    const float lo = fminf(x, 0.0f);
    const float top = a.renorm ? lanes_reduce<L>(lo, larger) : 0.0f;
    if (have && x > -kInf) w = expf(lo - top) * rcp_f32(1.0f + expf(-fabsf(x)));
  }
  if (a.renorm) {
    const float sum = lanes_reduce<L>(w, plus);
    w = sum > 0.0f ? w * rcp_f32(sum) : 0.0f;
  }
  const float dot = lanes_reduce<L>(g * w, plus);  // sum g_j w_j / scale, or sum g_j s_j
  float d = a.scale * w * (a.renorm || DENSE ? g_e - n * dot : g_e);
  if (a.func == MOE_SCORE_SIGMOID) d *= sigmoid_f32(-x);
  const float f = DENSE ? -a.scale * dot * z_inv : 0.0f;
  if (copy) {
#pragma unroll
    for (int p = 0; p < TOK; ++p) {
      if (t0 + p >= a.T) break;
      float* out = a.grad_scores + (t0 + p) * E;
      if constexpr (U > 0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int c = u * 128 + lane * 4;
          float4& r = v[p][u];
          if constexpr (DENSE) {
            r.x = __fmaf_rn(y[u].x, f, r.x), r.y = __fmaf_rn(y[u].y, f, r.y);
            r.z = __fmaf_rn(y[u].z, f, r.z), r.w = __fmaf_rn(y[u].w, f, r.w);
          }
          if (c < E)
            st_stream_v4(out + c, make_uint4(__float_as_uint(r.x), __float_as_uint(r.y),
                                             __float_as_uint(r.z), __float_as_uint(r.w)));
        }
      } else {
        const float* add = a.add ? a.add + (t0 + p) * E : nullptr;
        const float* row = a.scores + (t0 + p) * E;
        for (int c = lane; c < E; c += 32)
          out[c] = (add ? add[c] : 0.0f) + (DENSE ? expf(row[c] - m) * f : 0.0f);
      }
    }
  }
  __syncwarp();
  if (have) a.grad_scores[t * E + e] = before + d;
}

template <int U, int L, bool DENSE>
cudaError_t launch_backward(const LaunchCtx& c, const RouterArgs& a) {
  const int64_t per_block = kWarps * (DENSE ? 1 : 32 / L);
  return launch_pdl(router_gate_backward_kernel<U, L, DENSE>,
                    dim3((unsigned)((a.T + per_block - 1) / per_block)), kWarps * 32, 0, c.stream, a,
                    c.err);
}
template <int U>
cudaError_t launch_backward_u(const LaunchCtx& c, const RouterArgs& a) {
  if (a.func == MOE_SCORE_SOFTMAX && !a.renorm) return launch_backward<U, 32, true>(c, a);
  if (a.k <= 8 && U <= 2) return launch_backward<U, 8, false>(c, a);
  if (a.k <= 16 && U <= 4) return launch_backward<U, 16, false>(c, a);
  return launch_backward<U, 32, false>(c, a);
}

}  // namespace

cudaError_t launch_router_gate(const LaunchCtx& c, const RouterArgs& a) {
  const bool al = reinterpret_cast<uintptr_t>(a.scores) % 16 == 0;
  // compared by c, and tokens enough: several per warp, where groups are whole lanes and
  // the lanes' two largest of the open groups are at least k values
  if (al && (a.bias || (a.g < a.G && a.group_score == MOE_GROUP_TOP2)) &&
      a.T > kLanesFrom * (int64_t)c.num_sms) {
    if (a.E == 16 && a.k <= 4 && 4 % a.G == 0 && a.k * a.G <= 8 * a.g)
      return launch_lanes<4, 4>(c, a);
    if (a.k <= 8 && 8 % a.G == 0 && a.k * a.G <= 16 * a.g) {
      if (a.E == 32) return launch_lanes<8, 4>(c, a);
      if (a.E == 64) return launch_lanes<8, 8>(c, a);
      if (a.E == 128) return launch_lanes<8, 16>(c, a);
      if (a.E == 160) return launch_lanes<8, 20>(c, a);
      if (a.E == 192) return launch_lanes<8, 24>(c, a);
      if (a.E == 256) return launch_lanes<8, 32>(c, a);
    }
    if (a.k <= 16 && 16 % a.G == 0 && a.k * a.G <= 32 * a.g) {
      if (a.E == 384) return launch_lanes<16, 24>(c, a);
      if (a.E == 512) return launch_lanes<16, 32>(c, a);
    }
  }
  // the fewest experts per lane; a few widths more than powers of two, as groups are then
  // more often whole lanes
  if (a.E <= 32) return launch_v<1, false>(c, a);
  if (a.E <= 64) return launch_v<2, false>(c, a);
  if (a.E <= 96) return launch_v<3, false>(c, a);
  if (a.E <= 128) return launch_v<4, false>(c, a);
  if (a.E <= 160) return launch_v<5, false>(c, a);
  if (a.E <= 192) return launch_v<6, false>(c, a);
  if (a.E <= 256) return a.E == 256 && al ? launch_v<8, true>(c, a) : launch_v<8, false>(c, a);
  if (a.E <= 384) return launch_v<12, false>(c, a);
  if (a.E <= 512) return launch_v<16, false>(c, a);
  return launch_v<32, false>(c, a);
}

cudaError_t launch_router_gate_backward(const LaunchCtx& c, const RouterArgs& a) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.add) |
                       reinterpret_cast<uintptr_t>(a.grad_scores) |
                       reinterpret_cast<uintptr_t>(a.scores);
  if (a.E % 4 != 0 || at % 16 != 0) return launch_backward_u<0>(c, a);
  if (a.E <= 128) return launch_backward_u<1>(c, a);
  if (a.E <= 256) return launch_backward_u<2>(c, a);
  if (a.E <= 512) return launch_backward_u<4>(c, a);
  return launch_backward_u<8>(c, a);
}

}  // namespace moe
