// router_gate.cu -- the router with a bias for balance and groups of experts, and
// the gradient of its weights.
//
//   s = softmax(x) or sigmoid(x);  c = s + bias, -inf where x is -inf
//   the g groups with the largest max, or sum of the two largest, of c; among their
//   experts the k with the largest c; ties to the lower group and expert
//   w_j = scale s_j / sum s, or scale s_j
//
// The selection is that of the real numbers.  Without a bias c orders the experts as
// x does, and they are compared by x, exactly.  Otherwise c is taken in f32, whose
// error is bounded (kErr below); where two values at a border of the selection lie
// closer than that and are not the same (x, bias), the token is decided again in f64,
// one value per candidate, which f32's spacing makes rare: about one token in a
// thousand for 8 of 256 experts.
//
// One warp per token, lane l holding the V consecutive experts l V .. l V + V - 1, so
// that a group is a run of lanes.  The selection is topk_warp.cuh's: a lower bound of
// the k-th value from the lanes' maxima leaves a few candidates, one per lane, ranked
// against one another.
#include "block/block_ops.cuh"
#include "topk_warp.cuh"

namespace moe {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kWarps = 8;
constexpr float kInf = __builtin_huge_valf();

// |f32 c - c| <= kErr[func] * (largest s of the row) + 2^-23 |c|.
// Sigmoid: expf, the reciprocal and two products, each within 2 ulp of s <= 1.
// Softmax: x - max is off by up to 2^-24 |x - max|, which e^ turns into a relative
// error of that size: below 100 * 2^-24 as far as e^ does not vanish, plus the sum's.
__device__ __forceinline__ float score_err(int func, float top) {
  return func == MOE_SCORE_SIGMOID ? 0x1p-20f : 0x1p-16f * top;
}

// Two values of a group or of two groups: the largest and the second.
struct Top2 {
  float a, b;
};
__device__ __forceinline__ void merge(Top2& t, Top2 o) {
  const float lo = fminf(t.a, o.a);
  t.a = fmaxf(t.a, o.a);
  t.b = fmaxf(lo, fmaxf(t.b, o.b));
}
__device__ __forceinline__ float group_value(const Top2& t, int kind) {
  return kind == MOE_GROUP_TOP2 && t.b > -kInf ? t.a + t.b : t.a;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
__device__ __forceinline__ float warp_min(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fminf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
__device__ __forceinline__ double warp_sum64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

__device__ __forceinline__ double sigmoid64(double x) {
  const double e = exp(-fabs(x));
  return x < 0.0 ? e / (1.0 + e) : 1.0 / (1.0 + e);
}

// One token's scores as every step of the kernel sees them.
struct Token {
  const float* row;
  const float* bias;
  int func;
  float m;         // largest x (softmax)
  double z;        // sum of exp(x - m) in f64, 0 until it is needed
};

// c of expert e in f64.
__device__ __noinline__ double choice64(const Token& t, int e) {
  const float x = t.row[e];
  if (x == -kInf) return -__builtin_huge_val();
  const double s = t.func == MOE_SCORE_SIGMOID ? sigmoid64((double)x)
                                               : exp((double)x - (double)t.m) / t.z;
  return t.bias ? s + (double)t.bias[e] : s;
}
// The softmax's sum in f64.
__device__ __noinline__ double sum64(const Token& t, int E, int lane) {
  double z = 0.0;
  for (int e = lane; e < E; e += 32) z += exp((double)t.row[e] - (double)t.m);
  return warp_sum64(z);
}

// The groups of rank < g, by values one per lane (lane i < G), in f64: a bit per group.
__device__ __noinline__ uint32_t groups64(const Token& t, int E, int G, int g, int kind,
                                          int lane) {
  const int n = E / G;
  double v = 0.0;
  // each group in turn by the whole warp
  for (int i = 0; i < G; ++i) {
    double a = -__builtin_huge_val(), b = a;
    for (int e = lane; e < n; e += 32) {
      const double c = choice64(t, i * n + e);
      if (c > a) {
        b = a, a = c;
      } else if (c > b) {
        b = c;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double oa = __shfl_xor_sync(kAll, a, o), ob = __shfl_xor_sync(kAll, b, o);
      const double lo = fmin(a, oa);
      a = fmax(a, oa);
      b = fmax(lo, fmax(b, ob));
    }
    const double s = kind == MOE_GROUP_TOP2 && b > -__builtin_huge_val() ? a + b : a;
    if (lane == i) v = s;
  }
  int rank = 0;
  for (int i = 0; i < G; ++i) {
    const double o = __shfl_sync(kAll, v, i);
    rank += o > v || (o == v && i < lane) ? 1 : 0;
  }
  return __ballot_sync(kAll, lane < G && rank < g);
}

// The k winners of the open groups one after the other in f64, the r-th in lane r.
__device__ __noinline__ int select64(const Token& t, int E, int G, uint32_t open, int k,
                                     int lane, double* list) {
  // list: this warp's values, [E], retired ones NaN
  const int n = E / G;
  for (int e = lane; e < E; e += 32)
    list[e] = (open >> (e / n)) & 1u ? choice64(t, e) : __longlong_as_double(-1ll);
  __syncwarp();
  int mine = -1;
  for (int r = 0; r < k; ++r) {
    double best = -__builtin_huge_val();
    int at = -1;
    for (int e = lane; e < E; e += 32) {
      const double c = list[e];
      if (c == c && (at < 0 || c > best)) best = c, at = e;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double ob = __shfl_xor_sync(kAll, best, o);
      const int oa = __shfl_xor_sync(kAll, at, o);
      if (oa >= 0 && (at < 0 || ob > best || (ob == best && oa < at))) best = ob, at = oa;
    }
    if (lane == r) mine = at;
    if (lane == 0) list[at] = __longlong_as_double(-1ll);
    __syncwarp();
  }
  return mine;
}

// The scores of the selected experts (one per lane, e < 0: none) for the weights: s
// itself, or with `ratio` s times a factor that all of them share.
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

struct WarpScratch {
  unsigned long long cand[32];
  float x[32];
};

// V experts per lane.  VEC: E = 32 V, V % 4 == 0 and 16-byte aligned rows.
template <int V, bool VEC>
__global__ void __launch_bounds__(kWarps * 32)
    router_gate_kernel(const RouterArgs a) {
  __shared__ WarpScratch s_scratch[kWarps];
  extern __shared__ double s_list[];  // [kWarps][E]
  pdl_enter();
  const int lane = threadIdx.x & 31, wib = threadIdx.x >> 5;
  WarpScratch& ws = s_scratch[wib];
  const int E = VEC ? 32 * V : a.E;
  const int k = a.k, n = E / a.G;
  double* list = s_list + (size_t)wib * E;
  float* s_c = reinterpret_cast<float*>(list);
  const int64_t warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  // lanes per group, where a group is a power of two of whole lanes
  const int run = n % V == 0 ? n / V : 0;
  const bool runs = run > 0 && (run & (run - 1)) == 0;
  int L = 32;  // lanes that share a group otherwise
  while (L > 1 && L * a.G > 32) L >>= 1;
  float bias[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane * V + i;
    bias[i] = a.bias != nullptr && e < E ? __ldg(a.bias + e) : 0.0f;
  }
  const bool by_x = a.bias == nullptr;  // c orders the experts as x does
  const bool need_c = !by_x || (a.G > 1 && a.group_score == MOE_GROUP_TOP2);
  const bool need_z = a.func == MOE_SCORE_SOFTMAX && (need_c || !a.renorm);

  for (int64_t t = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; t < a.T; t += warps) {
    Token tok;
    tok.row = a.scores + t * E;
    tok.bias = a.bias;
    tok.func = a.func;
    tok.m = 0.0f;
    tok.z = 0.0;
    float x[V];
    if constexpr (VEC) {
#pragma unroll
      for (int h = 0; h < V / 4; ++h) {
        const float4 f =
            __ldg(reinterpret_cast<const float4*>(tok.row + lane * V + 4 * h));
        x[4 * h] = f.x, x[4 * h + 1] = f.y, x[4 * h + 2] = f.z, x[4 * h + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = lane * V + i;
        x[i] = e < E ? __ldg(tok.row + e) : -kInf;
      }
    }
    // ---- scores and choices
    float c[V];
    float top = 1.0f, z_inv = 0.0f;
    if (a.func == MOE_SCORE_SOFTMAX && need_z) {
      float m = x[0];
#pragma unroll
      for (int i = 1; i < V; ++i) m = fmaxf(m, x[i]);
      m = warp_max(m);
      if (m == -kInf) m = 0.0f;
      tok.m = m;
      float z = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        c[i] = expf(x[i] - m);
        z += c[i];
      }
      z = warp_sum(z);
      z_inv = z > 0.0f ? __fdiv_rn(1.0f, z) : 0.0f;
      top = z_inv;
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = x[i] > -kInf ? c[i] * z_inv + bias[i] : -kInf;
    } else if (need_c) {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = x[i] > -kInf ? sigmoid_f32(x[i]) + bias[i] : -kInf;
    }
    if (!need_c) {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = x[i];
    }
    const float err = need_c ? score_err(a.func, top) : 0.0f;

    // ---- groups
    uint32_t open = kAll;
    if (a.G > 1 && a.g < a.G) {
      Top2 g2 = {-kInf, -kInf};
      if (runs) {
#pragma unroll
        for (int i = 0; i < V; ++i) merge(g2, Top2{c[i], -kInf});
        for (int o = 1; o < run; o <<= 1)
          merge(g2, Top2{__shfl_xor_sync(kAll, g2.a, o), __shfl_xor_sync(kAll, g2.b, o)});
      } else {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (lane * V + i < E) s_c[lane * V + i] = c[i];
        __syncwarp();
        const int gi = lane / L;
        if (gi < a.G)
          for (int e = lane % L; e < n; e += L) merge(g2, Top2{s_c[gi * n + e], -kInf});
        for (int o = 1; o < L; o <<= 1)
          merge(g2, Top2{__shfl_xor_sync(kAll, g2.a, o), __shfl_xor_sync(kAll, g2.b, o)});
      }
      const float mine = group_value(g2, a.group_score);
      const float gv = __shfl_sync(kAll, mine, (lane * (runs ? run : L)) & 31);
      int rank = 0;
      bool near = false;  // to a group on the other side of the border
      for (int i = 0; i < a.G; ++i) {
        const float o = __shfl_sync(kAll, gv, i);
        rank += o > gv || (o == gv && i < lane) ? 1 : 0;
      }
      const bool in = lane < a.G && rank < a.g;
      open = __ballot_sync(kAll, in);
      if (need_c) {
        // the lowest inside against the highest outside
        const float low = warp_min(in ? gv : kInf);
        const float high = warp_max(lane < a.G && !in ? gv : -kInf);
        near = low - high <= 4.0f * err + 0x1p-21f * fmaxf(fabsf(low), fabsf(high)) &&
               high > -kInf;
      }
      if (near) {
        // unless the whole row is one value: those ties are exact
        float xl = kInf, xh = -kInf, bl = kInf, bh = -kInf;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (lane * V + i >= E) continue;
          xl = fminf(xl, x[i]), xh = fmaxf(xh, x[i]);
          bl = fminf(bl, bias[i]), bh = fmaxf(bh, bias[i]);
        }
        if (warp_min(xl) != warp_max(xh) || warp_min(bl) != warp_max(bh)) {
          if (a.func == MOE_SCORE_SOFTMAX) tok.z = sum64(tok, E, lane);
          open = groups64(tok, E, a.G, a.g, a.group_score, lane);
        }
      }
    }

    // ---- keys: c, or x without a bias; 0 for closed groups and absent slots
    uint32_t key[V], lmax = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane * V + i;
      const bool in = (VEC || e < E) && (a.G == 1 || (open >> (e / n)) & 1u);
      key[i] = in ? score_key(by_x ? x[i] : c[i]) : 0u;
      lmax = max(lmax, key[i]);
    }
    // the k-th largest distinct value among the lanes' maxima, less what the errors
    // of two values may hide
    uint32_t theta = 0;
    {
      uint32_t lm = lmax;
      for (int r = 0; r < k; ++r) {
        theta = __reduce_max_sync(kAll, lm);
        if (lm == theta) lm = 0u;
      }
    }
    if (!by_x && theta > 0) {
      const float f = key_score(theta);
      theta = f > -kInf ? score_key(f - (2.0f * err + 0x1p-22f * fabsf(f))) : theta;
    }
    uint32_t cmask = 0;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (key[i] != 0u && key[i] >= theta) cmask |= 1u << i;
    const int nc = __popc(cmask);
    const int C = (int)__reduce_add_sync(kAll, (unsigned)nc);
    int sel = -1, slot_out = -1;  // this lane's selected expert and its slot
    bool again = false;           // f32 cannot tell
    __syncwarp();
    if (C <= 32) {
      int slot = warp_incl_scan(nc, lane) - nc;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (cmask & (1u << i)) {
          ws.cand[slot] = ((unsigned long long)key[i] << 32) | (uint32_t) ~(uint32_t)(lane * V + i);
          ws.x[slot++] = x[i];
        }
      __syncwarp();
      const unsigned long long cand = lane < C ? ws.cand[lane] : 0ull;
      const float cx = lane < C ? ws.x[lane] : 0.0f;
      int rank = 0;
      for (int j = 0; j < C; ++j) rank += ws.cand[j] > cand ? 1 : 0;
      const int e = (int)~(uint32_t)cand;
      if (!by_x) {
        // neighbours in rank that are too close, and not the same x and bias
        __syncwarp();
        if (lane < C) {
          ws.cand[rank] = cand;
          ws.x[rank] = cx;
        }
        __syncwarp();
        bool near = false;
        if (lane < k && lane + 1 < C) {
          const unsigned long long p = ws.cand[lane], q = ws.cand[lane + 1];
          const float cp = key_score((uint32_t)(p >> 32)), cq = key_score((uint32_t)(q >> 32));
          near = cq > -kInf && cp - cq <= 2.0f * err + 0x1p-22f * fmaxf(fabsf(cp), fabsf(cq));
          if (near && ws.x[lane] == ws.x[lane + 1] &&
              __ldg(a.bias + (int)~(uint32_t)p) == __ldg(a.bias + (int)~(uint32_t)q))
            near = false;
        }
        again = __any_sync(kAll, near);
      }
      if (again) {
        if (a.func == MOE_SCORE_SOFTMAX && tok.z == 0.0) tok.z = sum64(tok, E, lane);
        const double d = lane < C ? choice64(tok, e) : 0.0;
        rank = 0;
        for (int j = 0; j < C; ++j) {
          const double od = __shfl_sync(kAll, d, j);
          const int oe = __shfl_sync(kAll, e, j);
          rank += od > d || (od == d && oe < e) ? 1 : 0;
        }
      }
      if (lane < C && rank < k) {
        sel = e;
        slot_out = rank;
      }
    } else {
      // many candidates: round by round, one more round for the border
      float last_c = 0.0f, last_x = 0.0f, last_b = 0.0f;
      for (int r = 0; r <= k; ++r) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (key[i] > best) best = key[i], at = i;
        const uint32_t m = __reduce_max_sync(kAll, best);
        const int win = (int)__reduce_min_sync(
            kAll, best == m ? (uint32_t)(lane * V + at) : 0xFFFFFFFFu);
        if (m == 0u) break;
        if (!by_x) {
          const float wc = key_score(m), wx = __ldg(tok.row + win), wb = __ldg(a.bias + win);
          if (r > 0 && wc > -kInf && !(wx == last_x && wb == last_b) &&
              last_c - wc <= 2.0f * err + 0x1p-22f * fmaxf(fabsf(wc), fabsf(last_c)))
            again = true;
          last_c = wc, last_x = wx, last_b = wb;
        }
        if (r == k) break;
        if (lane == r) sel = win, slot_out = r;
        if (win / V == lane) {
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (lane * V + i == win) key[i] = 0u;
        }
      }
      if (again) {
        if (a.func == MOE_SCORE_SOFTMAX && tok.z == 0.0) tok.z = sum64(tok, E, lane);
        sel = select64(tok, E, a.G, open, k, lane, list);
        slot_out = lane < k ? lane : -1;
      }
    }

    // ---- weights
    const bool have = slot_out >= 0;
    const float xs = have ? __ldg(tok.row + sel) : -kInf;
    float w = weight_score(a.func, a.renorm, xs, have, tok.m, z_inv);
    if (a.renorm) {
      const float sum = warp_sum(w);
      w = sum > 0.0f ? __fdiv_rn(w, sum) : 0.0f;
    }
    if (have) {
      a.idx[t * k + slot_out] = sel;
      a.w[t * k + slot_out] = w * a.scale;
    }
    __syncwarp();
  }
}

template <int V, bool VEC>
cudaError_t launch_v(const LaunchCtx& c, const RouterArgs& a) {
  auto* kernel = router_gate_kernel<V, VEC>;
  const size_t smem = (size_t)kWarps * a.E * 8;
  if (smem > 40 * 1024) {
    static SmemOptIn opt_in;
    const cudaError_t e = opt_in.once(kernel);
    if (e != cudaSuccess) return e;
  }
  const int64_t need = (a.T + kWarps - 1) / kWarps, cap = (int64_t)c.num_sms * 8;
  return launch_pdl(kernel, dim3((unsigned)(need < cap ? need : cap)), kWarps * 32, smem, c.stream,
                    a);
}

// ------------------------------------------------------------------ backward

// One warp per token.  The row is copied (or zeroed) first; the selected entries are
// then written over by their lanes, from add's values read before.  For the softmax
// without renormalisation every entry changes.
template <int VEC>
__global__ void __launch_bounds__(kWarps * 32)
    router_gate_backward_kernel(const RouterArgs a, unsigned* err) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t t = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (t >= a.T) return;
  const int E = a.E, k = a.k;
  const float* row = a.scores + t * E;
  const float* add = a.add ? a.add + t * E : nullptr;
  float* out = a.grad_scores + t * E;
  int e = -1;
  float g = 0.0f, x = -kInf, before = 0.0f;
  if (lane < k) {
    e = a.idx[t * k + lane];
    if (e < 0 || e >= E) {
      flag_error(err, MOE_DEVERR_EXPERT_RANGE);
      e = -1;
    }
  }
  const bool have = e >= 0;
  if (have) {
    g = a.grad_w[t * k + lane];
    x = row[e];
    if (add) before = add[e];
  }
  const bool dense = a.func == MOE_SCORE_SOFTMAX && !a.renorm;
  float m = 0.0f, z_inv = 0.0f;
  if (dense) {
    m = -kInf;
    for (int c = lane; c < E; c += 32) m = fmaxf(m, row[c]);
    m = warp_max(m);
    if (m == -kInf) m = 0.0f;
    float z = 0.0f;
    for (int c = lane; c < E; c += 32) z += expf(row[c] - m);
    z = warp_sum(z);
    z_inv = z > 0.0f ? __fdiv_rn(1.0f, z) : 0.0f;
  }
  float w = weight_score(a.func, a.renorm, x, have, m, z_inv);
  if (a.renorm) {
    const float sum = warp_sum(w);
    w = sum > 0.0f ? __fdiv_rn(w, sum) : 0.0f;
  }
  const float dot = warp_sum(g * w);  // sum_j g_j w_j / scale, or sum_j g_j s_j
  float d = a.scale * w * (a.renorm || dense ? g - dot : g);
  if (a.func == MOE_SCORE_SIGMOID) d *= sigmoid_f32(-x);
  if (dense) {
    const float f = a.scale * dot;
    for (int c = lane; c < E; c += 32)
      out[c] = (add ? add[c] : 0.0f) - expf(row[c] - m) * z_inv * f;
  } else if (add != out) {
    if constexpr (VEC == 4) {
      for (int c = lane * 4; c < E; c += 128) {
        const uint4 v = add ? ld_once_v4(add + c) : make_uint4(0, 0, 0, 0);
        st_stream_v4(out + c, v);
      }
    } else {
      for (int c = lane; c < E; c += 32) out[c] = add ? add[c] : 0.0f;
    }
  }
  __syncwarp();
  if (have) out[e] = before + d;
}

}  // namespace

cudaError_t launch_router_gate(const LaunchCtx& c, const RouterArgs& a) {
  const bool al = reinterpret_cast<uintptr_t>(a.scores) % 16 == 0;
  if (a.E <= 32) return launch_v<1, false>(c, a);
  if (a.E <= 64) return launch_v<2, false>(c, a);
  if (a.E <= 128) return a.E == 128 && al ? launch_v<4, true>(c, a) : launch_v<4, false>(c, a);
  if (a.E <= 256) return a.E == 256 && al ? launch_v<8, true>(c, a) : launch_v<8, false>(c, a);
  if (a.E <= 512) return a.E == 512 && al ? launch_v<16, true>(c, a) : launch_v<16, false>(c, a);
  return launch_v<32, false>(c, a);
}

cudaError_t launch_router_gate_backward(const LaunchCtx& c, const RouterArgs& a) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.add) |
                       reinterpret_cast<uintptr_t>(a.grad_scores);
  const unsigned blocks = (unsigned)((a.T + kWarps - 1) / kWarps);
  if (a.E % 4 == 0 && at % 16 == 0)
    return launch_pdl(router_gate_backward_kernel<4>, dim3(blocks), kWarps * 32, 0, c.stream, a,
                      c.err);
  return launch_pdl(router_gate_backward_kernel<1>, dim3(blocks), kWarps * 32, 0, c.stream, a,
                    c.err);
}

}  // namespace moe
