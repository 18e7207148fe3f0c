// Scored router: softmax or sigmoid scores, a bias that only the choice
// sees, expert groups, top-k, renormalised weights.
//
//   l[t][e] = x[t] . W[e],  s = sigmoid(l) or softmax(l),  c = s + bias
//   group score = the largest c of the group, or the sum of its two largest;
//   the best groups stay, and the k largest c of their experts are picked
//
// The choice must be that of c evaluated in fp64.  As in the softmax router,
// logits are summed in fp32 with a proven bound |L - l| <= D, the bound is
// carried through to c (|C - c| <= Dc), and only what the intervals
// [C - Dc, C + Dc] leave open is evaluated in fp64, where every bf16 x fp32
// product is exact: the experts that could change which groups stay, then
// the experts whose order among the picks, or whose place in or out of
// them, is open.  A token's rows that hold no finite bound (overflow, NaN,
// Inf) are evaluated in fp64 throughout.
//
// Where the scores do not need each other (sigmoid) an open expert costs one
// fp64 dot product.  Without a bias and without sums of two, c rises with l,
// so the logits themselves are compared, in softmax mode too; a softmax with
// a bias (or sums of two) needs the denominator, so an open token is
// evaluated whole.
//
// Carrying the bound (u = 2^-24): sigmoid' = s (1 - s), and over an interval
// of half width D <= 0.05 it grows by at most e^0.05 < 1.06; expf (2 ulp), the
// sum and the division err by less than 8 u s, the bias addition by u |c|.
// Softmax: every numerator and the denominator err by a relative
// 2 D_max + 4 u (|l - max|) + (E / 32 + 16) u at most, D_max <= 0.05.
#include "common.cuh"

namespace moeq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMinCtas = 3;

struct Scored {
  const __nv_bfloat16* x;
  const float* w;
  const float* bias;
  RoutePartials lg;
  int T, d, E, k;
  int sigmoid, groups, kept, group_top, renorm;
  int by_logits;  // c rises with l: compare the logits
  float scale;
  int32_t* out_idx;
  float* out_w;
};

// NaN counts as -inf.
__device__ __forceinline__ double ordered(double v) { return v == v ? v : -INFINITY; }

// The k largest of the values v[m] (expert lane + 32 m, those with bit m of
// `allowed`), descending, ties to the lower index; lane j < k receives pick
// j.  There are at least k allowed experts.
template <typename V, int P>
__device__ __forceinline__ int pick_topk(const V (&v)[P], uint32_t allowed, int k, int lane) {
  int mine = 0;
  for (int j = 0; j < k; ++j) {
    V best = -INFINITY;
    int e = 0x7fffffff;
#pragma unroll
    for (int m = 0; m < P; ++m)
      if (((allowed >> m) & 1u) && (e == 0x7fffffff || v[m] > best)) {
        best = v[m];
        e = lane + 32 * m;
      }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const V ov = __shfl_xor_sync(0xffffffffu, best, o);
      const int oe = __shfl_xor_sync(0xffffffffu, e, o);
      if (oe != 0x7fffffff && (e == 0x7fffffff || ov > best || (ov == best && oe < e))) {
        best = ov;
        e = oe;
      }
    }
    if (lane == j) mine = e;
    if ((e & 31) == lane) allowed &= ~(1u << (e >> 5));
  }
  return mine;
}

// Group score of group g (experts g gs .. + gs - 1): the largest, or the sum
// of the two largest, of f(e).
template <typename F>
__device__ __forceinline__ auto group_score(int g, int gs, int top, F f) {
  auto a = f(g * gs);
  decltype(a) b = -INFINITY;
  for (int i = 1; i < gs; ++i) {
    const auto v = f(g * gs + i);
    if (v > a) {
      b = a;
      a = v;
    } else if (v > b) {
      b = v;
    }
  }
  return top == 2 ? a + b : a;
}

template <int P>
__global__ void __launch_bounds__(kThreads, kMinCtas) k_route_scored(const Scored A) {
  pdl_wait();
  pdl_trigger();
  __shared__ float c_s[kWarps][32 * P], d_s[kWarps][32 * P];  // choice values and bounds
  __shared__ double l64[kWarps][32 * P];                      // refined logits
  __shared__ uint8_t cand[kWarps][32 * P];
  __shared__ int n_cand[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T = A.T, E = A.E, k = A.k, G = A.groups, gs = E / G;
  const int t = blockIdx.x * kWarps + warp;
  const bool grouped = A.kept < G;
  float L[P], C[P], D[P];
  uint32_t in_range = 0, refined = 0;  // bit m: expert lane + 32 m
  bool hard = false;                   // the whole row goes to fp64
  float row_max = 0.f, row_sum = 1.f;  // softmax
#pragma unroll
  for (int m = 0; m < P; ++m)
    if (lane + 32 * m < E) in_range |= 1u << m;

  if (t < T) {
    float xq = 0.f;
    for (int s = 0; s < A.lg.splits; ++s) xq += A.lg.xsq[static_cast<size_t>(s) * T + t];
    const float xn = sqrtf(xq);
    float d_max = 0.f;
#pragma unroll
    for (int m = 0; m < P; ++m) {
      const int e = lane + 32 * m;
      L[m] = -INFINITY;
      D[m] = 0.f;
      if (e < E) {
        float v = 0.f, wq = 0.f;
        for (int s = 0; s < A.lg.splits; ++s) {
          v += A.lg.partial[(static_cast<size_t>(s) * T + t) * E + e];
        }
        for (int s = 0; s < A.lg.w_splits; ++s) wq += A.lg.wsq[static_cast<size_t>(s) * E + e];
        L[m] = v;
        D[m] = A.lg.gamma * xn * sqrtf(wq) * (1.0f + 0.00390625f) + 1.2e-7f * fabsf(v) +
                 5e-37f * (xn + sqrtf(wq)) + 1e-30f;
        d_max = fmaxf(d_max, D[m]);
        hard |= !(fabsf(v) <= 3.0e38f) || !(D[m] <= 3.0e38f);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) d_max = fmaxf(d_max, __shfl_xor_sync(0xffffffffu, d_max, o));
    hard = __any_sync(0xffffffffu, hard);
    if (!A.sigmoid) {
      float mx = -INFINITY;
#pragma unroll
      for (int m = 0; m < P; ++m) mx = fmaxf(mx, L[m]);
#pragma unroll
      for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      float sum = 0.f;
#pragma unroll
      for (int m = 0; m < P; ++m) sum += (in_range >> m) & 1u ? expf(L[m] - mx) : 0.f;
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      row_max = mx;
      row_sum = sum;
    }
    bool wide = false;
#pragma unroll
    for (int m = 0; m < P; ++m) {
      const int e = lane + 32 * m;
      C[m] = L[m];
      if (!A.by_logits && e < E) {
        const float b = A.bias ? A.bias[e] : 0.f;
        float s, ds;
        if (A.sigmoid) {
          s = 1.0f / (1.0f + expf(-L[m]));
          ds = 1.06f * D[m] * (s * (1.0f - s) + 2.0e-7f) + 5.0e-7f * s;
        } else {
          s = expf(L[m] - row_max) / row_sum;
          ds = s * (2.2f * d_max + 2.4e-7f * (row_max - L[m]) + 6.0e-8f * (E / 32 + 16)) * 1.06f;
        }
        wide |= !(d_max <= 0.05f) || b != b || b == INFINITY;
        C[m] = s + b;
        D[m] = C[m] == -INFINITY ? 0.f : ds + 1.2e-7f * fabsf(C[m]) + 1e-37f;
      }
      c_s[warp][lane + 32 * m] = C[m];
      d_s[warp][lane + 32 * m] = D[m];
    }
    hard |= __any_sync(0xffffffffu, wide);
  }
  __syncwarp();

  // fp64 logits of the experts that every token of the CTA has listed (bit m
  // of `open`), spread over its warps; `refined` gains them
  auto refine = [&](uint32_t open) {
    open &= ~refined;
    int n = 0;
#pragma unroll
    for (int m = 0; m < P; ++m) {
      const unsigned bal = __ballot_sync(0xffffffffu, (open >> m) & 1u);
      if ((open >> m) & 1u) cand[warp][n + __popc(bal & ((1u << lane) - 1u))] = static_cast<uint8_t>(lane + 32 * m);
      n += __popc(bal);
    }
    if (lane == 0) n_cand[warp] = n;
    __syncthreads();
    int total = 0;
    for (int w = 0; w < kWarps; ++w) total += n_cand[w];
    for (int item = warp; item < total; item += kWarps) {
      int w = 0, r = item;
      while (r >= n_cand[w]) r -= n_cand[w++];
      const int tu = blockIdx.x * kWarps + w, e = cand[w][r];
      const double v = dot_bf16_f32_fp64(A.x + static_cast<size_t>(tu) * A.d, A.w + static_cast<size_t>(e) * A.d, A.d,
                                         lane);
      if (lane == 0) l64[w][e] = v;
    }
    __syncthreads();  // also: the lists may be rewritten
    refined |= open;
  };
  // fp64 choice value of a refined expert (sigmoid or logits; a softmax that
  // needs its denominator is `hard` whenever it is open)
  auto value64 = [&](int e) -> double {
    const double l = l64[warp][e];
    if (A.by_logits) return ordered(l);
    return ordered(1.0 / (1.0 + exp(-l)) + (A.bias ? static_cast<double>(A.bias[e]) : 0.0));
  };

  // ---- which groups stay ------------------------------------------------------
  uint32_t group_in = 0, group_open = 0;  // bit g, the same in every lane
  uint32_t open = 0;
  if (t < T && grouped && !hard) {
    float lo = -INFINITY, up = -INFINITY, cut = 0.f;
    if (lane < G) {
      const float* cs = c_s[warp];
      const float* ds = d_s[warp];
      float a = -INFINITY, b = -INFINITY;  // two largest lower bounds
      float ua = -INFINITY, ub = -INFINITY;
      for (int i = 0; i < gs; ++i) {
        const float v = cs[lane * gs + i], dv = ds[lane * gs + i];
        const float l = v - dv, h = v + dv;
        if (l > a) { b = a; a = l; } else if (l > b) { b = l; }
        if (h > ua) { ub = ua; ua = h; } else if (h > ub) { ub = h; }
      }
      cut = A.group_top == 2 ? b : a;
      // outward rounding of the two sums
      lo = A.group_top == 2 ? a + b - 1.2e-7f * (fabsf(a) + fabsf(b)) : a;
      up = A.group_top == 2 ? ua + ub + 1.2e-7f * (fabsf(ua) + fabsf(ub)) : ua;
      if (lo != lo) lo = -INFINITY;
      if (up != up) up = -INFINITY;
    }
    int may = 0, sure = 0;  // groups that may, that certainly do, come before this one
    for (int h = 0; h < G; ++h) {
      const float ol = __shfl_sync(0xffffffffu, lo, h), ou = __shfl_sync(0xffffffffu, up, h);
      if (h != lane) {
        may += ou >= lo;
        sure += ol > up;
      }
    }
    group_in = __ballot_sync(0xffffffffu, lane < G && may < A.kept);
    group_open = __ballot_sync(0xffffffffu, lane < G && may >= A.kept && sure < A.kept);
    if (group_open) {
      if (!A.sigmoid && !A.by_logits) {
        hard = true;
      } else {
#pragma unroll
        for (int m = 0; m < P; ++m) {
          const int e = lane + 32 * m, g = min(e / gs, G - 1);
          const float gc = __shfl_sync(0xffffffffu, cut, g);
          if (e < E && ((group_open >> g) & 1u) && C[m] + D[m] >= gc) open |= 1u << m;
        }
      }
    }
  }
  if (hard) open = in_range;
  if (t >= T) open = 0;
  if (grouped || __syncthreads_or(hard)) refine(open);
  __syncwarp();

  // ---- the picks -----------------------------------------------------------------
  double H[P];  // hard rows: fp64 choice values
  double row_max64 = 0.0, row_sum64 = 1.0;
  if (t < T && hard) {
    if (!A.sigmoid) {
      double mx = -INFINITY;
      bool nan = false;
#pragma unroll
      for (int m = 0; m < P; ++m)
        if ((in_range >> m) & 1u) {
          const double l = l64[warp][lane + 32 * m];
          nan |= l != l;
          mx = fmax(mx, l);
        }
#pragma unroll
      for (int o = 16; o; o >>= 1) mx = fmax(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      if (__any_sync(0xffffffffu, nan)) mx = NAN;
      double sum = 0.0;
#pragma unroll
      for (int m = 0; m < P; ++m)
        if ((in_range >> m) & 1u) sum += exp(l64[warp][lane + 32 * m] - mx);
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      row_max64 = mx;
      row_sum64 = sum;
    }
#pragma unroll
    for (int m = 0; m < P; ++m) {
      const int e = lane + 32 * m;
      H[m] = -INFINITY;
      if (e < E) {
        const double l = l64[warp][e];
        if (A.by_logits) {
          // (a softmax row with a NaN, or two infinities' difference, is NaN throughout)
          // (a sigmoid of -inf is 0: above a NaN, which counts as -inf)
          H[m] = A.sigmoid || (row_max64 - row_max64 == 0.0) ? ordered(l) : -INFINITY;
          if (A.sigmoid && l == -INFINITY) H[m] = -1.7e308;
        } else {
          const double s = A.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - row_max64) / row_sum64;
          H[m] = ordered(s + (A.bias ? static_cast<double>(A.bias[e]) : 0.0));
        }
      }
    }
  }
  if (t < T && grouped) {
    // the groups still open, or (hard rows) all of them, by their fp64 scores
    if (hard) {
      group_in = 0;
      group_open = G == 32 ? 0xffffffffu : (1u << G) - 1u;
    }
    if (group_open) {
      // hard rows: the values go through l64 (the row's logits are kept apart)
      double keep[P];
      if (hard) {
#pragma unroll
        for (int m = 0; m < P; ++m) keep[m] = (in_range >> m) & 1u ? l64[warp][lane + 32 * m] : 0.0;
        __syncwarp();
#pragma unroll
        for (int m = 0; m < P; ++m)
          if ((in_range >> m) & 1u) l64[warp][lane + 32 * m] = H[m];
        __syncwarp();
      }
      // mark of the experts refined for the groups: a bound of -1 in d_s
      if (!hard) {
#pragma unroll
        for (int m = 0; m < P; ++m)
          if ((refined >> m) & 1u) d_s[warp][lane + 32 * m] = -1.f;
        __syncwarp();
      }
      double gv = -INFINITY;
      if (lane < G && ((group_open >> lane) & 1u)) {
        gv = group_score(lane, gs, A.group_top, [&](int e) -> double {
          if (hard) return l64[warp][e];
          return d_s[warp][e] < 0.f ? value64(e) : -INFINITY;  // the others are below the group's best
        });
        gv = ordered(gv);
      }
      int before = 0;
      for (int h = 0; h < G; ++h) {
        const double o = __shfl_sync(0xffffffffu, gv, h);
        if (((group_open >> h) & 1u) && (o > gv || (o == gv && h < lane))) ++before;
      }
      const int room = A.kept - __popc(group_in);
      const bool stay = lane < G && ((group_open >> lane) & 1u) && before < room;
      group_in |= __ballot_sync(0xffffffffu, stay);
      if (hard) {
        __syncwarp();
#pragma unroll
        for (int m = 0; m < P; ++m)
          if ((in_range >> m) & 1u) l64[warp][lane + 32 * m] = keep[m];
        __syncwarp();
      }
    }
  }
  uint32_t allowed = in_range;
  if (grouped) {
#pragma unroll
    for (int m = 0; m < P; ++m)
      if (!((group_in >> min((lane + 32 * m) / gs, 31)) & 1u)) allowed &= ~(1u << m);
  }
  int mine = 0;
  open = 0;
  bool again = false;
  if (t < T && !hard) {
    mine = pick_topk(C, allowed, k, lane);
    // intervals of the picks, lane j holding pick j's
    const float* cs = c_s[warp];
    float lo = INFINITY, up = -INFINITY;
    {
      // bound of pick j, from its lane (d_s may hold marks)
      float dv = 0.f;
#pragma unroll
      for (int m = 0; m < P; ++m) {
        const float o = __shfl_sync(0xffffffffu, D[m], mine & 31);
        if ((mine >> 5) == m) dv = o;
      }
      if (lane < k) {
        lo = cs[mine] - dv;
        up = cs[mine] + dv;
      }
    }
    // pick j is open when its interval meets another pick's ...
    bool mark = false;
    for (int i = 0; i < k; ++i) {
      const float ol = __shfl_sync(0xffffffffu, lo, i), ou = __shfl_sync(0xffffffffu, up, i);
      if (lane < k && i != lane) mark |= ol <= up && lo <= ou;
    }
    // ... or that of an expert left out
    float lo_min = lo;
#pragma unroll
    for (int o = 16; o; o >>= 1) lo_min = fminf(lo_min, __shfl_xor_sync(0xffffffffu, lo_min, o));
    float hi = -INFINITY;
    bool any_out = false;
    uint32_t picked = 0;
    for (int j = 0; j < k; ++j) {
      const int e = __shfl_sync(0xffffffffu, mine, j);
      if ((e & 31) == lane) picked |= 1u << (e >> 5);
    }
#pragma unroll
    for (int m = 0; m < P; ++m)
      if (((allowed & ~picked) >> m) & 1u) {
        hi = any_out ? fmaxf(hi, C[m] + D[m]) : C[m] + D[m];
        any_out = true;
        if (C[m] + D[m] >= lo_min) open |= 1u << m;
      }
    any_out = __any_sync(0xffffffffu, any_out);
#pragma unroll
    for (int o = 16; o; o >>= 1) hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    if (lane < k && any_out) mark |= lo <= hi;
    unsigned marks = __ballot_sync(0xffffffffu, mark);
    again = marks != 0;
    while (marks) {
      const int e = __shfl_sync(0xffffffffu, mine, __ffs(marks) - 1);
      marks &= marks - 1;
      if ((e & 31) == lane) open |= 1u << (e >> 5);
    }
    if (again && !A.sigmoid && !A.by_logits) open = in_range;
  }
  refine(open);
  if (t >= T) return;
  __syncwarp();
  const bool whole = !hard && again && !A.sigmoid && !A.by_logits;  // softmax with a bias: now evaluated throughout
  if (whole) {
    double mx = -INFINITY, sum = 0.0;
#pragma unroll
    for (int m = 0; m < P; ++m)
      if ((in_range >> m) & 1u) mx = fmax(mx, l64[warp][lane + 32 * m]);
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmax(mx, __shfl_xor_sync(0xffffffffu, mx, o));
#pragma unroll
    for (int m = 0; m < P; ++m)
      if ((in_range >> m) & 1u) sum += exp(l64[warp][lane + 32 * m] - mx);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
    for (int m = 0; m < P; ++m) {
      const int e = lane + 32 * m;
      H[m] = e < E ? ordered(exp(l64[warp][e] - mx) / sum + (A.bias ? static_cast<double>(A.bias[e]) : 0.0))
                   : -INFINITY;
    }
    row_max64 = mx;
    row_sum64 = sum;
  }
  const bool exact = hard || whole;
  if (exact) {
    mine = pick_topk(H, allowed, k, lane);
  } else if (again) {
#pragma unroll
    for (int m = 0; m < P; ++m)
      H[m] = (refined >> m) & 1u ? value64(lane + 32 * m) : static_cast<double>(C[m]);
    mine = pick_topk(H, allowed, k, lane);
  }

  // ---- weights: lane j < k holds pick j ----------------------------------------------
  double l = 0.0;
#pragma unroll
  for (int m = 0; m < P; ++m) {
    const float o = __shfl_sync(0xffffffffu, L[m], mine & 31);
    const bool r = (__shfl_sync(0xffffffffu, refined, mine & 31) >> m) & 1u;
    if ((mine >> 5) == m) l = r ? l64[warp][mine] : static_cast<double>(o);
  }
  float wt;
  if (exact) {
    double s = A.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - row_max64) / row_sum64;
    if (A.renorm) {
      double sum = lane < k ? s : 0.0;
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      s = sum == 0.0 ? 0.0 : s / sum;
    }
    wt = static_cast<float>(s * A.scale);
  } else {
    const float lf = static_cast<float>(l);
    float s = A.sigmoid ? 1.0f / (1.0f + expf(-lf)) : expf(lf - row_max);
    if (A.renorm) {
      // scores so small that they leave fp32's range: taken from the largest
      float top = lane < k ? (A.sigmoid ? lf : 0.f) : -INFINITY;
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (A.sigmoid && top < -60.f) {
        s = expf(lf - top);  // sigmoid(l) = e^l (1 + tiny)
      } else if (!A.sigmoid) {
        float mx = lane < k ? lf : -INFINITY;
#pragma unroll
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        s = expf(lf - mx);
      }
      float sum = lane < k ? s : 0.f;
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      s /= sum;
    } else if (!A.sigmoid) {
      s /= row_sum;
    }
    wt = s * A.scale;
  }
  if (lane < k) {
    A.out_idx[static_cast<size_t>(t) * k + lane] = mine;
    A.out_w[static_cast<size_t>(t) * k + lane] = wt;
  }
}

// The logits' kernel: the tensor cores for batches that fill a tile's tokens.
constexpr int kTensorT = 128;

}  // namespace
}  // namespace moeq

using namespace moeq;

extern "C" {

size_t moe_route_scored_workspace_bytes(int T, int d, int E) {
  if (T <= 0 || d <= 0 || E <= 0) return 256;
  const size_t small = route_workspace_bytes(std::min(T, kTensorT - 1), d, E);
  return T >= kTensorT ? std::max(small, route_tc_workspace_bytes(T, d, E)) : small;
}

moe_status_t moe_route_scored(const void* x, const float* w_router, const float* bias, int T, int d, int E, int k,
                              int scoring, int n_groups, int topk_groups, int group_top, int renorm, double scale,
                              int32_t* topk_idx, float* topk_w, void* workspace, size_t workspace_bytes,
                              int32_t* status, moe_stream_t stream) {
  const char* fn = "moe_route_scored";
  moe_status_t st = route_check_args(x, w_router, T, d, E, k, topk_idx, topk_w, fn);
  if (st != MOE_OK) return st;
  if (scoring != MOE_SCORE_SOFTMAX && scoring != MOE_SCORE_SIGMOID) {
    set_error("%s: unknown scoring %d", fn, scoring);
    return MOE_ERR_INVALID_ARG;
  }
  if (n_groups <= 0 || topk_groups <= 0 || topk_groups > n_groups || (group_top != 1 && group_top != 2) ||
      E % n_groups) {
    set_error("%s: bad groups: n_groups=%d (of E=%d) topk_groups=%d group_top=%d", fn, n_groups, E, topk_groups,
              group_top);
    return MOE_ERR_INVALID_ARG;
  }
  if (n_groups > 32 || E / n_groups < group_top || topk_groups * (E / n_groups) < k) {
    set_error("%s: at most 32 groups, of group_top=%d or more experts, the kept ones with k=%d or more", fn, group_top,
              k);
    return MOE_ERR_UNSUPPORTED_SHAPE;
  }
  if (T == 0) return MOE_OK;
  if (!workspace || workspace_bytes < moe_route_scored_workspace_bytes(T, d, E)) {
    set_error("%s: workspace %zu < %zu bytes", fn, workspace_bytes, moe_route_scored_workspace_bytes(T, d, E));
    return MOE_ERR_WORKSPACE;
  }
  if (reinterpret_cast<uintptr_t>(workspace) & 15u) {
    set_error("%s: workspace must be 16-byte aligned", fn);
    return MOE_ERR_INVALID_ARG;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Scored A{};
  st = T >= kTensorT ? launch_route_partials_tc(x, w_router, T, d, E, workspace, status, &A.lg, s)
                          : launch_route_partials(x, w_router, T, d, E, k, workspace, workspace_bytes, &A.lg, s);
  if (st != MOE_OK) return st;
  A.x = static_cast<const __nv_bfloat16*>(x);
  A.w = w_router;
  A.bias = bias;
  A.T = T;
  A.d = d;
  A.E = E;
  A.k = k;
  A.sigmoid = scoring == MOE_SCORE_SIGMOID;
  A.groups = n_groups;
  A.kept = topk_groups;
  A.group_top = group_top;
  A.renorm = renorm != 0;
  A.by_logits = !bias && (group_top == 1 || topk_groups == n_groups);
  A.scale = static_cast<float>(scale);
  A.out_idx = topk_idx;
  A.out_w = topk_w;
  auto kern = E <= 32 ? k_route_scored<1> : E <= 64 ? k_route_scored<2> : E <= 128 ? k_route_scored<4> : k_route_scored<8>;
  return cuda_check(launch_pdl(pdl_for(static_cast<long>(T) * k), kern, dim3(ceil_div(T, kWarps)), dim3(kThreads), 0, s, A),
                    "moe_route_scored launch");
}

}  // extern "C"
