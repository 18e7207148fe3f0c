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
// Inf) are evaluated in fp64 throughout, and where scores are compared (not the
// logits) so are those with a bound above 0.05: |x| |W_e| above 3300 at d =
// 4096.  A batch of such tokens is slow: 250 of them, 256 experts, sigmoid with a
// bias, 1093 us in place of 39 (softmax with a bias, which lists them, 95).
//
// Where the scores do not need each other an open expert costs one fp64 dot
// product: sigmoid; without a bias and without sums of two, where c rises with
// l and the logits themselves are compared, in softmax mode too; and softmax
// without a bias, where the denominator is common to all and e^(l - a
// constant) is compared.  A softmax with a bias needs the denominator, so an
// open token is evaluated whole: such tokens are listed, and two more
// kernels compute their logits in fp64 as one product (k_route_rows64) and
// pick (k_route_whole).  4096 tokens, 256 experts, d = 4096, 330 of them
// open: 128 us (rows 55, picks 25), 689 when each CTA evaluated its own.
//
// Carrying the bound (u = 2^-24): sigmoid' = s (1 - s), and over an interval
// of half width D <= 0.05 it grows by at most e^0.05 < 1.06; __expf errs by (2 +
// 1.2 |l|) 2^-23 relative, of which s feels the part 1 - s, the sum and the
// division (2 ulp) by less than 6 u s, the bias addition by u |c|.
// Softmax: every numerator and the denominator err by a relative
// 2 D_max + 4 u (|l - max|) + (E / 32 + 20) u at most, D_max <= 0.05.
//
// A warp takes a token, its experts spread over the lanes, so the picks are
// warp reductions and the intervals stay in registers; what is open goes to
// the whole CTA, an expert's fp64 dot product to a warp, because the tokens
// of a CTA have very different numbers of open experts (a warp refining its
// own token's took 106 us in place of 94 for 8191 tokens, 256 experts, d =
// 4096).  The time goes into waiting, on those products' barriers and loads
// (41 % of the issue slots busy): of 91 us for that call the weights' split
// takes 5, the logits 50 and this kernel the rest.  4096 tokens, 256
// experts, 4 of 8 groups, d = 2048: 47 us; 250 tokens, 128 experts, d = 4096: 27
// us.  Up to 8 tokens with few logits run as one launch of a cluster (below).
#include "common.cuh"

namespace moeq {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct Scored {
  const __nv_bfloat16* x;
  const float* w;
  const float* bias;
  RoutePartials lg;
  int T, d, E, k;
  int sigmoid, groups, kept, group_top, renorm;
  int by_logits;  // c rises with l: compare the logits
  int alone;      // an expert's choice value needs no other's logit
  int32_t* list;  // where not: the tokens left for k_route_rows64 and k_route_whole (null: done here)
  float scale;
  int32_t* out_idx;
  float* out_w;
};

// A warp's token in shared memory.
template <int P>
struct Row {
  float l[32 * P], c[32 * P], d[32 * P];  // fp32 logits, choice values and their bounds
  double v[32 * P];                       // fp64: logits (raw rows) or choice values of the refined experts
  uint8_t cand[32 * P];                   // experts to refine; later the experts left out that may come in
  int n;
  int raw;  // v holds logits
  float shift;  // softmax without a bias: values are e^(l - shift)
};

// 2^-23 relative (the bounds have 2^-8 to spare for the norms).
__device__ __forceinline__ float sqrt_approx(float v) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// NaN counts as -inf.
__device__ __forceinline__ double ordered(double v) { return v == v ? v : -INFINITY; }

// a before b: larger value, of equal ones the lower index.
template <typename V>
__device__ __forceinline__ bool before(V va, int a, V vb, int b) {
  return va > vb || (va == vb && a < b);
}

// The k largest of v (shared memory, expert lane + 32 m for bit m of
// `allowed`), descending, ties to the lower index; lane j < k receives pick j.
template <int P>
__device__ __forceinline__ int pick_slow(const double* v, uint32_t allowed, int k, int lane) {
  int mine = 0;
  for (int j = 0; j < k; ++j) {
    double best = -INFINITY;
    int e = 0x7fffffff;
#pragma unroll 1
    for (int m = 0; m < P; ++m)
      if (((allowed >> m) & 1u) && (e == 0x7fffffff || v[lane + 32 * m] > best)) {
        best = v[lane + 32 * m];
        e = lane + 32 * m;
      }
#pragma unroll 1
    for (int o = 16; o; o >>= 1) {
      const double ov = __shfl_xor_sync(0xffffffffu, best, o);
      const int oe = __shfl_xor_sync(0xffffffffu, e, o);
      if (oe != 0x7fffffff && (e == 0x7fffffff || before(ov, oe, best, e))) {
        best = ov;
        e = oe;
      }
    }
    if (lane == j) mine = e;
    if ((e & 31) == lane) allowed &= ~(1u << (e >> 5));
  }
  return mine;
}

// Two largest of a stream of values.
struct Top2 {
  float a = -INFINITY, b = -INFINITY;
  __device__ __forceinline__ void add(float v) {
    b = fmaxf(b, fminf(a, v));
    a = fmaxf(a, v);
  }
  __device__ __forceinline__ void merge(int o) {
    const float oa = __shfl_xor_sync(0xffffffffu, a, o), ob = __shfl_xor_sync(0xffffffffu, b, o);
    add(oa);
    add(ob);
  }
};

// The softmax's maximum and denominator in fp64, from a raw row; a NaN among
// the logits makes both NaN.
template <int P>
__device__ __forceinline__ void softmax64(const double* v, int E, int lane, double& mx, double& sum) {
  bool nan = false;
  mx = -INFINITY;
#pragma unroll 1
  for (int e = lane; e < E; e += 32) {
    nan |= v[e] != v[e];
    mx = fmax(mx, v[e]);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) mx = fmax(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (__any_sync(0xffffffffu, nan)) mx = NAN;
  sum = 0.0;
#pragma unroll 2
  for (int e = lane; e < E; e += 32) sum += exp(v[e] - mx);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
}

// A row evaluated in fp64 throughout (row.v: logits of all experts): picks
// (lane j < k) and their scores s.
template <int P>
__device__ __noinline__ int pick_whole(const Scored& A, Row<P>& row, int lane, double& s) {
  const int E = A.E, G = A.groups, gs = E / G;
  double mx = 0.0, sum = 1.0;
  if (!A.sigmoid) softmax64<P>(row.v, E, lane, mx, sum);
  auto score = [&](double l) { return A.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - mx) / sum; };
  // logits out of the way, choice values in their place
  double l[P];
  uint32_t allowed = 0;
#pragma unroll
  for (int m = 0; m < P; ++m) {
    const int e = lane + 32 * m;
    l[m] = 0.0;
    if (e < E) {
      l[m] = row.v[e];
      allowed |= 1u << m;
    }
  }
  __syncwarp();
#pragma unroll
  for (int m = 0; m < P; ++m) {
    const int e = lane + 32 * m;
    if (e < E) {
      double c;
      if (A.by_logits) {
        // (a softmax row with a NaN, or an infinite maximum, is NaN throughout;
        // a sigmoid of -inf is 0: above a NaN, which counts as -inf)
        c = A.sigmoid || mx - mx == 0.0 ? ordered(l[m]) : -INFINITY;
        if (A.sigmoid && l[m] == -INFINITY) c = -1.7e308;
      } else {
        c = ordered(score(l[m]) + (A.bias ? static_cast<double>(A.bias[e]) : 0.0));
      }
      row.v[e] = c;
    }
  }
  __syncwarp();
  if (A.kept < G) {
    double gv = -INFINITY;
    if (lane < G) {
      double a = -INFINITY, b = -INFINITY;
#pragma unroll 1
      for (int i = 0; i < gs; ++i) {
        const double v = row.v[lane * gs + i];
        if (v > a) { b = a; a = v; } else if (v > b) { b = v; }
      }
      gv = ordered(A.group_top == 2 ? a + b : a);
    }
    int ahead = 0;
    for (int h = 0; h < G; ++h) {
      const double o = __shfl_sync(0xffffffffu, gv, h);
      ahead += before(o, h, gv, lane);
    }
    const unsigned in = __ballot_sync(0xffffffffu, lane < G && ahead < A.kept);
#pragma unroll
    for (int m = 0; m < P; ++m)
      if (((allowed >> m) & 1u) && !((in >> ((lane + 32 * m) / gs)) & 1u)) allowed &= ~(1u << m);
  }
  const int mine = pick_slow<P>(row.v, allowed, A.k, lane);
  double lv = 0.0;
#pragma unroll
  for (int m = 0; m < P; ++m) {
    const double o = __shfl_sync(0xffffffffu, l[m], mine & 31);
    if ((mine >> 5) == m) lv = o;
  }
  s = score(lv);
  return mine;
}

// Picks whose largest score is below e^this are weighed in fp64, where scores
// below e^-709.78 (sigmoid) or e^-745 (softmax) are 0, and so may their sum be.
// Above it such a score is 0 beside the largest in fp32 too (e^-104 is).
constexpr float kFarScores = -600.f;

// The weight of lane j's pick (j < k) from its fp64 score.
__device__ __forceinline__ float weight64(const Scored& A, double s, int lane) {
  if (A.renorm) {
    double sum = lane < A.k ? s : 0.0;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    s = sum == 0.0 ? 0.0 : s / sum;
  }
  return static_cast<float>(s * A.scale);
}

// The tokens block * kWarps .. of a CTA, a warp to each; P experts per lane
// (expert lane + 32 m).
// load(t, L, D): the token's fp32 logits and bounds.
template <int P, typename Load>
__device__ __forceinline__ void select_block(const Scored& A, Row<P>* rows, int block, Load load) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T = A.T, E = A.E, k = A.k, G = A.groups, gs = E / G;
  const int t = block * kWarps + warp;
  const bool here = t < T, grouped = A.kept < G;
  const bool alone = A.alone;
  Row<P>& row = rows[warp];
  float C[P], D[P];
  uint32_t in_range = 0, refined = 0;  // bit m: expert lane + 32 m
  bool hard = false;                   // the whole row goes to fp64
  float row_max = 0.f, row_sum = 1.f;  // softmax
#pragma unroll
  for (int m = 0; m < P; ++m)
    if (lane + 32 * m < E) in_range |= 1u << m;

  if (here) {
    float L[P];
    load(t, L, D);
    float d_max = 0.f, mx = -INFINITY;
#pragma unroll
    for (int m = 0; m < P; ++m) {
      hard |= !(fabsf(L[m]) <= 3.0e38f) || !(D[m] <= 3.0e38f);
      if (lane + 32 * m < E) {
        d_max = fmaxf(d_max, D[m]);
        mx = fmaxf(mx, L[m]);
      } else {
        L[m] = -INFINITY;
      }
      row.l[lane + 32 * m] = L[m];
    }
    // magnitudes order like their bits
    d_max = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(d_max)));
    hard = __any_sync(0xffffffffu, hard);
    if (!A.sigmoid) {
#pragma unroll
      for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      float sum = 0.f;
#pragma unroll
      for (int m = 0; m < P; ++m) sum += (in_range >> m) & 1u ? expf(L[m] - mx) : 0.f;
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      row_max = mx;
      row_sum = sum;
      if (lane == 0) row.shift = mx;
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
          s = __fdividef(1.0f, 1.0f + __expf(-L[m]));
          ds = (1.06f * D[m] + 1.2e-7f * (2.0f + 1.2f * fabsf(L[m]))) * (s * (1.0f - s) + 2.0e-7f) + 4.0e-7f * s;
        } else if (!A.bias) {
          s = expf(L[m] - row_max);
          ds = s * (1.06f * D[m] + 2.4e-7f * (row_max - L[m]) + 6e-7f);
        } else {
          s = __fdividef(expf(L[m] - row_max), row_sum);
          ds = s * (2.2f * d_max + 2.4e-7f * (row_max - L[m]) + 6.0e-8f * (E / 32 + 20)) * 1.06f;
        }
        wide |= !(d_max <= 0.05f) || b != b || b == INFINITY;
        C[m] = s + b;
        D[m] = C[m] == -INFINITY ? 0.f : ds + 1.2e-7f * fabsf(C[m]) + 1e-37f;
      }
      row.c[e] = C[m];
      row.d[e] = D[m];
    }
    hard |= __any_sync(0xffffffffu, wide);
  }

  // fp64 evaluation of the experts that the CTA's tokens have listed (bit m
  // of `open`), a warp to each; `refined` gains them
  auto refine = [&](uint32_t open) {
    open &= ~refined;
    if (!__syncthreads_or(open != 0)) return;
    int n = 0;
#pragma unroll
    for (int m = 0; m < P; ++m) {
      const unsigned bal = __ballot_sync(0xffffffffu, (open >> m) & 1u);
      if ((open >> m) & 1u) row.cand[n + __popc(bal & ((1u << lane) - 1u))] = static_cast<uint8_t>(lane + 32 * m);
      n += __popc(bal);
    }
    if (lane == 0) {
      row.n = n;
      row.raw = A.by_logits || hard || !alone;
    }
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += rows[w].n;
    for (int item = warp; item < total; item += kWarps) {
      int w = 0, r = item;
      while (r >= rows[w].n) r -= rows[w++].n;
      const int tu = block * kWarps + w, e = rows[w].cand[r];
      double v = dot_bf16_f32_fp64(A.x + static_cast<size_t>(tu) * A.d, A.w + static_cast<size_t>(e) * A.d, A.d, lane);
      if (!rows[w].raw)
        v = A.sigmoid ? ordered(1.0 / (1.0 + exp(-v)) + (A.bias ? static_cast<double>(A.bias[e]) : 0.0))
                      : exp(v - static_cast<double>(rows[w].shift));
      if (lane == 0) rows[w].v[e] = v;
    }
    __syncthreads();
    refined |= open;
  };

  // ---- which groups stay ------------------------------------------------------
  uint32_t group_in = 0, group_open = 0;  // bit g, the same in every lane
  uint32_t open = 0;
  if (here && grouped && !hard) {
    __syncwarp();
    // 32 / lpg groups at least, lpg lanes to a group
    const int lpg = G <= 2 ? 16 : G <= 4 ? 8 : G <= 8 ? 4 : G <= 16 ? 2 : 1;
    const int g = lane / lpg;
    Top2 lo2, up2;
    if (g < G)
      for (int i = lane % lpg; i < gs; i += lpg) {
        const float c = row.c[g * gs + i], dv = row.d[g * gs + i];
        lo2.add(c - dv);
        up2.add(c + dv);
      }
    for (int o = 1; o < lpg; o <<= 1) {
      lo2.merge(o);
      up2.merge(o);
    }
    // a sum's own rounding, outward
    float lo = lo2.a, up = up2.a, cut = lo2.a;
    if (A.group_top == 2) {
      cut = lo2.b;
      lo = lo2.a + lo2.b - 1.2e-7f * (fabsf(lo2.a) + fabsf(lo2.b));
      up = up2.a + up2.b + 1.2e-7f * (fabsf(up2.a) + fabsf(up2.b));
      if (lo != lo) lo = -INFINITY;  // -inf - (-inf): an empty group's
      if (up != up) up = -INFINITY;
    }
    int may = 0, sure = 0;  // groups that may, that certainly do, come before this one
    for (int h = 0; h < G; ++h) {
      const float ol = __shfl_sync(0xffffffffu, lo, h * lpg), ou = __shfl_sync(0xffffffffu, up, h * lpg);
      if (h != g) {
        may += ou >= lo;
        sure += ol > up;
      }
    }
    for (int h = 0; h < G; ++h) {
      const int m = __shfl_sync(0xffffffffu, may, h * lpg), u = __shfl_sync(0xffffffffu, sure, h * lpg);
      if (m < A.kept) group_in |= 1u << h;
      else if (u < A.kept) group_open |= 1u << h;
    }
    if (group_open) {
      if (!alone) {
        hard = true;
      } else {
#pragma unroll
        for (int m = 0; m < P; ++m) {
          const int e = lane + 32 * m, ge = min(e / gs, G - 1);
          const float gc = __shfl_sync(0xffffffffu, cut, ge * lpg);
          if (e < E && ((group_open >> ge) & 1u) && C[m] + D[m] >= gc) open |= 1u << m;
        }
      }
    }
  }
  if (!here) hard = false;
  bool listed = hard && A.list;
  if (hard) open = listed ? 0 : in_range;
  refine(open);
  if (here && group_open && !hard) {
    // the open groups by their fp64 scores: d = -1 marks the experts refined,
    // among which each open group's best are
    __syncwarp();
#pragma unroll
    for (int m = 0; m < P; ++m)
      if ((refined >> m) & 1u) row.d[lane + 32 * m] = -1.f;
    __syncwarp();
    double gv = -INFINITY;
    if (lane < G && ((group_open >> lane) & 1u)) {
      double a = -INFINITY, b = -INFINITY;
#pragma unroll 1
      for (int i = 0; i < gs; ++i) {
        const int e = lane * gs + i;
        if (row.d[e] < 0.f) {
          const double v = ordered(row.v[e]);
          if (v > a) { b = a; a = v; } else if (v > b) { b = v; }
        }
      }
      gv = ordered(A.group_top == 2 ? a + b : a);
    }
    int ahead = 0;
    for (int h = 0; h < G; ++h) {
      const double o = __shfl_sync(0xffffffffu, gv, h);
      ahead += ((group_open >> h) & 1u) && before(o, h, gv, lane);
    }
    const int room = A.kept - __popc(group_in);
    group_in |= __ballot_sync(0xffffffffu, lane < G && ((group_open >> lane) & 1u) && ahead < room);
  }

  // ---- the picks -----------------------------------------------------------------
  uint32_t allowed = in_range;
  int mine = 0, extra = 0;  // lane j < k: pick j; experts left out that may come in
  bool again = false;
  open = 0;
  if (here && !hard) {
    if (grouped) {
#pragma unroll
      for (int m = 0; m < P; ++m)
        if (!((group_in >> min((lane + 32 * m) / gs, 31)) & 1u)) allowed &= ~(1u << m);
    }
    uint32_t left = allowed, key[P];
#pragma unroll
    for (int m = 0; m < P; ++m) key[m] = order_key(C[m]);
    for (int j = 0; j < k; ++j) {
      uint32_t bk = 0;
      int be = 0x7fffffff;
#pragma unroll
      for (int m = 0; m < P; ++m)
        if (((left >> m) & 1u) && key[m] > bk) {  // the lane's lowest expert on equal keys
          bk = key[m];
          be = lane + 32 * m;
        }
      const uint32_t top = __reduce_max_sync(0xffffffffu, bk);
      const int e = __reduce_min_sync(0xffffffffu, bk == top ? be : 0x7fffffff);
      if ((e & 31) == lane) left &= ~(1u << (e >> 5));
      if (lane == j) mine = e;
    }
    // Settled when each pick's interval lies above the next one's, and the
    // last pick's above those of the experts left out.
    float dv = 0.f;
#pragma unroll
    for (int m = 0; m < P; ++m) {
      const float o = __shfl_sync(0xffffffffu, D[m], mine & 31);
      if ((mine >> 5) == m) dv = o;
    }
    const float lo = lane < k ? row.c[mine] - dv : INFINITY, up = lane < k ? row.c[mine] + dv : -INFINITY;
    const float lo_prev = __shfl_up_sync(0xffffffffu, lo, 1);
    float hi = -INFINITY;
    bool out = false;
#pragma unroll
    for (int m = 0; m < P; ++m)
      if ((left >> m) & 1u) {
        hi = fmaxf(hi, C[m] + D[m]);
        out = true;
      }
    const float lo_last = __shfl_sync(0xffffffffu, lo, k - 1);
    again = __any_sync(0xffffffffu, (out && hi >= lo_last) || (lane > 0 && lane < k && !(lo_prev > up)));
    if (again && !alone) {
      listed = A.list;
      open = listed ? 0 : in_range;
    } else if (again) {
      float lo_min = lo;
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        lo_min = fminf(lo_min, __shfl_xor_sync(0xffffffffu, lo_min, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      }
      // open: picks whose intervals meet another pick's or an expert's left out, and those experts
      const bool any_out = __any_sync(0xffffffffu, out);
      bool mark = lane < k && any_out && lo <= hi;
      for (int i = 0; i < k; ++i) {
        const float ol = __shfl_sync(0xffffffffu, lo, i), ou = __shfl_sync(0xffffffffu, up, i);
        if (lane < k && i != lane) mark |= ol <= up && lo <= ou;
      }
      unsigned marks = __ballot_sync(0xffffffffu, mark);
      while (marks) {
        const int e = __shfl_sync(0xffffffffu, mine, __ffs(marks) - 1);
        marks &= marks - 1;
        if ((e & 31) == lane) open |= 1u << (e >> 5);
      }
      uint32_t in = 0;
#pragma unroll
      for (int m = 0; m < P; ++m)
        if (((left >> m) & 1u) && C[m] + D[m] >= lo_min) in |= 1u << m;
      open |= in;
      extra = in;
    }
  }
  refine(open);
  if (!here) return;
  if (listed) {
    // (the order of the list changes from run to run; nothing depends on it)
    if (lane == 0) A.list[1 + atomicAdd(A.list, 1)] = t;
    return;
  }
  __syncwarp();
  double s64 = 0.0;
  const bool whole = hard || (again && !alone);
  if (whole) {
    mine = pick_whole<P>(A, row, lane, s64);
  } else if (again) {
    // candidates, one to a lane: the picks, then the experts that may come in
    // (more of them than lanes: from shared memory); values fp64 where
    // refined, else the fp32 ones, whose intervals meet no other's
    int n = 0;
#pragma unroll
    for (int m = 0; m < P; ++m) {
      const unsigned bal = __ballot_sync(0xffffffffu, (extra >> m) & 1u);
      if ((extra >> m) & 1u) row.cand[n + __popc(bal & ((1u << lane) - 1u))] = static_cast<uint8_t>(lane + 32 * m);
      n += __popc(bal);
    }
    __syncwarp();
    n += k;
    if (n <= 32) {
      const int e = lane < k ? mine : lane < n ? row.cand[lane - k] : 0;
      bool fp64 = false;
#pragma unroll
      for (int m = 0; m < P; ++m) {
        const uint32_t o = __shfl_sync(0xffffffffu, refined, e & 31);
        if ((e >> 5) == m) fp64 = (o >> m) & 1u;
      }
      const double v = lane >= n ? -INFINITY : fp64 ? ordered(row.v[e]) : static_cast<double>(row.c[e]);
      int rank = 0;
      for (int i = 0; i < n; ++i) {
        const double ov = __shfl_sync(0xffffffffu, v, i);
        const int oe = __shfl_sync(0xffffffffu, e, i);
        rank += before(ov, oe, v, e);
      }
      for (int j = 0; j < k; ++j) {
        const unsigned at = __ballot_sync(0xffffffffu, lane < n && rank == j);
        const int pe = __shfl_sync(0xffffffffu, e, __ffs(at) - 1);
        if (lane == j) mine = pe;
      }
    } else {
#pragma unroll
      for (int m = 0; m < P; ++m) {
        const int e = lane + 32 * m;
        if (e < E) row.v[e] = (refined >> m) & 1u ? ordered(row.v[e]) : static_cast<double>(C[m]);
      }
      __syncwarp();
      mine = pick_slow<P>(row.v, allowed, k, lane);
    }
  }

  // ---- weights: lane j < k holds pick j ----------------------------------------------
  float wt;
  if (whole) {
    wt = weight64(A, s64, lane);
  } else {
    const float l = row.l[mine];
    float top = 0.f;
    if (A.renorm) {
      top = lane < k ? l : -INFINITY;
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    if ((A.sigmoid ? top : top - row_max) < kFarScores && A.renorm) {
      // scores that leave fp64's range, or nearly: as a row evaluated in fp64 has them
      wt = weight64(A, A.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(l)))
                                 : exp(static_cast<double>(l) - row_max) / row_sum, lane);
    } else {
      float s;
      if (!A.sigmoid) {
        s = expf(l - (A.renorm ? top : row_max));
      } else if (A.renorm && top < -8.f) {
        // all scores times e^-top: those that would leave fp32's range keep their ratio to the largest
        s = expf(l - top) / (1.0f + expf(l));
      } else {  // (sigmoid(l) = e^l (1 + tiny) below -60, and e^-l soon overflows)
        s = l < -60.f ? expf(l) : 1.0f / (1.0f + expf(-l));
      }
      if (A.renorm) {
        float sum = lane < k ? s : 0.f;
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        s /= sum;
      } else if (!A.sigmoid) {
        s /= row_sum;
      }
      wt = s * A.scale;
    }
  }
  if (lane < k) {
    A.out_idx[static_cast<size_t>(t) * k + lane] = mine;
    A.out_w[static_cast<size_t>(t) * k + lane] = wt;
  }
}

template <int P>
__global__ void __launch_bounds__(kThreads, 3) k_route_scored(const __grid_constant__ Scored A) {
  __shared__ Row<P> rows[kWarps];
  pdl_wait();
  pdl_trigger();
  select_block<P>(A, rows, blockIdx.x, [&](int t, float (&L)[P], float (&D)[P]) {
    const int lane = threadIdx.x & 31, T = A.T, E = A.E;
    float xq = 0.f;
#pragma unroll
    for (int m = 0; m < P; ++m) L[m] = 0.f;
#pragma unroll 4
    for (int s = 0; s < A.lg.splits; ++s) {
      xq += A.lg.xsq[static_cast<size_t>(s) * T + t];
      const float* pl = A.lg.partial + (static_cast<size_t>(s) * T + t) * E + lane;
#pragma unroll
      for (int m = 0; m < P; ++m)
        if (lane + 32 * m < E) L[m] += pl[32 * m];
    }
    // What the squares lost below fp32's range: at most 2^-150 each, so d 2^-149
    // (the subnormal with the bits of d) covers a row of them.
    const float lost = __uint_as_float(static_cast<uint32_t>(A.d));
    const float xn = sqrt_approx(xq + lost);
#pragma unroll
    for (int m = 0; m < P; ++m) {
      const float wn = sqrt_approx(lane + 32 * m < E ? A.lg.wsq[lane + 32 * m] + lost : 0.f);
      D[m] = A.lg.gamma * xn * wn * (1.0f + 0.00390625f) + 1.2e-7f * fabsf(L[m]) + 7e-36f * (xn + wn) + 1e-30f;
    }
  });
}

// Tokens whose choice a softmax's denominator leaves open: fp64 logits of all
// their experts, as a product of tiles (a weight row read by one token at a
// time would cost 4 E d bytes a token: 4 MB and 40 us a CTA at 256 experts,
// d = 4096).  Tile: 32 listed tokens x 64 experts over a slice of d; 64 threads
// of 8 x 4 sums share a chunk of 32 with three more such groups, each with a
// quarter of its k (at 4 x 2 sums a thread, where loads from shared memory
// took five times as long as the products, 132 us in place of 55 for 330
// tokens, 256 experts, d = 4096: 12.6 TFLOP/s in fp64, short of the pipe's by
// the conversions; tokens kept as fp64 in shared memory or chunks loaded two
// ahead changed little, 4 x 4 sums took 66 us).  Few tokens: d is cut into slices
// while SMs are idle and there is room.  Slices' and groups' sums are added in
// order.
constexpr int kRT = 32, kRE = 64, kRK = 32;

struct Slices {
  int count, tiles_t, tiles_e, slices, per;  // per: chunks of kRK
};
__device__ __forceinline__ Slices slices_of(const int32_t* list, size_t room, int T, int E, int d) {
  Slices S;
  S.count = min(list[0], T);
  S.tiles_t = (S.count + kRT - 1) / kRT;
  S.tiles_e = (E + kRE - 1) / kRE;
  const int chunks = d / kRK, tiles = max(1, S.tiles_t * S.tiles_e);
  const size_t fit = room / (static_cast<size_t>(max(S.count, 1)) * E * 8);
  const int want = static_cast<int>(min(fit, static_cast<size_t>(min(max(1, 296 / tiles), 16))));
  S.per = (chunks + min(want, chunks) - 1) / min(want, chunks);
  S.slices = (chunks + S.per - 1) / S.per;
  return S;
}

__global__ void __launch_bounds__(256, 2) k_route_rows64(const __nv_bfloat16* __restrict__ x, const float* __restrict__ w,
                                                      const int32_t* list, size_t room, int T, int E, int d,
                                                      double* out) {
  __shared__ __align__(16) float xs[kRK][kRT], ws[kRK][kRE];
  __shared__ double red[32 * 64];  // a group's sums
  pdl_wait();
  pdl_trigger();
  const Slices S = slices_of(list, room, T, E, d);
  const int tid = threadIdx.x, chunks = d / kRK;
  const int group = tid >> 6, tx = (tid & 3) * 8, te = ((tid & 63) >> 2) * 4;  // the thread's k, tokens, experts
  const int units = S.tiles_t * S.tiles_e * S.slices;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const int sl = u % S.slices, tile = u / S.slices;
    const int i0 = tile / S.tiles_e * kRT, e0 = tile % S.tiles_e * kRE;
    const int c0 = sl * S.per, c1 = min(chunks, c0 + S.per);
    // loads: 8 elements of a token (threads below 128), two pieces of 4 of an expert
    const int lt = tid & 31, lk = (tid >> 5) * 8;
    const bool has_x = tid < 128 && i0 + lt < S.count;
    const __nv_bfloat16* xp = x + (has_x ? static_cast<size_t>(min(max(list[1 + i0 + lt], 0), T - 1)) * d + lk : 0);
    const int le = tid & 63, lj = (tid >> 6) * 4;
    const bool has_w = e0 + le < E;
    const float* wp = w + (has_w ? static_cast<size_t>(e0 + le) * d + lj : 0);
    uint4 xv = make_uint4(0, 0, 0, 0);
    float4 w0 = make_float4(0, 0, 0, 0), w1 = w0;
    auto load = [&](int c) {
      if (has_x) xv = *reinterpret_cast<const uint4*>(xp + c * kRK);
      if (has_w) {
        w0 = *reinterpret_cast<const float4*>(wp + c * kRK);
        w1 = *reinterpret_cast<const float4*>(wp + c * kRK + 16);
      }
    };
    double a[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) a[i][j] = 0.0;
    load(c0);
    for (int c = c0; c < c1; ++c) {
      __syncthreads();  // the chunk before has been read
      if (tid < 128) {
        const uint32_t q[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          xs[lk + 2 * j][lt] = __uint_as_float(q[j] << 16);
          xs[lk + 2 * j + 1][lt] = __uint_as_float(q[j] & 0xFFFF0000u);
        }
      }
      ws[lj][le] = w0.x; ws[lj + 1][le] = w0.y; ws[lj + 2][le] = w0.z; ws[lj + 3][le] = w0.w;
      ws[lj + 16][le] = w1.x; ws[lj + 17][le] = w1.y; ws[lj + 18][le] = w1.z; ws[lj + 19][le] = w1.w;
      __syncthreads();
      if (c + 1 < c1) load(c + 1);
#pragma unroll 2
      for (int k = group * (kRK / 4); k < (group + 1) * (kRK / 4); ++k) {
        const float4 p = *reinterpret_cast<const float4*>(&xs[k][tx]), q = *reinterpret_cast<const float4*>(&xs[k][tx + 4]);
        const float4 v = *reinterpret_cast<const float4*>(&ws[k][te]);
        const double xk[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w}, wk[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) a[i][j] = fma(xk[i], wk[j], a[i][j]);
      }
    }
    for (int g = 1; g < 4; ++g) {
      __syncthreads();
      if (group == g)
#pragma unroll
        for (int r = 0; r < 32; ++r) red[r * 64 + (tid & 63)] = a[r >> 2][r & 3];
      __syncthreads();
      if (group == 0)
#pragma unroll
        for (int r = 0; r < 32; ++r) a[r >> 2][r & 3] += red[r * 64 + tid];
    }
    if (group == 0)
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i0 + tx + i < S.count && e0 + te + j < E)
            out[(static_cast<size_t>(sl) * S.count + i0 + tx + i) * E + e0 + te + j] = a[i][j];
  }
}

// Picks and weights of the listed tokens, a warp to each.
template <int P>
__global__ void __launch_bounds__(kThreads) k_route_whole(const __grid_constant__ Scored A) {
  __shared__ Row<P> rows[kWarps];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Slices S = slices_of(A.list, A.lg.room, A.T, A.E, A.d);
  for (int i = blockIdx.x * kWarps + warp; i < S.count; i += gridDim.x * kWarps) {
    const size_t t = min(max(A.list[1 + i], 0), A.T - 1);
    double v[P];
#pragma unroll
    for (int m = 0; m < P; ++m) v[m] = 0.0;
#pragma unroll (P == 8 ? 4 : 8)
    for (int s = 0; s < S.slices; ++s) {
      const double* r = A.lg.rows64 + (static_cast<size_t>(s) * S.count + i) * A.E + lane;
#pragma unroll
      for (int m = 0; m < P; ++m)
        if (lane + 32 * m < A.E) v[m] += r[32 * m];
    }
#pragma unroll
    for (int m = 0; m < P; ++m) rows[warp].v[lane + 32 * m] = v[m];
    __syncwarp();
    double s = 0.0;
    const int mine = pick_whole<P>(A, rows[warp], lane, s);
    const float wt = weight64(A, s, lane);
    if (lane < A.k) {
      A.out_idx[t * A.k + lane] = mine;
      A.out_w[t * A.k + lane] = wt;
    }
    __syncwarp();
  }
}

// The smallest batches: logits and selection in one launch of a thread-block
// cluster.  A CTA sums one slice of d for all T E logits (fp32 FMA chains of
// the products and of their magnitudes, cluster_partial_dots_f32) into CTA 0,
// which selects:  |L - l| <= 2 cluster_gamma(d) (sum of magnitudes)(1 + 2^-8).
// Taken up to 128 logits, where it is the faster (us in a graph, this kernel
// against the tensor-core logits and k_route_scored): 64 experts, d = 2048: 1
// token 7.0 / 13.8, 2 tokens 10.1 / 12.7, 4 tokens 16.3 / 16.3, 8 tokens 28.3 /
// 16.3; 128 experts, d = 4096: 1 token 13.0 / 20.5, 2 tokens 21.2 / 15.4.
constexpr int kTinyLogits = 128;

template <int P>
__global__ void __launch_bounds__(kThreads) k_route_scored_tiny(const __grid_constant__ Scored A) {
  __shared__ Row<P> rows[kWarps];
  __shared__ float2 part[kClusterSlices * kTinyLogits];
  cluster_sync_start();
  pdl_wait();
  pdl_trigger();
  const int rank = blockIdx.x;  // the grid is one cluster
  const int n = A.T * A.E, dk = A.d / kClusterSlices;
  cluster_partial_dots_f32(
      n, rank * dk, dk,
      [&](int i, const __nv_bfloat16*& xr, const float*& wr) {
        const int t = i / A.E;
        xr = A.x + static_cast<size_t>(t) * A.d;
        wr = A.w + static_cast<size_t>(i - t * A.E) * A.d;
      },
      cluster_map_shared(part, 0) + 8u * static_cast<uint32_t>(rank * n));
  cluster_sync_publish();
  if (rank != 0) return;
  select_block<P>(A, rows, 0, [&](int t, float (&L)[P], float (&D)[P]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int m = 0; m < P; ++m) {
      float v = 0.f, mag = 0.f;
      if (lane + 32 * m < A.E) {
#pragma unroll
        for (int r = 0; r < kClusterSlices; ++r) {
          const float2 q = part[r * n + t * A.E + lane + 32 * m];
          v += q.x;
          mag += q.y;
        }
      }
      L[m] = v;
      D[m] = 2.0f * A.lg.gamma * mag * (1.0f + 0.00390625f) + 1e-30f;
    }
  });
}

bool tiny(int T, int d, int E) { return T <= kWarps && d % 64 == 0 && T * E <= kTinyLogits; }

}  // namespace
}  // namespace moeq

using namespace moeq;

extern "C" {

size_t moe_route_scored_workspace_bytes(int T, int d, int E) {
  if (T <= 0 || d <= 0 || E <= 0) return 256;
  return route_tc_workspace_bytes(T, d, E);
}

moe_status_t moe_route_scored(const void* x, const float* w_router, const float* bias, int T, int d, int E, int k,
                              int scoring, int n_groups, int topk_groups, int group_top, int renorm, double scale,
                              int32_t* topk_idx, float* topk_w, void* workspace, size_t workspace_bytes,
                              int32_t* status, moe_stream_t stream) {
  const char* fn = "moe_route_scored";
  moe_status_t st = route_check_args(x, w_router, T, d, E, k, topk_idx, topk_w, fn);
  if (st != MOE_OK) return st;
  if (d > 32768) {
    set_error("%s: d=%d exceeds 32768 (the logits' error bounds)", fn, d);
    return MOE_ERR_UNSUPPORTED_SHAPE;
  }
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
  if (!tiny(T, d, E)) st = launch_route_partials_tc(x, w_router, T, d, E, workspace, status, &A.lg, s);
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
  A.alone = A.sigmoid || !bias;
  A.scale = static_cast<float>(scale);
  A.out_idx = topk_idx;
  A.out_w = topk_w;
  if (tiny(T, d, E)) {
    A.lg.gamma = cluster_gamma(d);
    auto kern = E <= 32 ? k_route_scored_tiny<1> : E <= 64 ? k_route_scored_tiny<2> : k_route_scored_tiny<4>;
    return cuda_check(launch_cluster_pdl(kern, kClusterSlices, dim3(kThreads), 0, s, A), "moe_route_scored launch");
  }
  auto kern = E <= 32 ? k_route_scored<1> : E <= 64 ? k_route_scored<2> : E <= 128 ? k_route_scored<4> : k_route_scored<8>;
  if (!A.alone) A.list = A.lg.list;
  const bool pdl = pdl_for(static_cast<long>(T) * k);
  st = cuda_check(launch_pdl(pdl, kern, dim3(ceil_div(T, kWarps)), dim3(kThreads), 0, s, A), "moe_route_scored launch");
  if (st != MOE_OK || A.alone) return st;
  st = cuda_check(launch_pdl(true, k_route_rows64, dim3(std::min<long>(296, ceil_div(T, kRT) * 16L * ceil_div(E, kRE))),
                             dim3(256), 0, s, A.x, A.w, static_cast<const int32_t*>(A.list), A.lg.room, T, E, d,
                             A.lg.rows64),
                  "moe_route_scored fp64 launch");
  if (st != MOE_OK) return st;
  auto fin = E <= 32 ? k_route_whole<1> : E <= 64 ? k_route_whole<2> : E <= 128 ? k_route_whole<4> : k_route_whole<8>;
  return cuda_check(launch_pdl(true, fin, dim3(std::min(296, ceil_div(T, kWarps))), dim3(kThreads), 0, s, A),
                    "moe_route_scored selection launch");
}

}  // extern "C"
