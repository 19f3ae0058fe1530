// Grouped routing from fp32 logits and its gradient: softmax or sigmoid
// scores, a bias that acts on the selection alone, groups of experts, top-k,
// renormalised and scaled weights, and the balance statistics.
//
// Per token, with logits l (a logit that is not finite masks its expert):
//   s_e = softmax(l)_e or 1 / (1 + exp(-l_e));  c_e = s_e + b_e, -inf if masked
//   group value = sum of the group's g largest c; the best groups are kept
//   idx = top-k of c over the kept groups, w_j = scale * s_j / sum_j s_j
//
// Forward: P lanes share one token (32 P >= E), lane p holding the 16-byte pieces
// p, p + P, ... of its row, 32 experts: a warp routes 32 / P tokens at once, and
// what is done once per token (merging the lanes' lists, the weights) is shared
// by many experts. Only values are kept in order, never pairs of value and
// index: a second look at the row finds the experts whose values made it.
// Gradient: L lanes share a token and hold 16 experts each, in the same way.
//
// The choice is that of the formulas in 64 bits, exponentials to 2^-44. Scores
// are computed in fp32, and wherever two values that a decision compares are
// closer than the fp32 error allows, the token is decided again with more bits,
// which only those tokens pay for. Values that are equal are always decided
// there, so ties need no care elsewhere.
#include <math_constants.h>

#include "moe_internal.h"
#include "moe_ptx.cuh"

namespace moe {

namespace {

constexpr int kV = 16;         // experts per lane, gradient
constexpr int kWarps = 4;      // gradient
constexpr int kThreads = 32 * kWarps;
constexpr int kStatsWarps = 8;
constexpr int kStatsThreads = 32 * kStatsWarps;
static_assert(kStatsThreads >= kMaxExperts, "a thread per expert sums the balance loss");
constexpr int kFwdWarps = 4;
constexpr int kFwdThreads = 32 * kFwdWarps;
constexpr unsigned kFull = 0xffffffffu;
constexpr float kLowest = 3.402823466e38f;  // -kLowest: fp32's lowest value

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;
// Where a row's largest logit is below this, 1 + exp(l) is 1 to fp32 and far beyond
// for all of it, and shifting the row leaves the shares s / sum s of its sigmoid scores
// as they are: the gradient shifts it up to here, and they hold where the scores
// themselves are below fp32's smallest value.
constexpr float kLowRow = -41.f;
// The forward's rows that fp32 does not hold: their scores are below 1e-30, or they
// are no higher than what stands past E. They are decided again, and counted in P there.
__device__ __forceinline__ bool tiny_row(float m, bool softmax) { return m < (softmax ? -1e38f : -69.f); }

template <int L, class T, class Op>
__device__ __forceinline__ T lanes_reduce(T v, Op op) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  return lanes_reduce<L>(v, [](float a, float b) { return a + b; });
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
  if constexpr (L == 32) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
  }
  return lanes_reduce<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ bool masked(float l) { return !(fabsf(l) < CUDART_INF_F); }

// -------------------------------------------------- close decisions ----
// Order of fp64 values as integers (fp64 instructions take a warp 64 clocks each
// here). Its own inverse.
__device__ __forceinline__ long long order64(double v) {
  const long long b = __double_as_longlong(v);
  return b ^ ((b >> 63) & 0x7fffffffffffffffll);
}

// The k chosen experts in pick[] (shared memory) to outputs; lanes sub, sub + L,
// ... of the token take slots sub, sub + L, ...; logits from `row`; softmax
// scores are exp(l - m) iz.
template <int L>
__device__ __forceinline__ void write_slots(const GroupedArgs& a, int64_t t, const int* pick,
                                            const float* row, float m, float iz, int sub, bool write,
                                            int* cnt) {
  constexpr int kPer = (kMaxTopK + L - 1) / L;
  constexpr int kLanes = L < kMaxTopK ? L : kMaxTopK;  // lanes that hold slots
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  int e[kPer];
  float x[kPer], w[kPer];
  float top = -CUDART_INF_F;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int j = sub + q * L;
    const bool in = j < a.k;
    e[q] = in ? pick[j] : 0;
    x[q] = in ? row[e[q]] : -CUDART_INF_F;
    if (masked(x[q])) x[q] = -CUDART_INF_F;
    top = fmaxf(top, x[q]);
  }
  float f = a.scale;
  if (a.renormalize) {
    // Weights are ratios then, and scores, which could underflow, are taken relative
    // to the largest chosen logit: softmax scores, and sigmoid scores where that is
    // below zero, as exp(l - top) / (1 + exp(l)).
    top = lanes_reduce<kLanes>(top, [](float u, float v) { return fmaxf(u, v); });
    const bool ratio = softmax || top < 0.f;
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      float y = exp2_approx((ratio ? x[q] - top : -x[q]) * kLog2e);
      if (!softmax) y = (ratio ? y : 1.f) * rcp_approx(1.f + (ratio ? exp2_approx(x[q] * kLog2e) : y));
      w[q] = x[q] == -CUDART_INF_F ? 0.f : y;
      sum += w[q];
    }
    sum = lanes_sum<kLanes>(sum);
    f = sum > 0.f ? f * rcp_approx(sum) : 0.f;
  } else {
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const float y = softmax ? exp2_approx((x[q] - m) * kLog2e) * iz
                              : rcp_approx(1.f + exp2_approx(-x[q] * kLog2e));
      w[q] = x[q] == -CUDART_INF_F ? 0.f : y;
    }
  }
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int j = sub + q * L;
    if (write && j < a.k) {
      a.topk_idx[t * a.k + j] = e[q];
      a.topk_w[t * a.k + j] = w[q] * f;
      if (cnt != nullptr) atomicAdd(&cnt[e[q]], 1);
    }
  }
}

struct ExactScratch {     // shared memory of one warp
  long long* val;         // [kMaxExperts]: ordered fp64 values of the listed experts
  float* x;               // [kMaxExperts]: logits, -inf where masked
  float* c;               // [kMaxExperts]: selection values in fp32
  uint8_t* list;          // [kMaxExperts]: experts to evaluate
  int* pick;              // [kMaxTopK]
};

// Values as an unevaluated sum of two fp32 (Dekker, Knuth): 48 bits of fp32
// instructions, each of which takes a sixteenth of an fp64 one's time.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {  // exact
  const float s = __fadd_rn(a, b), v = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, v)), __fsub_rn(b, v))};
}
__device__ __forceinline__ Two ordered_sum(float a, float b) {  // exact for |a| >= |b|
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Two add(Two a, Two b) {
  const Two s = two_sum(a.hi, b.hi);
  return ordered_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
// a / b: a quotient of fp32 and one more for what it leaves.
__device__ __forceinline__ Two divide(Two a, Two b) {
  const float y = rcp_approx(b.hi), q = __fmul_rn(a.hi, y), p = __fmul_rn(q, b.hi);
  const float left = __fsub_rn(a.hi, p) - __fmaf_rn(q, b.hi, -p) + __fmaf_rn(-q, b.lo, a.lo);
  return ordered_sum(q, __fmul_rn(left, y));
}
__device__ __forceinline__ Two lanes_sum(Two v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = add(v, Two{__shfl_xor_sync(kFull, v.hi, o), __shfl_xor_sync(kFull, v.lo, o)});
  return v;
}
// 2^n of n in -126 .. 127
__device__ __forceinline__ float power2(int n) { return __int_as_float((n + 127) << 23); }

// exp(x) 2^-n to 45 bits: x = n ln 2 + r with |r| <= ln 2 / 2 (the reduction of Cody
// and Waite), and the Taylor series of exp(r) to r^13 / 13! (the next term is below
// 2^-57), its terms from r^7 on (below 2^-22) in plain fp32. x is held to 750 either
// way, past where fp64's exp is 0 or infinite.
__device__ __forceinline__ Two exp_parts(Two x, int& n) {
  if (!(fabsf(x.hi) < 750.f)) x = {copysignf(750.f, x.hi), 0.f};
  const float nf = rintf(x.hi * kLog2e);
  n = static_cast<int>(nf);
  // ln 2 in three parts; products of the first, of 12 bits, with n are exact
  Two r = two_sum(x.hi, __fmul_rn(nf, -0x1.62ep-1f));
  float tail = r.lo;
  r = two_sum(r.hi, x.lo);
  tail += r.lo;
  constexpr float kLn2b = 0x1.0bfbe8p-15f, kLn2c = 0x1.cf79acp-40f;
  const float p = __fmul_rn(nf, -kLn2b);
  tail += __fmaf_rn(nf, -kLn2c, __fmaf_rn(nf, -kLn2b, -p));
  r = two_sum(r.hi, p);
  r = ordered_sum(r.hi, tail + r.lo);
  float y = 1.f / 6227020800.f;
  y = fmaf(y, r.hi, 1.f / 479001600.f);
  y = fmaf(y, r.hi, 1.f / 39916800.f);
  y = fmaf(y, r.hi, 1.f / 3628800.f);
  y = fmaf(y, r.hi, 1.f / 362880.f);
  y = fmaf(y, r.hi, 1.f / 40320.f);
  y = fmaf(y, r.hi, 1.f / 5040.f);
  Two v{y, 0.f};
  auto step = [&](double c) {  // v = v r + c, c above |v r|
    const float ch = static_cast<float>(c), cl = static_cast<float>(c - static_cast<double>(ch));
    const float q = __fmul_rn(v.hi, r.hi);
    float e = __fmaf_rn(v.hi, r.hi, -q);
    e = __fmaf_rn(v.lo, r.hi, __fmaf_rn(v.hi, r.lo, e)) + cl;
    const Two s = ordered_sum(ch, q);
    v = ordered_sum(s.hi, s.lo + e);
  };
  step(1.0 / 720.0);
  step(1.0 / 120.0);
  step(1.0 / 24.0);
  step(1.0 / 6.0);
  step(0.5);
  step(1.0);
  step(1.0);
  return v;
}

// The score as fp64: exp(x - m) / z, or the sigmoid of x. The latter's last two
// steps are fp64's own: scores next to 1 are equal, or not, as they round there. 2^n
// comes in two factors, so that next to fp64's limits the result is rounded once, to
// the bits that are left, to 0 or to infinity.
__device__ __noinline__ double score64(float x, float m, bool softmax, Two z) {
  int n;
  Two v = exp_parts(softmax ? two_sum(x, -m) : Two{-x, 0.f}, n);
  if (softmax) v = divide(v, z);
  const int half = n >> 1;
  const double y = (static_cast<double>(v.hi) + static_cast<double>(v.lo)) *
                   __longlong_as_double(static_cast<long long>(half + 1023) << 52) *
                   __longlong_as_double(static_cast<long long>(n - half + 1023) << 52);
  return softmax ? y : 1.0 / (1.0 + y);
}

// Only experts that may matter are evaluated so: those whose fp32 value is
// within `slack` of the group_top-th of their group, then those within it of a
// lower bound of the kept groups' k-th. All others rank below them whatever the
// error. (A softmax with a bias needs its sum so too, hence all exponentials.)
// Few tokens come here, on any SM, and the last of them holds up the launch, so
// loads are made at once and loops kept short.
// known: the kept groups where they are not in doubt, else 0; kth: with them
// known, the k-th largest value found in fp32. bias: in shared memory. share: the
// warp's sums of the shares of rows that fp32 does not hold, or nullptr.
__device__ __noinline__ void route_exact(const GroupedArgs& a, int t, uint32_t known, float kth,
                                         const float* bias, const ExactScratch& sc, int* cnt, float* share) {
  constexpr int kPer = kMaxExperts / 32;  // lane l: experts l, l + 32, ...
  const int lane = threadIdx.x & 31;
  const int E = a.E, S = a.E / a.n_groups;
  const uint32_t inv = a.n_groups > 1 ? 65536u / static_cast<uint32_t>(S) + 1u : 0u;  // e / S = e inv >> 16, e < 256
  const float* row = a.logits + static_cast<int64_t>(t) * E;
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  const bool all = softmax && a.bias != nullptr;
  const long long kInf = order64(-CUDART_INF);
  float m = -CUDART_INF_F, smax = 0.f, z = 0.f, big = 0.f;
  float x[kPer], c[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) x[i] = lane + 32 * i < E ? row[lane + 32 * i] : -CUDART_INF_F;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (masked(x[i])) x[i] = -CUDART_INF_F;
    m = fmaxf(m, x[i]);
    sc.x[lane + 32 * i] = x[i];
  }
  m = lanes_max<32>(m);
  if (m == -CUDART_INF_F) m = 0.f;  // nothing unmasked
  Two zz{0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (32 * i < E) {  // the scores, 0 where masked
      const float y = exp2_approx((softmax ? x[i] - m : -x[i]) * kLog2e);
      c[i] = softmax ? y : rcp_approx(1.f + y);
      z += c[i];
      smax = fmaxf(smax, c[i]);
    }
  if (all) {
#pragma unroll 1
    for (int e = lane; e < E; e += 32) {
      const float l = sc.x[e];
      int n;
      const Two v = exp_parts(two_sum(l, -m), n);
      const float f = l == -CUDART_INF_F ? 0.f : power2(max(n, -120));
      zz = add(zz, Two{v.hi * f, v.lo * f});
    }
    zz = lanes_sum(zz);
  } else {
    zz.hi = 1.f;  // softmax scores are compared as exp(l - m) where nothing is added to them
  }
  z = lanes_sum<32>(z);
  smax = lanes_max<32>(smax);
  const float iz = softmax && z > 0.f ? rcp_approx(z) : 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (32 * i < E) {
      const int e = lane + 32 * i;
      const float b = e < E ? bias[e] : 0.f;
      c[i] = x[i] == -CUDART_INF_F ? x[i] : fmaf(c[i], softmax ? iz : 1.f, b);
      if (x[i] != -CUDART_INF_F) big = fmaxf(big, fabsf(c[i]));
      if (known == 0u) sc.c[e] = c[i];
    }
  smax = softmax ? smax * iz : smax;
  big = fmaxf(lanes_max<32>(big), smax);
  // fp32 errors are within 2^-18 of the largest value (2^-14 where the logits are
  // so low that exp's argument is what errs)
  float slack = big * (softmax || smax > 1e-3f ? 0x1p-17f : 0x1p-13f);
  if (tiny_row(m, softmax)) {
    slack = CUDART_INF_F;  // fp32 holds the scores as 0, or nearly so
    if (share != nullptr) {
      z = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) z += exp2_approx((x[i] - m) * kLog2e);
      z = rcp_approx(lanes_sum<32>(z));
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (lane + 32 * i < E) share[lane + 32 * i] += exp2_approx((x[i] - m) * kLog2e) * z;
    }
  }
  __syncwarp();
  uint32_t kept = a.n_groups > 1 ? known : 1u;
  int n = 0;
  // phase 0 settles the groups, phase 1 the experts
#pragma unroll 1
  for (int phase = kept == 0u ? 0 : 1; phase < 2; ++phase) {
    float bound = -CUDART_INF_F;  // phase 0, lane g: of group g
    if (phase == 0) {
      if (lane < a.n_groups) {
        float v1 = -CUDART_INF_F, v2 = -CUDART_INF_F;
#pragma unroll 4
        for (int q = 0; q < S; ++q) {
          const float v = sc.c[lane * S + q];
          v2 = fmaxf(v2, fminf(v, v1));
          v1 = fmaxf(v1, v);
        }
        bound = a.group_top == 2 ? v2 : v1;
      }
    } else if (known != 0u) {
      bound = kth;
    } else {
      // the k-th largest of the lanes' own maxima
      float own = -CUDART_INF_F;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint32_t g = (static_cast<uint32_t>(lane + 32 * i) * inv) >> 16;
        if (32 * i < E && ((kept >> (g & 31u)) & 1u)) own = fmaxf(own, c[i]);
      }
      for (int j = 0; j < a.k; ++j) {
        bound = lanes_max<32>(own);
        const unsigned who = __ballot_sync(kFull, own == bound);
        if (lane == __ffs(static_cast<int>(who)) - 1) own = -CUDART_INF_F;
      }
    }
    // the candidates
    uint32_t mine = 0u;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (32 * i < E) {
        const int e = lane + 32 * i;
        const uint32_t g = (static_cast<uint32_t>(e) * inv) >> 16;
        const float lim = phase == 0 ? __shfl_sync(kFull, bound, g) : bound;
        if (e < E && c[i] >= lim - slack && (phase == 0 || ((kept >> (g & 31u)) & 1u))) mine |= 1u << i;
      }
    n = 0;
    for (unsigned who; (who = __ballot_sync(kFull, mine != 0u)) != 0u; n += __popc(who)) {
      if (mine != 0u)
        sc.list[n + __popc(who & ((1u << lane) - 1u))] =
            static_cast<uint8_t>(lane + 32 * (__ffs(static_cast<int>(mine)) - 1));
      mine &= mine - 1u;
    }
    __syncwarp();
#pragma unroll 1
    for (int q = lane; q < n; q += 32) {
      const int e = sc.list[q];
      const float l = sc.x[e];
      double v = -CUDART_INF;
      if (l != -CUDART_INF_F) {
        v = score64(l, m, softmax, zz);
        if (a.bias != nullptr) v += static_cast<double>(bias[e]);
      }
      sc.val[q] = order64(v);
    }
    __syncwarp();
    if (phase == 0) {
      long long v1 = kInf, v2 = kInf;
#pragma unroll 4
      for (int q = 0; q < n; ++q)
        if (static_cast<int>((sc.list[q] * inv) >> 16) == lane) {
          const long long v = sc.val[q];
          v2 = max(v2, min(v, v1));
          v1 = max(v1, v);
        }
      if (lane < a.n_groups && a.group_top == 2)  // order64 is its own inverse
        v1 = order64(__longlong_as_double(order64(__longlong_as_double(v1))) +
                     __longlong_as_double(order64(__longlong_as_double(v2))));
      int ahead = 0;
#pragma unroll 4
      for (int h = 0; h < a.n_groups; ++h) {
        const long long o = __shfl_sync(kFull, v1, h);
        ahead += (o > v1 || (o == v1 && h < lane)) ? 1 : 0;
      }
      kept = __ballot_sync(kFull, lane < a.n_groups && ahead < a.topk_groups);
      __syncwarp();
    }
  }
  // the candidates' ranks, ties to the lower index
#pragma unroll 1
  for (int q = lane; q < n; q += 32) {
    const int e = sc.list[q];
    const long long v = sc.val[q];
    int rank = 0;
#pragma unroll 2
    for (int r = 0; r < n; ++r) {
      const long long o = sc.val[r];
      const int f = sc.list[r];
      rank += static_cast<int>(o > v) | (static_cast<int>(o == v) & static_cast<int>(f < e));
    }
    if (rank < a.k) sc.pick[rank] = e;
  }
  __syncwarp();
  write_slots<32>(a, t, sc.pick, sc.x, m, iz, lane, true, cnt);
  __syncwarp();
}

// ------------------------------------------------------------- kernel ----

// The lane's kV logits of row t, pieces of four: sub, sub + L, ...; `none` past E
// or T.
template <int L>
__device__ __forceinline__ void load_row(const float* __restrict__ logits, int64_t t, bool valid,
                                         int E, int sub, float none, float (&l)[kV]) {
  const float* row = logits + t * E;
  if ((E & 3) == 0) {
#pragma unroll
    for (int h = 0; h < kV / 4; ++h) {
      const int e = 4 * (sub + L * h);
      float4 v = make_float4(none, none, none, none);
      if (valid && e < E) v = __ldg(reinterpret_cast<const float4*>(row + e));
      l[4 * h] = v.x;
      l[4 * h + 1] = v.y;
      l[4 * h + 2] = v.z;
      l[4 * h + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int e = 4 * (sub + L * (i / 4)) + i % 4;
      l[i] = valid && e < E ? __ldg(row + e) : none;
    }
  }
}

// Experts of the lane that are masked, or past E (bits).
template <int L>
__device__ __forceinline__ uint32_t left_out(const float (&l)[kV], int E, int sub) {
  uint32_t mk = 0u;
#pragma unroll
  for (int i = 0; i < kV; ++i)
    if (masked(l[i]) || 4 * (sub + L * (i / 4)) + i % 4 >= E) mk |= 1u << i;
  return mk;
}

// The lane's softmax scores in pairs, exp(l - m) not yet divided by their sum over
// the row; 0 where masked and past E, where `l` holds the type's lowest value.
template <int L>
__device__ __forceinline__ void softmax_scores(float (&l)[kV], int E, int sub, uint64_t (&s)[kV / 2], float& m) {
  // a multiply-add per pair of logits finds whether one is not finite
  uint64_t chk = f32x2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kV; i += 2) chk = f32x2_fma(f32x2(l[i], l[i + 1]), f32x2(0.f, 0.f), chk);
  float c0, c1;
  f32x2_get(chk, c0, c1);
  uint32_t mk = 0u;
  if (__any_sync(kFull, !(c0 + c1 == 0.f))) {
    mk = left_out<L>(l, E, sub);
#pragma unroll
    for (int i = 0; i < kV; ++i)
      if ((mk >> i) & 1u) l[i] = -kLowest;
  }
  m = l[0];
#pragma unroll
  for (int i = 1; i + 1 < kV; i += 2) m = max3(m, l[i], l[i + 1]);
  m = fmaxf(m, l[kV - 1]);
  m = lanes_max<L>(m);
  if (__any_sync(kFull, m == -kLowest)) mk |= left_out<L>(l, E, sub);  // a row as low as what stands past E
  float x[kV];
#pragma unroll
  for (int i = 0; i < kV; i += 2)
    f32x2_get(f32x2_mul(f32x2_add(f32x2(l[i], l[i + 1]), f32x2(-m, -m)), f32x2(kLog2e, kLog2e)), x[i], x[i + 1]);
#pragma unroll
  for (int i = 0; i < kV; ++i) x[i] = exp2_approx(x[i]);
  if (mk != 0u) {
#pragma unroll
    for (int i = 0; i < kV; ++i)
      if ((mk >> i) & 1u) x[i] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < kV; i += 2) s[i / 2] = f32x2(x[i], x[i + 1]);
}

// The lane's sigmoid slopes s (1 - s) in pairs, from e = exp(-l) as e s s (of a score
// next to 1 the difference to 1 would be lost in s itself), and its sums of s and of
// s h. Past E, where h is 0, `l` holds kFar, whose score of 2^-121 is nothing beside
// the others' of logits above -60; `limit` tells by the sum of squares that all are
// within 60 of zero, or the careful way is taken: the clamp there changes nothing that
// counts beside the row's largest, which is at kLowRow or above.
constexpr float kFar = -84.f;
__device__ __forceinline__ float square_limit(int past) { return 3600.f + static_cast<float>(past) * (kFar * kFar); }
template <int L>
__device__ __forceinline__ void sigmoid_slopes(float (&l)[kV], const uint64_t (&h)[kV / 2], float limit, int E,
                                               int sub, uint64_t (&w)[kV / 2], float& sum, float& sum_h) {
  uint64_t sq = f32x2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kV; i += 2) sq = f32x2_fma(f32x2(l[i], l[i + 1]), f32x2(l[i], l[i + 1]), sq);
  float c0, c1;
  f32x2_get(sq, c0, c1);
  uint32_t mk = 0u;
  if (__any_sync(kFull, !(c0 + c1 < limit))) {
    mk = left_out<L>(l, E, sub);
    float m = -kLowest;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      if ((mk >> i) & 1u) l[i] = -kLowest;
      m = fmaxf(m, l[i]);
    }
    m = lanes_max<L>(m);
#pragma unroll
    for (int i = 0; i < kV; ++i) l[i] = fmaxf(m < kLowRow ? l[i] - m + kLowRow : l[i], kFar);
  }
  const uint64_t one = f32x2(1.f, 1.f);
  uint64_t z = f32x2(0.f, 0.f), zh = z;
#pragma unroll
  for (int i = 0; i < kV; i += 2) {
    float y0, y1;
    f32x2_get(f32x2_mul(f32x2(l[i], l[i + 1]), f32x2(-kLog2e, -kLog2e)), y0, y1);
    const uint64_t e = f32x2(exp2_approx(y0), exp2_approx(y1));
    f32x2_get(f32x2_add(e, one), y0, y1);
    uint64_t s = f32x2(rcp_approx(y0), rcp_approx(y1));
    if (mk != 0u) s = f32x2((mk >> i) & 1u ? 0.f : rcp_approx(y0), (mk >> (i + 1)) & 1u ? 0.f : rcp_approx(y1));
    z = f32x2_add(z, s);
    zh = f32x2_fma(s, h[i / 2], zh);
    w[i / 2] = f32x2_mul(f32x2_mul(e, s), s);
  }
  f32x2_get(z, c0, c1);
  sum = c0 + c1;
  f32x2_get(zh, c0, c1);
  sum_h = c0 + c1;
}
__device__ __forceinline__ float pairs_sum(const uint64_t (&s)[kV / 2]) {
  float a, b;
  uint64_t sum = s[0];
#pragma unroll
  for (int i = 1; i < kV / 2; ++i) sum = f32x2_add(sum, s[i]);
  f32x2_get(sum, a, b);
  return a + b;
}

// Descending order of the values of an array of registers.
__device__ __forceinline__ void order_pair(float& x, float& y) {
  const float hi = fmaxf(x, y);
  y = fminf(x, y);
  x = hi;
}
__device__ __forceinline__ void sort8(float (&k)[8]) {  // Batcher's odd-even merge sort
  auto o = [&](int x, int y) { order_pair(k[x], k[y]); };
  o(0, 1); o(2, 3); o(4, 5); o(6, 7);
  o(0, 2); o(1, 3); o(4, 6); o(5, 7);
  o(1, 2); o(5, 6);
  o(0, 4); o(1, 5); o(2, 6); o(3, 7);
  o(2, 4); o(3, 5);
  o(1, 2); o(3, 4); o(5, 6);
}

// The KD largest values seen (descending) and the largest of the others.
template <int KD>
struct TopList {
  float v[KD];
  float rest;
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < KD; ++i) v[i] = -CUDART_INF_F;
    rest = -CUDART_INF_F;
  }
  // With the descending list u: the larger of v[i] and u[KD-1-i] are the KD
  // largest of both, as a bitonic sequence.
  __device__ __forceinline__ void merge(const float (&u)[KD]) {
    float out = rest;
#pragma unroll
    for (int i = 0; i < KD; ++i) {
      const float x = v[i], y = u[KD - 1 - i];
      v[i] = fmaxf(x, y);
      out = fmaxf(out, fminf(x, y));
    }
    rest = out;
#pragma unroll
    for (int d = KD / 2; d > 0; d >>= 1)
#pragma unroll
      for (int i = 0; i < KD; ++i)
        if ((i & d) == 0) order_pair(v[i], v[i + d]);
  }
  // Eight values (unordered).
  __device__ __forceinline__ void add8(float (&x)[8]) {
    if constexpr (KD == 8) {
      sort8(x);
      merge(x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float c = x[e];
#pragma unroll
        for (int i = 0; i < KD; ++i) {
          const float hi = fmaxf(c, v[i]);
          c = fminf(c, v[i]);
          v[i] = hi;
        }
        rest = fmaxf(rest, c);
      }
    }
  }
};

// KD: at least k, of 2, 4 and 8. N: 16-byte pieces per lane (8, or 2 for few
// logits, which also keeps that code short). kWhole: E = 4 N P, no piece missing.
// 131072 tokens of 128 experts, top-2 with bias and statistics: 31 to 32 us, where the
// bytes take 10. 16 warps to an SM (128 registers a thread) issue in 44 % of the
// clocks, half of it comparisons of the lists; waits are for the row and for
// shuffles, and the last tokens decided again add 3 us. 16 experts to a lane gave
// 20 or 24 warps and 36 us; fetching the next row ahead changed nothing.
template <int P, int KD, int N, bool kWhole>
__global__ void __launch_bounds__(kFwdThreads, 4)
    route_grouped_kernel(const __grid_constant__ GroupedArgs a) {
  constexpr int kTok = 32 / P;                  // tokens per warp
  constexpr int kX = 4 * N;                     // experts per lane
  constexpr int kCols = kX * P;
  constexpr int kPitch = kCols + 4;             // 16-byte pieces of neighbour tokens in other banks
  constexpr int kGmax = kCols < 32 ? kCols : 32;
  constexpr int kList = 64;                     // tokens a warp puts off
  // selection values; room for route_exact's scratch
  constexpr int kExact = kMaxExperts * (sizeof(long long) + 2 * sizeof(float) + 1) / sizeof(float);
  __shared__ __align__(16) float sh_row[kFwdWarps][kTok * kPitch > kExact ? kTok * kPitch : kExact];
  __shared__ float sh_g[kFwdWarps][kTok][kGmax + 1];
  __shared__ int sh_pick[kFwdWarps][kTok][kMaxTopK];
  // token, its kept groups if certain, its k-th value
  __shared__ int sh_list[kFwdWarps][3][kList];
  __shared__ __align__(16) float sh_bias[kCols];  // -inf past E
  __shared__ int sh_cnt[kCols];
  __shared__ float sh_share[kFwdWarps][kCols];
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sub = lane & (P - 1), tok = lane / P;
  const int E = a.E, G = a.n_groups, S = E / G;
  const bool stats = a.tile_cnt != nullptr;
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  const bool vec = kWhole || (E & 3) == 0;
  for (int i = tid; i < kCols; i += kFwdThreads) {
    sh_cnt[i] = 0;
#pragma unroll
    for (int w = 0; w < kFwdWarps; ++w) sh_share[w][i] = 0.f;
    sh_bias[i] = i >= E ? -CUDART_INF_F : a.bias != nullptr ? a.bias[i] : 0.f;
  }
  // slots that nothing fills still name an expert
  for (int i = lane; i < kTok * kMaxTopK; i += 32) sh_pick[warp][i / kMaxTopK][i % kMaxTopK] = 0;
  if (blockIdx.x == 0 && tid == 0 && a.ticket != nullptr) *a.ticket = 0u;
  __syncthreads();
  float* row = sh_row[warp] + tok * kPitch;
  float* gv = sh_g[warp][tok];
  int* pick = sh_pick[warp][tok];
  int* cnt = stats ? sh_cnt : nullptr;
  uint64_t psum[kX / 2];
#pragma unroll
  for (int i = 0; i < kX / 2; ++i) psum[i] = f32x2(0.f, 0.f);
  uint32_t status = 0;
  int n_list = 0;
  auto flush = [&]() {
    __syncwarp();
    long long* val = reinterpret_cast<long long*>(sh_row[warp]);
    float* f = reinterpret_cast<float*>(val + kMaxExperts);
    const ExactScratch sc{val, f, f + kMaxExperts, reinterpret_cast<uint8_t*>(f + 2 * kMaxExperts), sh_pick[warp][0]};
    for (int q = 0; q < n_list; ++q) {
      const auto& w = sh_list[warp];
      route_exact(a, w[0][q], static_cast<uint32_t>(w[1][q]), __int_as_float(w[2][q]), sh_bias, sc, cnt,
                  stats ? sh_share[warp] : nullptr);
    }
    n_list = 0;
  };
  // piece i of the lane: experts 4 (sub + P i) .. + 3; the warp's pieces at i
  // start at 4 P i, so those from E on are skipped by all lanes
#define MOE_PIECES(i) _Pragma("unroll") for (int i = 0; i < N; ++i) if (kWhole || 4 * P * i < E)

  const int64_t per_pass = static_cast<int64_t>(gridDim.x) * kFwdWarps * kTok;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * kFwdWarps + warp) * kTok;
  for (int64_t base = first; base < a.T; base += per_pass) {
    const int64_t t = base + tok;
    const bool valid = t < a.T;
    const float* src = a.logits + (valid ? t : 0) * E;
    float x[kX];
#pragma unroll
    for (int i = 0; i < kX; ++i) x[i] = -kLowest;
    if (vec) {
      MOE_PIECES(i) {
        const int e = 4 * (sub + P * i);
        if (kWhole || e < E) {
          const float4 v = __ldcs(reinterpret_cast<const float4*>(src + e));
          x[4 * i] = v.x;
          x[4 * i + 1] = v.y;
          x[4 * i + 2] = v.z;
          x[4 * i + 3] = v.w;
        }
      }
    } else {
      MOE_PIECES(i) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int e = 4 * (sub + P * i) + q;
          if (e < E) x[4 * i + q] = __ldg(src + e);
        }
      }
    }
    // a logit that is not finite makes the sum NaN
    uint64_t chk = f32x2(0.f, 0.f);
    float m = -CUDART_INF_F;
    MOE_PIECES(i) {
      chk = f32x2_fma(f32x2(x[4 * i], x[4 * i + 1]), f32x2(0.f, 0.f), chk);
      chk = f32x2_fma(f32x2(x[4 * i + 2], x[4 * i + 3]), f32x2(0.f, 0.f), chk);
      m = max3(max3(m, x[4 * i], x[4 * i + 1]), x[4 * i + 2], x[4 * i + 3]);
    }
    float c0, c1;
    f32x2_get(chk, c0, c1);
    const bool has_mask = __any_sync(kFull, !(c0 + c1 == 0.f));
    uint32_t mk = 0u;
    if (has_mask) {
      m = -kLowest;
#pragma unroll
      for (int i = 0; i < kX; ++i) {
        if (masked(x[i])) {
          mk |= 1u << i;
          if (valid && x[i] != -CUDART_INF_F) status |= MOE_DEV_NONFINITE;
          x[i] = -kLowest;
        }
        m = fmaxf(m, x[i]);
      }
    }
    m = lanes_max<P>(m);
    // scores: softmax not yet divided by their sum. Past E they are those of the
    // lowest value: 0, unless the whole row is that low.
    if (softmax) {
      MOE_PIECES(i) {
#pragma unroll
        for (int q = 4 * i; q < 4 * i + 4; q += 2) {
          float u, v;
          f32x2_get(f32x2_mul(f32x2_add(f32x2(x[q], x[q + 1]), f32x2(-m, -m)), f32x2(kLog2e, kLog2e)), u, v);
          x[q] = exp2_approx(u);
          x[q + 1] = exp2_approx(v);
        }
      }
    } else {
      MOE_PIECES(i) {
#pragma unroll
        for (int q = 4 * i; q < 4 * i + 4; q += 2) {
          float u, v;
          f32x2_get(f32x2_mul(f32x2(x[q], x[q + 1]), f32x2(-kLog2e, -kLog2e)), u, v);
          f32x2_get(f32x2_add(f32x2(exp2_approx(u), exp2_approx(v)), f32x2(1.f, 1.f)), u, v);
          x[q] = rcp_approx(u);
          x[q + 1] = rcp_approx(v);
        }
      }
    }
    if (has_mask) {
#pragma unroll
      for (int i = 0; i < kX; ++i)
        if ((mk >> i) & 1u) x[i] = 0.f;
    }
    uint64_t zz = f32x2(0.f, 0.f);
    if (softmax || stats) {
      MOE_PIECES(i) {
        zz = f32x2_add(zz, f32x2(x[4 * i], x[4 * i + 1]));
        zz = f32x2_add(zz, f32x2(x[4 * i + 2], x[4 * i + 3]));
      }
    }
    float iz = 0.f;
    if (softmax || stats) {
      f32x2_get(zz, c0, c1);
      const float z = lanes_sum<P>(c0 + c1);
      iz = z > 0.f ? rcp_approx(z) : 0.f;
    }
    const bool tiny = tiny_row(m, softmax);
    const float smax = tiny ? 0.f : softmax ? iz : rcp_approx(1.f + exp2_approx(-m * kLog2e));
    if (stats) {
      const float f = valid && !tiny ? iz : 0.f;
      MOE_PIECES(i) {
        psum[2 * i] = f32x2_fma(f32x2(x[4 * i], x[4 * i + 1]), f32x2(f, f), psum[2 * i]);
        psum[2 * i + 1] = f32x2_fma(f32x2(x[4 * i + 2], x[4 * i + 3]), f32x2(f, f), psum[2 * i + 1]);
      }
    }
    // selection values, -inf where masked or past E
    const float f = softmax ? iz : 1.f;
    MOE_PIECES(i) {
      const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(sh_bias + 4 * (sub + P * i));
      f32x2_get(f32x2_fma(f32x2(x[4 * i], x[4 * i + 1]), f32x2(f, f), b.x), x[4 * i], x[4 * i + 1]);
      f32x2_get(f32x2_fma(f32x2(x[4 * i + 2], x[4 * i + 3]), f32x2(f, f), b.y), x[4 * i + 2], x[4 * i + 3]);
    }
    if (has_mask) {
#pragma unroll
      for (int i = 0; i < kX; ++i)
        if ((mk >> i) & 1u) x[i] = -CUDART_INF_F;
    }
    MOE_PIECES(i) {
      *reinterpret_cast<float4*>(row + 4 * (sub + P * i)) =
          make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    }
    __syncwarp();
    // Values closer than `near` are decided again. With u = 2^-24, a rounding's share,
    // 4 u of itself for ex2 and 2 u for rcp, a score is off by at most:
    //  sigmoid: s (1 - s) (1.23 |l| + 4) u + 3 s u (the argument -l log2e and its
    //    constant, ex2; the sum and rcp), over all l <= m below (5 + 2 max(0, -m)) u smax;
    //  softmax: (2.23 d + 4) exp(-d) u, at most 4 u of the largest, d = m - l. The divisor is
    //    off by 32.5 u (the terms' average, 2.23 x 3.34 + 4; 19 roundings of the sum;
    //    rcp), one factor for the row, which counts only where a bias is added: by that
    //    much of the scores' difference.
    // Two values: twice that. The bias adds a rounding to each, u of the value.
    // Group values that are sums of two scores: twice as much again, and a rounding. Of
    // two values that cancel more is left of their own roundings, 2 u of the smaller for
    // each sum: with that above smax / 4 + |sum| / 8, or a sum past fp32's range (as
    // biases can make both), the groups are in doubt.
    constexpr float kU = 0x1p-24f;
    const float near_one = smax * (softmax ? (a.bias != nullptr ? 44.f * kU : 11.f * kU)
                                           : fmaf(fmaxf(-m, 0.f), 4.1f * kU, 11.f * kU));
    auto near = [](float u, float v, float rel, float abs) {  // false where either is not finite
      return fabsf(u - v) < fmaf(rel, fmaxf(fabsf(u), fabsf(v)), abs);
    };
    bool unsure = tiny;
    uint32_t certain = 1u;  // the kept groups, or 0 where they are in doubt
    if (G > 1) {
      const float near_group = a.group_top == 2 ? fmaf(kU, smax, 2.f * near_one) : near_one;
      for (int g = sub; g < G; g += P) {
        float v1 = -CUDART_INF_F, v2 = -CUDART_INF_F;
        auto see = [&](float u) {
          v2 = fmaxf(v2, fminf(u, v1));
          v1 = fmaxf(v1, u);
        };
        if ((S & 3) == 0) {
          for (int q = 0; q < S; q += 4) {
            const float4 u = *reinterpret_cast<const float4*>(row + g * S + q);
            see(u.x);
            see(u.y);
            see(u.z);
            see(u.w);
          }
        } else {
          for (int q = 0; q < S; ++q) see(row[g * S + q]);
        }
        float v = v1;
        if (a.group_top == 2) {
          v = v1 + v2;
          unsure |= v2 != -CUDART_INF_F &&
                    (!(fabsf(v) < CUDART_INF_F) || fminf(v1, -v2) > fmaf(0.125f, fabsf(v), 0.25f * smax));
        }
        gv[g] = v;
      }
      __syncwarp();
      uint32_t kept = 0u;
      for (int g = sub; g < G; g += P) {
        const float u = gv[g];
        int ahead = 0, sure = 0, maybe = 0;
        for (int h = 0; h < G; ++h) {
          const float o = gv[h];
          const bool close = near(o, u, 4.5f * kU, near_group);
          ahead += (o > u || (o == u && h < g)) ? 1 : 0;
          sure += (o > u && !close) ? 1 : 0;
          maybe += (h != g && (o > u || close)) ? 1 : 0;
        }
        if (ahead < a.topk_groups) kept |= 1u << g;
        unsure |= u != -CUDART_INF_F && sure < a.topk_groups && maybe >= a.topk_groups;
      }
      kept = lanes_reduce<P>(kept, [](uint32_t u, uint32_t v) { return u | v; });
      const uint32_t vague = __ballot_sync(kFull, unsure);
      certain = ((vague >> (tok * P)) & (0xffffffffu >> (32 - P))) != 0u ? 0u : kept;
      MOE_PIECES(i) {
        const int e = 4 * (sub + P * i);
        int g = e / S, left = S - (e - g * S);  // experts left in the group, this one included
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (!((kept >> (g & 31)) & 1u)) x[4 * i + q] = -CUDART_INF_F;
          if (--left == 0) {
            ++g;
            left = S;
          }
        }
      }
    }
    TopList<KD> top;
    top.clear();
#pragma unroll
    for (int i = 0; i < N; i += 2)
      if (kWhole || 4 * P * i < E) {
        float u[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          u[q] = kWhole || 4 * P * (i + q / 4) < E ? x[4 * i + q] : -CUDART_INF_F;
        top.add8(u);
      }
#pragma unroll
    for (int o = 1; o < P; o <<= 1) {
      float u[KD];
#pragma unroll
      for (int i = 0; i < KD; ++i) u[i] = __shfl_xor_sync(kFull, top.v[i], o);
      const float r = __shfl_xor_sync(kFull, top.rest, o);
      top.merge(u);
      top.rest = fmaxf(top.rest, r);
    }
    float last = top.v[0];  // the k-th
#pragma unroll
    for (int i = 0; i < KD; ++i)
      if (i < a.k) {
        unsure |= near(top.v[i], i + 1 < KD ? top.v[i + 1] : top.rest, 4.f * kU, near_one);
        last = top.v[i];
      }
    unsure |= last == -CUDART_INF_F;  // fewer than k left
    // the experts at or above the k-th, k of them unless the token is in doubt
    uint32_t found = 0u;
    MOE_PIECES(i) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (x[4 * i + q] >= last) found |= 1u << (4 * i + q);
    }
    if (unsure) found = 0u;
    while (found != 0u) {
      const int b = __ffs(static_cast<int>(found)) - 1;
      found &= found - 1u;
      const int e = 4 * (sub + P * (b >> 2)) + (b & 3);
      const float u = row[e];
      int rank = 0;
#pragma unroll
      for (int i = 0; i < KD; ++i) rank += top.v[i] > u ? 1 : 0;
      if (rank < a.k) pick[rank] = e;
    }
    __syncwarp();
    const uint32_t doubt = __ballot_sync(kFull, unsure && valid);
    const bool mine = ((doubt >> (tok * P)) & (0xffffffffu >> (32 - P))) != 0u;
    write_slots<P>(a, t, pick, src, m, iz, sub, valid && !mine, cnt);
    if (doubt != 0u) {
      const uint32_t heads = __ballot_sync(kFull, mine && sub == 0);
      if (mine && sub == 0) {
        const int q = n_list + __popc(heads & ((1u << lane) - 1u));
        sh_list[warp][0][q] = static_cast<int>(t);
        sh_list[warp][1][q] = static_cast<int>(certain);
        sh_list[warp][2][q] = __float_as_int(last);
      }
      n_list += __popc(heads);
      if (n_list > kList - kTok) flush();
    }
    __syncwarp();
  }
  flush();
  if (status) atomicOr(a.dev_status, status);
  if (stats) {
    // per warp into its own rows' space, then over the block's warps and tokens
    __syncthreads();
    MOE_PIECES(i) {
      const int e = 4 * (sub + P * i);
      f32x2_get(psum[2 * i], row[e], row[e + 1]);
      f32x2_get(psum[2 * i + 1], row[e + 2], row[e + 3]);
    }
    __syncthreads();
    for (int e = tid; e < E; e += kFwdThreads) {
      float p = 0.f;
      for (int w = 0; w < kFwdWarps; ++w) {
#pragma unroll
        for (int q = 0; q < kTok; ++q) p += sh_row[w][q * kPitch + e];
        p += sh_share[w][e];
      }
      a.ppart[static_cast<size_t>(e) * gridDim.x + blockIdx.x] = p;
      a.tile_cnt[static_cast<size_t>(e) * gridDim.x + blockIdx.x] = sh_cnt[e];
    }
  }
#undef MOE_PIECES
}

// The blocks' counts and probability sums to routed, P and aux: a warp per
// expert, then the last block to finish. (The dispatch's scan, which could do
// this too, also forms prefixes: 7.2 us instead of 4 for 608 blocks.)
__global__ void __launch_bounds__(kStatsThreads) grouped_stats_kernel(GroupedStatsArgs a) {
  __shared__ int last;
  __shared__ float sh[kStatsWarps];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e = blockIdx.x * kStatsWarps + warp;
  if (e < a.E) {
    const int32_t* cnt = a.cnt + static_cast<size_t>(e) * a.blocks;
    const float* pp = a.ppart + static_cast<size_t>(e) * a.blocks;
    int n = 0;
    float p = 0.f;
#pragma unroll 4
    for (int i = lane; i < a.blocks; i += 32) {
      n += cnt[i];
      p += pp[i];
    }
    n = lanes_reduce<32>(n, [](int u, int v) { return u + v; });
    p = lanes_sum<32>(p);
    if (lane == 0) {
      a.routed[e] = n;
      a.P[e] = p / static_cast<float>(a.T);
    }
  }
  if (a.aux == nullptr) return;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(a.ticket, 1u) == gridDim.x - 1 ? 1 : 0;
  __syncthreads();
  if (!last) return;
  __threadfence();
  const int i = threadIdx.x;
  float v = i < a.E ? static_cast<float>(__ldcg(a.routed + i)) * __ldcg(a.P + i) : 0.f;
  v = lanes_sum<32>(v);
  if (lane == 0) sh[warp] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    float sum = 0.f;
    for (int w = 0; w < kStatsWarps; ++w) sum += sh[w];
    *a.aux = static_cast<float>(a.E) * sum / (static_cast<float>(a.T) * static_cast<float>(a.k));
  }
}

// ----------------------------------------------------------- gradient ----
// With q_j = s_j / sum of the chosen s and gradient g_j of weight j:
//   softmax, renormalised  dl_j = scale q_j (g_j - sum q g)
//   softmax                dl_e = p_e (G_e - sum_j p_j G_j), G_e = scale g_j if chosen
//   sigmoid, renormalised  dl_j = scale q_j (1 - s_j) (g_j - sum q g)
//   sigmoid                dl_j = scale g_j s_j (1 - s_j)
// and the balance loss, aux = E sum_e f_e mean_t p_te with f taken as constant,
// h_e = grad_aux E f_e / T, p = s / sum s:
//   softmax  dl_e += p_e (h_e - sum p h);  sigmoid  dl_e += p_e (1 - s_e) (h_e - sum p h)
// 65536 tokens of 256 experts, sigmoid with the balance loss: 27 us for 138 MB,
// 5.1 TB/s (26 in replays); 16 warps to an SM issue in 58 % of the clocks, and waits
// are for shuffles and arithmetic. With 8 experts to a lane, whose sums over lanes
// serve half as much work, it took 29.5 us; with 32 (a quarter of the threads) 31.
template <int L>
__global__ void __launch_bounds__(kThreads, 4) route_grouped_bwd_kernel(const __grid_constant__ GroupedBwdArgs a) {
  constexpr int kTok = 32 / L;
  constexpr int kPer = (kMaxTopK + L - 1) / L;  // chosen slots per lane: sub, sub + L, ...
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sub = lane & (L - 1), tok = lane / L;
  const int E = a.E;
  const bool softmax = a.score == MOE_SCORE_SOFTMAX, aux = a.grad_aux != nullptr;
  const bool need_p = aux || (softmax && !a.renormalize);  // the whole row's scores
  __shared__ __align__(16) float sh_row[kWarps][kTok][L * kV];
  uint64_t h[kV / 2];
#pragma unroll
  for (int i = 0; i < kV / 2; ++i) h[i] = f32x2(0.f, 0.f);
  if (aux) {
    const float T = static_cast<float>(a.T);
    const float f = *a.grad_aux * (static_cast<float>(E) / T) / (T * static_cast<float>(a.k));
#pragma unroll
    for (int i = 0; i < kV / 2; ++i) {
      const int e = 4 * (sub + L * (i / 2)) + 2 * (i % 2);
      h[i] = f32x2(e < E ? f * static_cast<float>(a.routed[e]) : 0.f,
                   e + 1 < E ? f * static_cast<float>(a.routed[e + 1]) : 0.f);
    }
  }
  const float none = softmax ? -kLowest : kFar;  // past E
  int past = 0;
#pragma unroll
  for (int i = 0; i < kV; ++i) past += 4 * (sub + L * (i / 4)) + i % 4 >= E ? 1 : 0;
  const float limit = square_limit(past);
  const int64_t per_pass = static_cast<int64_t>(gridDim.x) * kWarps * kTok;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kTok;
  // The next token's row and chosen logits, and the slots of the one after it,
  // are fetched while one is worked on. The row itself is not needed where only
  // chosen experts have a gradient.
  float next[kV], next_g[kPer], next_x[kPer], after_g[kPer];
  int next_e[kPer], after_e[kPer];
#pragma unroll
  for (int i = 0; i < kV; ++i) next[i] = 0.f;
  auto fetch_slots = [&](int64_t t) {
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int j = sub + q * L;
      const bool in = t < a.T && j < a.k;
      after_e[q] = in ? a.topk_idx[t * a.k + j] : -1;
      after_g[q] = in ? a.grad_w[t * a.k + j] : 0.f;
    }
  };
  auto fetch = [&](int64_t t) {  // the token whose slots were fetched last
    if (need_p) load_row<L>(a.logits, t < a.T ? t : 0, t < a.T, E, sub, none, next);
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      next_e[q] = after_e[q];
      next_g[q] = after_g[q];
      next_x[q] = -CUDART_INF_F;
      if (next_e[q] >= 0 && next_e[q] < E) next_x[q] = a.logits[t * E + next_e[q]];
    }
  };
  fetch_slots(first + tok);
  fetch(first + tok);
  fetch_slots(first + tok + per_pass);
  for (int64_t base = first; base < a.T; base += per_pass) {
    const int64_t t = base + tok;
    const bool valid = t < a.T;
    float l[kV];
    uint64_t s[kV / 2], grad[kV / 2];
    int ej[kPer];
    float gj[kPer], x[kPer];
#pragma unroll
    for (int i = 0; i < kV; ++i) l[i] = next[i];
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      x[q] = next_x[q];
      ej[q] = masked(x[q]) ? -1 : next_e[q];
      gj[q] = ej[q] < 0 ? 0.f : next_g[q];  // whatever stands there
    }
    fetch(t + per_pass);
    fetch_slots(t + 2 * per_pass);
    // s: softmax scores, or slopes of sigmoid scores
    float m = 0.f, iz = 0.f, ph = 0.f;
    if (need_p) {
      float z;
      if (softmax) {
        softmax_scores<L>(l, E, sub, s, m);
        z = pairs_sum(s);
        if (aux) {
          uint64_t acc = f32x2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < kV / 2; ++i) acc = f32x2_fma(s[i], h[i], acc);
          float u, v;
          f32x2_get(acc, u, v);
          ph = u + v;
        }
      } else {
        sigmoid_slopes<L>(l, h, limit, E, sub, s, z, ph);
      }
      z = lanes_sum<L>(z);
      iz = z > 0.f ? rcp_approx(z) : 0.f;
      if (aux) ph = lanes_sum<L>(ph) * iz;
    }
    // the chosen slots: in the first lanes of the token
    constexpr int kLanes = L < kMaxTopK ? L : kMaxTopK;
    float top = 0.f;
    if (a.renormalize) {
      top = -CUDART_INF_F;
#pragma unroll
      for (int q = 0; q < kPer; ++q)
        if (ej[q] >= 0) top = fmaxf(top, x[q]);
      top = lanes_reduce<kLanes>(top, [](float u, float v) { return fmaxf(u, v); });
    }
    const bool ratio = a.renormalize && (softmax || top < 0.f);
    const float shift = ratio ? top : m;
    float sj[kPer], dj[kPer];
    float sum = 0.f, dot = 0.f;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      dj[q] = softmax ? 1.f : rcp_approx(1.f + exp2_approx(x[q] * kLog2e));  // 1 - s
      const float y = exp2_approx((ratio || softmax ? x[q] - shift : -x[q]) * kLog2e);
      sj[q] = ej[q] < 0 ? 0.f : ratio ? y * dj[q] : softmax ? y * iz : rcp_approx(1.f + y);
      sum += sj[q];
    }
    if (a.renormalize) {
      sum = lanes_sum<kLanes>(sum);
      const float inv = sum > 0.f ? rcp_approx(sum) : 0.f;
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        sj[q] *= inv;
        dot += sj[q] * gj[q];
      }
      dot = lanes_sum<kLanes>(dot);
#pragma unroll
      for (int q = 0; q < kPer; ++q) dj[q] *= a.scale * sj[q] * (gj[q] - dot);
      dot = 0.f;
    } else {
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        dj[q] *= a.scale * sj[q] * gj[q];
        dot += softmax ? dj[q] : 0.f;
      }
      dot = lanes_sum<L>(dot);
    }
    // the whole row's part: p_e slope_e (h_e - sum p h - dot)
#pragma unroll
    for (int i = 0; i < kV / 2; ++i) grad[i] = f32x2(0.f, 0.f);
    if (need_p) {
      if (softmax && !a.renormalize) ph += dot;
      const float c = -ph * iz;
#pragma unroll
      for (int i = 0; i < kV / 2; ++i) {
        grad[i] = f32x2_mul(s[i], f32x2_fma(h[i], f32x2(iz, iz), f32x2(c, c)));
      }
    }
    // the chosen experts' part is added in shared memory
    float* row = sh_row[warp][tok];
#pragma unroll
    for (int q = 0; q < kV / 4; ++q)
      *reinterpret_cast<ulonglong2*>(row + 4 * (sub + L * q)) = make_ulonglong2(grad[2 * q], grad[2 * q + 1]);
    __syncwarp();
#pragma unroll
    for (int q = 0; q < kPer; ++q)
      if (ej[q] >= 0) row[ej[q]] += dj[q];
    __syncwarp();
    if (valid) {
      float* out = a.grad_logits + t * E;
      if ((E & 3) == 0) {
#pragma unroll
        for (int q = 0; q < kV / 4; ++q) {
          const int e = 4 * (sub + L * q);
          if (e < E) __stcs(reinterpret_cast<float4*>(out + e), *reinterpret_cast<const float4*>(row + e));
        }
      } else {
        for (int e = sub; e < E; e += L) out[e] = row[e];
      }
    }
    __syncwarp();  // the next token's stores to the row come after other lanes' reads of it
  }
}

// Gradient: lanes per token.
int lanes_of(int E) {
  int L = 2;
  while (L * kV < E) L <<= 1;
  return L;
}
// Forward: experts per lane. 32 do the least work per token; where there are too
// few logits to fill the GPU so, 8 have the answer sooner. In us, 8 against 32:
// 1 token of 64 experts 2.5, 3.1; 1024 of 256 4.2, 4.9; 2048 of 256 8.6, 8.7;
// 4096 of 256 11.7, 9.8; 8192 of 64 7.0, 7.3; 16384 of 64 9.2, 7.9; 131072 of 64
// 36.7, 20.6.
bool few_logits(int64_t T, int E) { return T * E <= 512 * 1024; }
int parts_of(int T, int E) {
  const int each = few_logits(T, E) ? 8 : 32;
  int P = 1;
  while (each * P < E) P <<= 1;
  return P;
}

// 131072 tokens: a list of 2 for k = 2 takes 39 us at 256 experts, 21.6 at 128,
// with one of 8 56 and 28; of 4 for k = 4 49 and 28.4, with 8 58 and 30.5. Without
// kWhole the lists of 2 take 48 and 25, those of 8 72 instead of 63 at 256 experts.
template <int P, int KD>
cudaError_t launch_many(const GroupedArgs& a, dim3 grid, cudaStream_t st) {
  const dim3 block(kFwdThreads);
  if (a.E == 32 * P) return launch_pdl(route_grouped_kernel<P, KD, 8, true>, grid, block, 0, st, a);
  return launch_pdl(route_grouped_kernel<P, KD, 8, false>, grid, block, 0, st, a);
}
template <int P>
cudaError_t launch_forward(const GroupedArgs& a, cudaStream_t st) {
  const dim3 grid(route_grouped_blocks(a.T, a.E));
  if constexpr (P <= kMaxExperts / 32)
    if (!few_logits(a.T, a.E)) {
      if (a.k <= 2) return launch_many<P, 2>(a, grid, st);
      if (a.k <= 4) return launch_many<P, 4>(a, grid, st);
      return launch_many<P, 8>(a, grid, st);
    }
  return launch_pdl(route_grouped_kernel<P, 8, 2, false>, grid, dim3(kFwdThreads), 0, st, a);
}

}  // namespace

int route_grouped_blocks(int T, int E) {
  const int per_block = kFwdWarps * (32 / parts_of(T, E));
  const int64_t n = (static_cast<int64_t>(T) + per_block - 1) / per_block;
  return static_cast<int>(n < kGroupedMaxBlocks ? n : kGroupedMaxBlocks);
}

cudaError_t launch_route_grouped(const GroupedArgs& a, cudaStream_t st) {
  switch (parts_of(a.T, a.E)) {
    case 1: return launch_forward<1>(a, st);
    case 2: return launch_forward<2>(a, st);
    case 4: return launch_forward<4>(a, st);
    case 8: return launch_forward<8>(a, st);
    case 16: return launch_forward<16>(a, st);
    default: return launch_forward<32>(a, st);
  }
}

cudaError_t launch_grouped_stats(const GroupedStatsArgs& a, cudaStream_t st) {
  return launch_pdl(grouped_stats_kernel, dim3((a.E + kStatsWarps - 1) / kStatsWarps), dim3(kStatsThreads), 0, st, a);
}

cudaError_t launch_route_grouped_bwd(const GroupedBwdArgs& a, cudaStream_t st) {
  const int L = lanes_of(a.E);
  const int64_t blocks = (static_cast<int64_t>(a.T) + kWarps * (32 / L) - 1) / (kWarps * (32 / L));
  const dim3 grid(static_cast<unsigned>(blocks < kGroupedMaxBlocks ? blocks : kGroupedMaxBlocks)), block(kThreads);
  switch (L) {
    case 2: return launch_pdl(route_grouped_bwd_kernel<2>, grid, block, 0, st, a);
    case 4: return launch_pdl(route_grouped_bwd_kernel<4>, grid, block, 0, st, a);
    case 8: return launch_pdl(route_grouped_bwd_kernel<8>, grid, block, 0, st, a);
    default: return launch_pdl(route_grouped_bwd_kernel<16>, grid, block, 0, st, a);
  }
}

}  // namespace moe
