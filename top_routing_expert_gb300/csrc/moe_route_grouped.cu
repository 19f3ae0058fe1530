// Grouped routing from fp32 logits and its gradient: softmax or sigmoid
// scores, a bias that acts on the selection alone, groups of experts, top-k,
// renormalised and scaled weights, and the balance statistics.
//
// Per token, with logits l (a logit that is not finite masks its expert):
//   s_e = softmax(l)_e or 1 / (1 + exp(-l_e));  c_e = s_e + b_e, -inf if masked
//   group value = sum of the group's g largest c; the best groups are kept
//   idx = top-k of c over the kept groups, w_j = scale * s_j / sum_j s_j
//
// L lanes share one token and hold 8 consecutive experts each (L * 8 >= E), so
// a warp routes 32 / L tokens at once and a row is read in 16-byte vectors.
//
// The choice is that of the formulas in 64 bits. Scores are computed in fp32,
// and wherever two values that a decision compares are closer than the fp32
// error allows, the token is decided again in fp64 (fp64 runs at a small
// fraction of the fp32 rate here, so only those tokens pay for it).
#include <math_constants.h>

#include "moe_internal.h"
#include "moe_ptx.cuh"

namespace moe {

namespace {

constexpr int kV = 8;          // experts per lane
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr unsigned kFull = 0xffffffffu;
constexpr float kLowest = 3.402823466e38f;  // -kLowest: fp32's lowest value

// Keys order selection values as floats: the lowest 3 bits replaced by 7 - slot,
// so that a lane's keys differ and carry the slot. Keys below kRegular mark
// experts that come after every other one: masked experts of kept groups, by
// index (their bits end in 7 - slot too), then experts that are not to be had.
constexpr float kRegular = -2.9e38f;
__device__ __forceinline__ float key_of(float c, int slot) {
  return __uint_as_float((__float_as_uint(c) & ~7u) | static_cast<uint32_t>(7 - slot));
}
__device__ __forceinline__ float key_masked(int e) {  // -3.0e38 and a little below
  return __uint_as_float(0xff61b000u + 8u * static_cast<uint32_t>(e) + static_cast<uint32_t>(7 - (e & 7)));
}
__device__ __forceinline__ float key_out(int slot) {  // -3.3e38 and a little below
  return __uint_as_float(0xff784000u + static_cast<uint32_t>(7 - slot));
}

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
__device__ __forceinline__ bool masked(float l) { return !(fabsf(l) < CUDART_INF_F); }

// ------------------------------------------------------------- fp64 ----
// The choice of one token in fp64, by a whole warp (lane l: experts l, l + 32,
// ...), then its weights. fp64 instructions run at 1/64 of the fp32 rate, so
// comparisons are made on the values' bits as ordered integers.
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
    // Weights are ratios then: softmax scores are taken relative to the largest
    // chosen logit, and so are sigmoid scores far below zero (where 1 + exp(l)
    // is 1), which would underflow.
    top = lanes_reduce<kLanes>(top, [](float u, float v) { return fmaxf(u, v); });
    const bool ratio = softmax || top < -40.f;
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const float y = ratio ? exp2_approx((x[q] - top) * kLog2e) : rcp_approx(1.f + exp2_approx(-x[q] * kLog2e));
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
  long long* cs;          // [kMaxExperts]: ordered fp64 values
  float* cf;              // [kMaxExperts]: fp32 values
  uint8_t* list;          // [kMaxExperts]: experts to evaluate
  int* pick;              // [kMaxTopK]
};

__device__ __noinline__ double score64(float x, float m, bool softmax) {
  const double y = exp(softmax ? static_cast<double>(x) - static_cast<double>(m) : -static_cast<double>(x));
  return softmax ? y : 1.0 / (1.0 + y);
}

// Only experts that may matter are evaluated in fp64: those whose fp32 value is
// within `slack` of the group_top-th of their group, then those within it of a
// lower bound of the kept groups' k-th. All others rank below them whatever the
// error. (A softmax with a bias needs its fp64 sum too, hence all exponentials.)
// Few tokens come here, on any SM, so the code is kept short: fetching
// instructions for the first time costs more than running them.
__device__ __noinline__ void route_exact(const GroupedArgs& a, int t, const ExactScratch& sc,
                                         int* cnt) {
  const int lane = threadIdx.x & 31;
  const int E = a.E, S = a.E / a.n_groups;
  const float* row = a.logits + static_cast<int64_t>(t) * E;
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  const bool all = softmax && a.bias != nullptr;
  const long long kInf = order64(-CUDART_INF);
  const long long kNever = -0x7fffffffffffffffll - 1;  // not evaluated: below -inf
  float m = -CUDART_INF_F, smax = 0.f, z = 0.f, big = 0.f;
#pragma unroll 1
  for (int e = lane; e < E; e += 32) {
    const float x = row[e];
    sc.cf[e] = masked(x) ? -CUDART_INF_F : x;
    m = fmaxf(m, sc.cf[e]);
  }
  m = lanes_max<32>(m);
  if (m == -CUDART_INF_F) m = 0.f;  // nothing unmasked
  double z64 = 0.0;
#pragma unroll 1
  for (int e = lane; e < E; e += 32) {  // cf: the scores, -inf where masked
    const float x = sc.cf[e];
    sc.cs[e] = x == -CUDART_INF_F ? kInf : kNever;
    if (x != -CUDART_INF_F) {
      const float y = softmax ? expf(x - m) : 1.f / (1.f + expf(-x));
      sc.cf[e] = y;
      z += y;
      smax = fmaxf(smax, y);
      if (all) z64 += score64(x, m, true);
    }
  }
  z = lanes_sum<32>(z);
  smax = lanes_max<32>(smax);
  const float iz = softmax && z > 0.f ? 1.f / z : 0.f;
  if (all) z64 = lanes_reduce<32>(z64, [](double x, double y) { return x + y; });
  // softmax scores are compared as exp(l - m) where nothing is added to them
#pragma unroll 1
  for (int e = lane; e < E; e += 32)
    if (a.bias != nullptr && sc.cf[e] != -CUDART_INF_F) {
      sc.cf[e] = fmaf(sc.cf[e], all ? iz : 1.f, a.bias[e]);
      big = fmaxf(big, fabsf(sc.cf[e]));
    }
  big = fmaxf(lanes_max<32>(big), all ? smax * iz : smax);
  // fp32 errors are within 2^-18 of the largest value (2^-14 where the logits are
  // so low that exp's argument is what errs)
  const float slack = big * (softmax || smax > 1e-3f ? 0x1p-17f : 0x1p-13f);
  __syncwarp();
  uint32_t kept = 0xffffffffu;
  int n = 0;
  // phase 0 settles the groups, phase 1 the experts
#pragma unroll 1
  for (int phase = a.n_groups > 1 ? 0 : 1; phase < 2; ++phase) {
    float bound = -CUDART_INF_F;  // lane g: of group g
    if (phase == 0) {
      if (lane < a.n_groups) {
        float v1 = -CUDART_INF_F, v2 = -CUDART_INF_F;
#pragma unroll 1
        for (int q = 0; q < S; ++q) {
          const float v = sc.cf[lane * S + q];
          v2 = fmaxf(v2, fminf(v, v1));
          v1 = fmaxf(v1, v);
        }
        bound = a.group_top == 2 ? v2 : v1;
      }
    } else {
      // the k-th largest of the lanes' own maxima
      float own = -CUDART_INF_F;
#pragma unroll 1
      for (int e = lane; e < E; e += 32)
        if ((kept >> (a.n_groups > 1 ? e / S : 0)) & 1u) own = fmaxf(own, sc.cf[e]);
#pragma unroll 1
      for (int j = 0; j < a.k; ++j) {
        bound = lanes_max<32>(own);
        const unsigned who = __ballot_sync(kFull, own == bound);
        if (lane == __ffs(static_cast<int>(who)) - 1) own = -CUDART_INF_F;
      }
    }
    // the candidates, in order of their index
    n = 0;
#pragma unroll 1
    for (int b = 0; b < E; b += 32) {
      const int e = b + lane, g = e < E && a.n_groups > 1 ? e / S : 0;
      const float lim = phase == 0 ? __shfl_sync(kFull, bound, g) : bound;
      const bool in = e < E && sc.cf[e] >= lim - slack && (phase == 0 || ((kept >> g) & 1u));
      const unsigned who = __ballot_sync(kFull, in);
      if (in) sc.list[n + __popc(who & ((1u << lane) - 1u))] = static_cast<uint8_t>(e);
      n += __popc(who);
    }
    __syncwarp();
#pragma unroll 1
    for (int q = lane; q < n; q += 32) {
      const int e = sc.list[q];
      if (sc.cs[e] == kNever) {
        double v = score64(row[e], m, softmax);
        if (all) v /= z64;
        if (a.bias != nullptr) v += static_cast<double>(a.bias[e]);
        sc.cs[e] = order64(v);
      }
    }
    __syncwarp();
    if (phase == 0) {
      long long v1 = kInf, v2 = kInf;
      if (lane < a.n_groups) {
#pragma unroll 1
        for (int q = 0; q < S; ++q) {
          const long long v = sc.cs[lane * S + q];
          v2 = max(v2, min(v, v1));
          v1 = max(v1, v);
        }
        if (a.group_top == 2)  // order64 is its own inverse
          v1 = order64(__longlong_as_double(order64(__longlong_as_double(v1))) +
                       __longlong_as_double(order64(__longlong_as_double(v2))));
      }
      int ahead = 0;
#pragma unroll 1
      for (int h = 0; h < a.n_groups; ++h) {
        const long long o = __shfl_sync(kFull, v1, h);
        ahead += (o > v1 || (o == v1 && h < lane)) ? 1 : 0;
      }
      kept = __ballot_sync(kFull, lane < a.n_groups && ahead < a.topk_groups);
    }
  }
  // the candidates' ranks: ties go to the lower index, which comes first here
#pragma unroll 1
  for (int q = lane; q < n; q += 32) {
    const int e = sc.list[q];
    const long long v = sc.cs[e];
    int rank = 0;
#pragma unroll 1
    for (int r = 0; r < n; ++r) {
      const long long o = sc.cs[sc.list[r]];
      rank += (o > v || (o == v && r < q)) ? 1 : 0;
    }
    if (rank < a.k) sc.pick[rank] = e;
  }
  __syncwarp();
  write_slots<32>(a, t, sc.pick, row, m, iz, lane, true, cnt);
  __syncwarp();
}

// ------------------------------------------------------------- kernel ----

// The lane's 8 logits of row t, the type's lowest value past E or T.
template <int L>
__device__ __forceinline__ void load_row(const float* __restrict__ logits, int64_t t, bool valid,
                                         int E, int sub, float (&l)[kV]) {
  const float* row = logits + t * E;
  const int e0 = sub * kV;
  if ((E & 3) == 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float4 v = make_float4(-kLowest, -kLowest, -kLowest, -kLowest);
      if (valid && e0 + 4 * h < E) v = __ldg(reinterpret_cast<const float4*>(row + e0 + 4 * h));
      l[4 * h] = v.x;
      l[4 * h + 1] = v.y;
      l[4 * h + 2] = v.z;
      l[4 * h + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kV; ++i) l[i] = valid && e0 + i < E ? __ldg(row + e0 + i) : -kLowest;
  }
}

// Masked experts of the lane (bits), their logits set to the lowest value. A
// multiply-add per pair of logits finds whether there is any.
__device__ __forceinline__ uint32_t find_masked(float (&l)[kV], uint32_t& status) {
  uint64_t chk = f32x2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kV; i += 2) chk = f32x2_fma(f32x2(l[i], l[i + 1]), f32x2(0.f, 0.f), chk);
  float c0, c1;
  f32x2_get(chk, c0, c1);
  if (!__any_sync(kFull, !(c0 + c1 == 0.f))) return 0u;
  uint32_t mk = 0u;
#pragma unroll
  for (int i = 0; i < kV; ++i)
    if (masked(l[i])) {
      mk |= 1u << i;
      if (l[i] != -CUDART_INF_F) status |= MOE_DEV_NONFINITE;
      l[i] = -kLowest;
    }
  return mk;
}

// The lane's scores in pairs (softmax: exp(l - m), not yet divided by their sum
// over the row), 0 where masked.
template <int L>
__device__ __forceinline__ void scores(const float (&l)[kV], uint32_t mk, bool softmax,
                                       uint64_t (&s)[kV / 2], float& m) {
  m = 0.f;
  float x[kV];
  if (softmax) {
    m = fmaxf(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])), fmaxf(fmaxf(l[4], l[5]), fmaxf(l[6], l[7])));
    m = lanes_max<L>(m);
#pragma unroll
    for (int i = 0; i < kV; i += 2)
      f32x2_get(f32x2_mul(f32x2_add(f32x2(l[i], l[i + 1]), f32x2(-m, -m)), f32x2(kLog2e, kLog2e)), x[i],
                x[i + 1]);
#pragma unroll
    for (int i = 0; i < kV; ++i) x[i] = exp2_approx(x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kV; i += 2) {
      float y0, y1;
      f32x2_get(f32x2_mul(f32x2(l[i], l[i + 1]), f32x2(-kLog2e, -kLog2e)), y0, y1);
      f32x2_get(f32x2_add(f32x2(exp2_approx(y0), exp2_approx(y1)), f32x2(1.f, 1.f)), y0, y1);
      x[i] = rcp_approx(y0);
      x[i + 1] = rcp_approx(y1);
    }
  }
  if (mk != 0u) {
#pragma unroll
    for (int i = 0; i < kV; ++i)
      if ((mk >> i) & 1u) x[i] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < kV; i += 2) s[i / 2] = f32x2(x[i], x[i + 1]);
}
__device__ __forceinline__ float pairs_sum(const uint64_t (&s)[kV / 2]) {
  float a, b;
  f32x2_get(f32x2_add(f32x2_add(s[0], s[1]), f32x2_add(s[2], s[3])), a, b);
  return a + b;
}

template <int L>
__global__ void __launch_bounds__(kThreads, 3) route_grouped_kernel(const __grid_constant__ GroupedArgs a) {
  constexpr int kTok = 32 / L;                       // tokens per warp
  constexpr int kCols = L * kV;
  constexpr int kGmax = kCols < 32 ? kCols : 32;     // groups per token at most
  constexpr int kList = 32;                          // tokens a warp puts off
  // per warp: logits and selection values of its tokens; route_exact's values
  __shared__ __align__(16) float sh_row[kWarps][2][kTok][kCols];
  __shared__ float sh_g[kWarps][kTok][kGmax];
  __shared__ uint8_t sh_eval[kWarps][kMaxExperts];
  __shared__ int sh_pick[kWarps][kTok][kMaxTopK];
  __shared__ int sh_list[kWarps][kList];
  __shared__ __align__(16) float sh_bias[kCols];
  __shared__ float sh_p[kWarps][kTok][kCols];        // sums of p at the end; route_exact's fp32 values
  __shared__ int sh_cnt[kCols];
  static_assert(sizeof(sh_row[0]) == kMaxExperts * sizeof(long long), "route_exact's scratch");
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sub = lane & (L - 1), tok = lane / L;
  const int E = a.E, G = a.n_groups, S = E / G;
  const bool stats = a.tile_cnt != nullptr;
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  for (int i = tid; i < kCols; i += kThreads) {
    sh_cnt[i] = 0;
    sh_bias[i] = a.bias != nullptr && i < E ? a.bias[i] : 0.f;
  }
  if (blockIdx.x == 0 && tid == 0 && a.ticket != nullptr) *a.ticket = 0u;
  __syncthreads();
  float* row = sh_row[warp][0][tok];
  float* cs = sh_row[warp][1][tok];
  float* gv = sh_g[warp][tok];
  int* pick = sh_pick[warp][tok];
  int* cnt = stats ? sh_cnt : nullptr;
  // which of the lane's experts exist, and their groups (a byte each)
  uint32_t exist = 0;
  uint64_t gids = 0;
#pragma unroll
  for (int i = 0; i < kV; ++i)
    if (sub * kV + i < E) {
      exist |= 1u << i;
      gids |= static_cast<uint64_t>((sub * kV + i) / S) << (8 * i);
    }
  // Lanes per group where groups are whole lanes, a power of two of them.
  const int gl = G > 1 && S % kV == 0 && ((S / kV) & (S / kV - 1)) == 0 ? S / kV : 0;
  uint64_t psum[kV / 2];
#pragma unroll
  for (int i = 0; i < kV / 2; ++i) psum[i] = f32x2(0.f, 0.f);
  uint32_t status = 0;
  int n_list = 0;
  auto flush = [&]() {
    __syncwarp();
    for (int q = 0; q < n_list; ++q)
      route_exact(a, sh_list[warp][q],
                  ExactScratch{reinterpret_cast<long long*>(sh_row[warp]), sh_p[warp][0], sh_eval[warp],
                               sh_pick[warp][0]},
                  cnt);
    n_list = 0;
  };

  const int64_t per_pass = static_cast<int64_t>(gridDim.x) * kWarps * kTok;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kTok;
  float next[kV];
  load_row<L>(a.logits, first + tok < a.T ? first + tok : 0, first + tok < a.T, E, sub, next);
  for (int64_t base = first; base < a.T; base += per_pass) {
    const int64_t t = base + tok;
    const bool valid = t < a.T;
    float l[kV], c[kV];
    uint64_t s[kV / 2];
#pragma unroll
    for (int i = 0; i < kV; ++i) l[i] = next[i];
    // the next token's row is fetched while this one is worked on
    const int64_t tn = t + per_pass;
    load_row<L>(a.logits, tn < a.T ? tn : 0, tn < a.T, E, sub, next);
    const uint32_t mk = find_masked(l, status);
    float m, smax, iz = 0.f;
    scores<L>(l, mk, softmax, s, m);
    if (softmax || stats) {
      const float z = lanes_sum<L>(pairs_sum(s));
      iz = z > 0.f ? rcp_approx(z) : 0.f;
    }
    if (softmax) {
#pragma unroll
      for (int i = 0; i < kV / 2; ++i) s[i] = f32x2_mul(s[i], f32x2(iz, iz));
      smax = iz;  // exp(0) / z
    }
    if (stats) {
      const float f = !valid ? 0.f : softmax ? 1.f : iz;
#pragma unroll
      for (int i = 0; i < kV / 2; ++i) psum[i] = f32x2_fma(s[i], f32x2(f, f), psum[i]);
    }
    {
      const ulonglong2 b0 = *reinterpret_cast<const ulonglong2*>(sh_bias + sub * kV);
      const ulonglong2 b1 = *reinterpret_cast<const ulonglong2*>(sh_bias + sub * kV + 4);
      if (!softmax) {
#pragma unroll
        for (int i = 0; i < kV / 2; ++i) f32x2_get(s[i], c[2 * i], c[2 * i + 1]);
        smax = fmaxf(fmaxf(fmaxf(c[0], c[1]), fmaxf(c[2], c[3])), fmaxf(fmaxf(c[4], c[5]), fmaxf(c[6], c[7])));
        smax = lanes_max<L>(smax);
      }
      f32x2_get(f32x2_add(s[0], b0.x), c[0], c[1]);
      f32x2_get(f32x2_add(s[1], b0.y), c[2], c[3]);
      f32x2_get(f32x2_add(s[2], b1.x), c[4], c[5]);
      f32x2_get(f32x2_add(s[3], b1.y), c[6], c[7]);
    }
    if (mk != 0u) {
#pragma unroll
      for (int i = 0; i < kV; ++i)
        if ((mk >> i) & 1u) {
          c[i] = -CUDART_INF_F;
          l[i] = -CUDART_INF_F;
        }
    }
    *reinterpret_cast<float4*>(row + sub * kV) = make_float4(l[0], l[1], l[2], l[3]);
    *reinterpret_cast<float4*>(row + sub * kV + 4) = make_float4(l[4], l[5], l[6], l[7]);
    // A score's error is within 2^-21 of the row's largest score (2^-17 where
    // all logits are far below zero and the exponent's rounding counts), the
    // bias adds a rounding, and the keys drop 3 bits (2^-20): values closer
    // than `near` are decided in fp64.
    const float near_abs = smax * (softmax || smax > 1e-3f ? 0x1p-20f : 0x1p-16f);
    auto near = [&](float x, float y) {
      return fabsf(x - y) < fmaf(0x1p-19f, fmaxf(fabsf(x), fabsf(y)), near_abs);
    };
    bool unsure = smax < 1e-30f;
    uint32_t avail = exist;
    if (G > 1) {
      float v = 0.f;
      int g0 = 0, step = 0;
      if (gl > 0) {
        float v1 = c[0], v2 = -CUDART_INF_F;
#pragma unroll
        for (int i = 1; i < kV; ++i) {
          v2 = fmaxf(v2, fminf(c[i], v1));
          v1 = fmaxf(v1, c[i]);
        }
        for (int o = 1; o < gl; o <<= 1) {
          const float o1 = __shfl_xor_sync(kFull, v1, o), o2 = __shfl_xor_sync(kFull, v2, o);
          v2 = fmaxf(fmaxf(v2, o2), fminf(v1, o1));
          v1 = fmaxf(v1, o1);
        }
        v = a.group_top == 2 ? v1 + v2 : v1;
        if ((sub & (gl - 1)) == 0 && sub / gl < G) gv[sub / gl] = v;
        g0 = sub / gl;
        step = G;  // the lane's own group alone
      } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) cs[sub * kV + i] = c[i];
        __syncwarp();
        for (int g = sub; g < G; g += L) {
          float v1 = -CUDART_INF_F, v2 = -CUDART_INF_F;
          for (int q = 0; q < S; ++q) {
            const float x = cs[g * S + q];
            v2 = fmaxf(v2, fminf(x, v1));
            v1 = fmaxf(v1, x);
          }
          gv[g] = a.group_top == 2 ? v1 + v2 : v1;
        }
        g0 = sub;
        step = L;
      }
      __syncwarp();
      uint32_t kept = 0u;
      for (int g = g0; g < G; g += step) {
        const float x = gv[g];
        int ahead = 0, sure = 0, maybe = 0;
        for (int h = 0; h < G; ++h) {
          const float o = gv[h];
          ahead += (o > x || (o == x && h < g)) ? 1 : 0;
          const bool close = near(o, x);  // false where either is -inf: their difference is not finite
          sure += (o > x && !close) ? 1 : 0;
          maybe += (h != g && (o > x || close)) ? 1 : 0;
        }
        if (ahead < a.topk_groups) kept |= 1u << g;
        unsure |= x != -CUDART_INF_F && sure < a.topk_groups && maybe >= a.topk_groups;
      }
      if (gl > 0) {
        avail = kept != 0u ? exist : 0u;
      } else {
        kept = lanes_reduce<L>(kept, [](uint32_t x, uint32_t y) { return x | y; });
        avail = 0u;
#pragma unroll
        for (int i = 0; i < kV; ++i)
          avail |= ((kept >> ((gids >> (8 * i)) & 31u)) & 1u) << i;
        avail &= exist;
      }
    }
    float key[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) key[i] = key_of(c[i], i);
    if (avail != 0xffu || mk != 0u) {
#pragma unroll
      for (int i = 0; i < kV; ++i)
        key[i] = !((avail >> i) & 1u) ? key_out(i) : ((mk >> i) & 1u) ? key_masked(sub * kV + i) : key[i];
    }
    // the lane's keys, largest first (Batcher's odd-even merge sort of 8)
    auto swap = [&](int x, int y) {
      const float hi = fmaxf(key[x], key[y]), lo = fminf(key[x], key[y]);
      key[x] = hi;
      key[y] = lo;
    };
    swap(0, 1); swap(2, 3); swap(4, 5); swap(6, 7);
    swap(0, 2); swap(1, 3); swap(4, 6); swap(5, 7);
    swap(1, 2); swap(5, 6);
    swap(0, 4); swap(1, 5); swap(2, 6); swap(3, 7);
    swap(2, 4); swap(3, 5);
    swap(1, 2); swap(3, 4); swap(5, 6);
    float prev = CUDART_INF_F;
    for (int j = 0; j <= a.k; ++j) {
      const float best = lanes_max<L>(key[0]);
      // regular values in descending order (against the first, inf, false)
      unsure |= best > kRegular && near(prev, best);
      prev = best;
      // the owner takes it out; two owners are a tie
      const uint32_t owners = (__ballot_sync(kFull, key[0] == best) >> (tok * (L & 31))) & (0xffffffffu >> (32 - L));
      unsure |= best > kRegular && (owners & (owners - 1u)) != 0u;
      if (key[0] == best && j < a.k) {
        pick[j] = sub * kV + 7 - static_cast<int>(__float_as_uint(best) & 7u);
#pragma unroll
        for (int i = 0; i + 1 < kV; ++i) key[i] = key[i + 1];
        key[kV - 1] = -CUDART_INF_F;
      }
    }
    __syncwarp();
    const uint32_t doubt = __ballot_sync(kFull, unsure && valid);
    const bool mine = ((doubt >> (tok * (L & 31))) & (0xffffffffu >> (32 - L))) != 0u;
    write_slots<L>(a, t, pick, row, m, iz, sub, valid && !mine, cnt);
    if (doubt != 0u) {
      const uint32_t heads = __ballot_sync(kFull, mine && sub == 0);
      if (mine && sub == 0) sh_list[warp][n_list + __popc(heads & ((1u << lane) - 1u))] =
          static_cast<int>(t);
      n_list += __popc(heads);
      if (n_list > kList - kTok) flush();
    }
    __syncwarp();
  }
  flush();
  if (status) atomicOr(a.dev_status, status);
  if (stats) {
#pragma unroll
    for (int i = 0; i < kV / 2; ++i)
      f32x2_get(psum[i], sh_p[warp][tok][sub * kV + 2 * i], sh_p[warp][tok][sub * kV + 2 * i + 1]);
    __syncthreads();
    for (int e = tid; e < E; e += kThreads) {
      float p = 0.f;
      for (int w = 0; w < kWarps; ++w)
#pragma unroll
        for (int q = 0; q < kTok; ++q) p += sh_p[w][q][e];
      a.ppart[static_cast<size_t>(e) * gridDim.x + blockIdx.x] = p;
      a.tile_cnt[static_cast<size_t>(e) * gridDim.x + blockIdx.x] = sh_cnt[e];
    }
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
      const int e = sub * kV + 2 * i;
      h[i] = f32x2(e < E ? f * static_cast<float>(a.routed[e]) : 0.f,
                   e + 1 < E ? f * static_cast<float>(a.routed[e + 1]) : 0.f);
    }
  }
  uint32_t status = 0;  // the forward has reported
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
    if (need_p) load_row<L>(a.logits, t < a.T ? t : 0, t < a.T, E, sub, next);
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
      gj[q] = next_g[q];
      x[q] = next_x[q];
      ej[q] = masked(x[q]) ? -1 : next_e[q];
    }
    fetch(t + per_pass);
    fetch_slots(t + 2 * per_pass);
    float m = 0.f, iz = 0.f;
    if (need_p) {
      const uint32_t mk = find_masked(l, status);
      scores<L>(l, mk, softmax, s, m);
      const float z = lanes_sum<L>(pairs_sum(s));
      iz = z > 0.f ? rcp_approx(z) : 0.f;
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
    const bool ratio = a.renormalize && (softmax || top < -40.f);
    const float shift = ratio ? top : m;
    float sj[kPer], dj[kPer];
    float sum = 0.f, dot = 0.f;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const float y = exp2_approx((ratio || softmax ? x[q] - shift : -x[q]) * kLog2e);
      sj[q] = ej[q] < 0 ? 0.f : ratio ? y : softmax ? y * iz : rcp_approx(1.f + y);
      sum += sj[q];
      dj[q] = softmax ? 1.f : rcp_approx(1.f + exp2_approx(x[q] * kLog2e));  // 1 - s
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
      float ph = 0.f;
      if (aux) {
        uint64_t acc = f32x2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kV / 2; ++i) acc = f32x2_fma(s[i], h[i], acc);
        float u, v;
        f32x2_get(acc, u, v);
        ph = lanes_sum<L>(u + v) * iz;
      }
      if (softmax && !a.renormalize) ph += dot;
      const float c = -ph * iz;
#pragma unroll
      for (int i = 0; i < kV / 2; ++i) {
        const uint64_t d = f32x2_fma(h[i], f32x2(iz, iz), f32x2(c, c));
        const uint64_t p = softmax ? s[i] : f32x2_fma(f32x2_mul(s[i], f32x2(-1.f, -1.f)), s[i], s[i]);
        grad[i] = f32x2_mul(p, d);
      }
    }
    // the chosen experts' part is added in shared memory
    float* row = sh_row[warp][tok];
    *reinterpret_cast<ulonglong2*>(row + sub * kV) = make_ulonglong2(grad[0], grad[1]);
    *reinterpret_cast<ulonglong2*>(row + sub * kV + 4) = make_ulonglong2(grad[2], grad[3]);
    __syncwarp();
#pragma unroll
    for (int q = 0; q < kPer; ++q)
      if (ej[q] >= 0) row[ej[q]] += dj[q];
    __syncwarp();
    if (valid) {
      float* out = a.grad_logits + t * E;
      const int e0 = sub * kV;
      if ((E & 3) == 0) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
          if (e0 + 4 * q < E)
            __stcs(reinterpret_cast<float4*>(out + e0 + 4 * q),
                   *reinterpret_cast<const float4*>(row + e0 + 4 * q));
      } else {
#pragma unroll
        for (int i = 0; i < kV; ++i)
          if (e0 + i < E) out[e0 + i] = row[e0 + i];
      }
    }
  }
}

int lanes_of(int E) {
  int L = 2;
  while (L * kV < E) L <<= 1;
  return L;
}

}  // namespace

int route_grouped_blocks(int T, int E) {
  const int per_block = kWarps * (32 / lanes_of(E));
  const int n = (T + per_block - 1) / per_block;
  return n < kGroupedMaxBlocks ? n : kGroupedMaxBlocks;
}

cudaError_t launch_route_grouped(const GroupedArgs& a, cudaStream_t st) {
  const dim3 grid(route_grouped_blocks(a.T, a.E)), block(kThreads);
  switch (lanes_of(a.E)) {
    case 2: return launch_pdl(route_grouped_kernel<2>, grid, block, 0, st, a);
    case 4: return launch_pdl(route_grouped_kernel<4>, grid, block, 0, st, a);
    case 8: return launch_pdl(route_grouped_kernel<8>, grid, block, 0, st, a);
    case 16: return launch_pdl(route_grouped_kernel<16>, grid, block, 0, st, a);
    default: return launch_pdl(route_grouped_kernel<32>, grid, block, 0, st, a);
  }
}

cudaError_t launch_route_grouped_bwd(const GroupedBwdArgs& a, cudaStream_t st) {
  const dim3 grid(route_grouped_blocks(a.T, a.E)), block(kThreads);
  switch (lanes_of(a.E)) {
    case 2: return launch_pdl(route_grouped_bwd_kernel<2>, grid, block, 0, st, a);
    case 4: return launch_pdl(route_grouped_bwd_kernel<4>, grid, block, 0, st, a);
    case 8: return launch_pdl(route_grouped_bwd_kernel<8>, grid, block, 0, st, a);
    case 16: return launch_pdl(route_grouped_bwd_kernel<16>, grid, block, 0, st, a);
    default: return launch_pdl(route_grouped_bwd_kernel<32>, grid, block, 0, st, a);
  }
}

}  // namespace moe
