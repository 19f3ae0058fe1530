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

// Keys order selection values as unsigned integers: the float's bits made
// monotonic, their lowest 3 bits replaced by 7 - slot so that a lane's keys
// differ and carry the slot. Smaller keys mark experts that come after every
// regular one: masked experts of kept groups by index (16 + 255 - e, whose
// lowest 3 bits are 7 - slot too), then experts of other groups (7 - slot).
__device__ __forceinline__ uint32_t key_masked(int e) { return 16u + static_cast<uint32_t>(255 - e); }
__device__ __forceinline__ uint32_t key_of(float c, int slot) {
  const uint32_t u = __float_as_uint(c);
  const uint32_t o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return (o & ~7u) | static_cast<uint32_t>(7 - slot);
}
__device__ __forceinline__ bool key_regular(uint32_t key) { return key >= 512u; }
__device__ __forceinline__ float key_value(uint32_t key) {
  const uint32_t o = key & ~7u;
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

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
  return lanes_reduce<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int L>
__device__ __forceinline__ uint32_t lanes_max_u32(uint32_t v) {
  if constexpr (L == 32) return __reduce_max_sync(kFull, v);
  return lanes_reduce<L>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

__device__ __forceinline__ bool masked(float l) { return !(fabsf(l) < CUDART_INF_F); }

// The lane's 8 logits of row t; masked past E or T.
template <int L>
__device__ __forceinline__ void load_row(const float* __restrict__ logits, int64_t t, bool valid,
                                         int E, int sub, float (&l)[kV]) {
  const float* row = logits + t * E;
  const int e0 = sub * kV;
  if ((E & 3) == 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float4 v = make_float4(-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F);
      if (valid && e0 + 4 * h < E) v = __ldg(reinterpret_cast<const float4*>(row + e0 + 4 * h));
      l[4 * h] = v.x;
      l[4 * h + 1] = v.y;
      l[4 * h + 2] = v.z;
      l[4 * h + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kV; ++i) l[i] = valid && e0 + i < E ? __ldg(row + e0 + i) : -CUDART_INF_F;
  }
}

// ------------------------------------------------------------- fp64 ----
// The same token decided in fp64: slot j's expert ends up in lane j of the
// token's lanes (and in every 8th lane when L < 8, see `pick`).
template <int L>
__device__ __noinline__ void route_exact(const GroupedArgs& a, const float (&l)[kV], int sub,
                                         double* cs, double* gv, int* pick) {
  double c[kV];
  double m = -CUDART_INF;
  if (a.score == MOE_SCORE_SOFTMAX) {
#pragma unroll
    for (int i = 0; i < kV; ++i)
      if (!masked(l[i])) m = fmax(m, static_cast<double>(l[i]));
    m = lanes_reduce<L>(m, [](double x, double y) { return fmax(x, y); });
  }
  double z = 0.0;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const double x = l[i];
    if (masked(l[i])) {
      c[i] = 0.0;
    } else if (a.score == MOE_SCORE_SOFTMAX) {
      c[i] = exp(x - m);
      z += c[i];
    } else {
      c[i] = 1.0 / (1.0 + exp(-x));
    }
  }
  if (a.score == MOE_SCORE_SOFTMAX) {
    z = lanes_reduce<L>(z, [](double x, double y) { return x + y; });
#pragma unroll
    for (int i = 0; i < kV; ++i) c[i] = z > 0.0 ? c[i] / z : 0.0;
  }
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int e = sub * kV + i;
    if (masked(l[i])) c[i] = -CUDART_INF;
    else if (a.bias != nullptr && e < a.E) c[i] += static_cast<double>(a.bias[e]);
    if (e < a.E) cs[e] = c[i];
  }
  __syncwarp();
  uint32_t kept = 0xffffffffu;
  const int S = a.E / a.n_groups;
  if (a.n_groups > 1) {
    for (int g = sub; g < a.n_groups; g += L) {
      double v1 = -CUDART_INF, v2 = -CUDART_INF;
      for (int q = 0; q < S; ++q) {
        const double v = cs[g * S + q];
        if (v > v1) {
          v2 = v1;
          v1 = v;
        } else if (v > v2) {
          v2 = v;
        }
      }
      gv[g] = a.group_top == 2 ? v1 + v2 : v1;
    }
    __syncwarp();
    kept = 0u;
    for (int g = sub; g < a.n_groups; g += L) {
      int ahead = 0;
      for (int h = 0; h < a.n_groups; ++h)
        ahead += (gv[h] > gv[g] || (gv[h] == gv[g] && h < g)) ? 1 : 0;
      if (ahead < a.topk_groups) kept |= 1u << g;
    }
    kept = lanes_reduce<L>(kept, [](uint32_t x, uint32_t y) { return x | y; });
  }
  uint32_t left = 0;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int e = sub * kV + i;
    if (e < a.E && ((kept >> (a.n_groups > 1 ? e / S : 0)) & 1u)) left |= 1u << i;
  }
  for (int j = 0; j < a.k; ++j) {
    double best = -CUDART_INF;
    int at = 1 << 20;
#pragma unroll
    for (int i = 0; i < kV; ++i)
      if ((left >> i) & 1u) {
        const int e = sub * kV + i;
        if (at == (1 << 20) || c[i] > best) {
          best = c[i];
          at = e;
        }
      }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) {
      const double ob = __shfl_xor_sync(kFull, best, o);
      const int oa = __shfl_xor_sync(kFull, at, o);
      const bool take = oa != (1 << 20) && (at == (1 << 20) || ob > best || (ob == best && oa < at));
      if (take) {
        best = ob;
        at = oa;
      }
    }
    if (at / kV == sub) left &= ~(1u << (at % kV));
    if (sub == 0) pick[j] = at;
  }
  __syncwarp();
}

// ------------------------------------------------------------- kernel ----

template <int L>
__global__ void __launch_bounds__(kThreads) route_grouped_kernel(GroupedArgs a) {
  constexpr int kTok = 32 / L;                       // tokens per warp
  constexpr int kGmax = L * kV < 32 ? L * kV : 32;   // groups per token at most
  __shared__ double sh_c[kWarps][kTok * L * kV];
  __shared__ double sh_g[kWarps][kTok * kGmax];
  __shared__ int sh_pick[kWarps][kTok * kMaxTopK];
  __shared__ float sh_p[kWarps][kTok][L * kV];
  __shared__ int sh_cnt[L * kV];
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sub = lane & (L - 1), tok = lane / L;
  const int E = a.E, G = a.n_groups, S = E / G;
  const bool stats = a.tile_cnt != nullptr;
  double* cs = sh_c[warp] + tok * L * kV;
  float* csf = reinterpret_cast<float*>(cs);
  double* gv = sh_g[warp] + tok * kGmax;
  float* gvf = reinterpret_cast<float*>(gv);
  int* pick = sh_pick[warp] + tok * kMaxTopK;
  if (stats)
    for (int i = tid; i < L * kV; i += kThreads) sh_cnt[i] = 0;
  if (blockIdx.x == 0 && tid == 0 && a.ticket != nullptr) *a.ticket = 0u;
  __syncthreads();
  float b[kV], psum[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int e = sub * kV + i;
    b[i] = a.bias != nullptr && e < E ? a.bias[e] : 0.f;
    psum[i] = 0.f;
  }
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  uint32_t bits = 0;
  const int per_pass = gridDim.x * kWarps * kTok;
  for (int base = (blockIdx.x * kWarps + warp) * kTok; base < a.T; base += per_pass) {
    const int t = base + tok;
    const bool valid = t < a.T;
    float l[kV], s[kV];
    load_row<L>(a.logits, valid ? t : 0, valid, E, sub, l);
    // scores
    float m = 0.f;
    if (softmax) {
      m = -CUDART_INF_F;
#pragma unroll
      for (int i = 0; i < kV; ++i)
        if (!masked(l[i])) m = fmaxf(m, l[i]);
      m = lanes_max<L>(m);
    }
    float z = 0.f, smax = 0.f;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      if (masked(l[i])) {
        if (valid && sub * kV + i < E && l[i] != -CUDART_INF_F) bits |= MOE_DEV_NONFINITE;
        s[i] = 0.f;
      } else {
        s[i] = softmax ? __expf(l[i] - m) : __fdividef(1.f, 1.f + __expf(-l[i]));
      }
      z += s[i];
      smax = fmaxf(smax, s[i]);
    }
    z = lanes_sum<L>(z);
    if (softmax) {
      const float iz = z > 0.f ? 1.f / z : 0.f;
#pragma unroll
      for (int i = 0; i < kV; ++i) s[i] *= iz;
      smax = iz;  // exp(0) / z
    } else {
      smax = lanes_max<L>(smax);
    }
    // Selection values. A score's error is within 2^-21 of the row's largest
    // score (2^-17 where all logits are far below zero and the exponent's
    // rounding counts), the sum adds its own rounding, and the keys drop 3
    // bits (2^-20): values closer than `near` are decided in fp64.
    float c[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) c[i] = masked(l[i]) ? -CUDART_INF_F : s[i] + b[i];
    const float near_abs = smax * (softmax || smax > 1e-3f ? 0x1p-20f : 0x1p-16f);
    auto near = [&](float x, float y) {
      return fabsf(x - y) <= near_abs + 0x1p-19f * fmaxf(fabsf(x), fabsf(y));
    };
    bool unsure = smax < 1e-30f;
    uint32_t kept = 0xffffffffu;
    if (G > 1) {
#pragma unroll
      for (int i = 0; i < kV; ++i)
        if (sub * kV + i < E) csf[sub * kV + i] = c[i];
      __syncwarp();
      for (int g = sub; g < G; g += L) {
        float v1 = -CUDART_INF_F, v2 = -CUDART_INF_F;
        for (int q = 0; q < S; ++q) {
          const float v = csf[g * S + q];
          v2 = fmaxf(v2, fminf(v, v1));
          v1 = fmaxf(v1, v);
        }
        gvf[g] = a.group_top == 2 ? v1 + v2 : v1;
      }
      __syncwarp();
      kept = 0u;
      for (int g = sub; g < G; g += L) {
        const float v = gvf[g];
        int ahead = 0, sure = 0, maybe = 0;
        for (int h = 0; h < G; ++h) {
          const float o = gvf[h];
          ahead += (o > v || (o == v && h < g)) ? 1 : 0;
          const bool close = v != -CUDART_INF_F && o != -CUDART_INF_F && near(o, v);
          sure += (o > v && !close) ? 1 : 0;
          maybe += (h != g && (o > v || close)) ? 1 : 0;
        }
        if (ahead < a.topk_groups) kept |= 1u << g;
        unsure |= v != -CUDART_INF_F && sure < a.topk_groups && maybe >= a.topk_groups;
      }
      kept = lanes_reduce<L>(kept, [](uint32_t x, uint32_t y) { return x | y; });
      __syncwarp();
    }
    uint32_t key[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int e = sub * kV + i;
      const bool in = e < E && ((kept >> (G > 1 ? e / S : 0)) & 1u);
      key[i] = !in ? static_cast<uint32_t>(7 - i)
                   : c[i] == -CUDART_INF_F ? key_masked(e)
                                           : key_of(c[i], i);
    }
    // the lane's keys, largest first (Batcher's odd-even merge sort of 8)
    auto swap = [&](int x, int y) {
      const uint32_t hi = max(key[x], key[y]), lo = min(key[x], key[y]);
      key[x] = hi;
      key[y] = lo;
    };
    swap(0, 1); swap(2, 3); swap(4, 5); swap(6, 7);
    swap(0, 2); swap(1, 3); swap(4, 6); swap(5, 7);
    swap(1, 2); swap(5, 6);
    swap(0, 4); swap(1, 5); swap(2, 6); swap(3, 7);
    swap(2, 4); swap(3, 5);
    swap(1, 2); swap(3, 4); swap(5, 6);
    uint32_t prev = 0;
    for (int j = 0; j <= a.k; ++j) {
      const uint32_t best = lanes_max_u32<L>(key[0]);
      if (j > 0 && key_regular(prev) && key_regular(best))
        unsure |= near(key_value(prev), key_value(best));
      prev = best;
      const uint32_t owners = __ballot_sync(kFull, key[0] == best);
      const int first = __ffs(static_cast<int>(L == 32 ? owners : (owners >> (tok * L)) & ((1u << (L & 31)) - 1u))) - 1;
      if (sub == first && j < a.k) {
        pick[j] = sub * kV + 7 - static_cast<int>(best & 7u);
#pragma unroll
        for (int i = 0; i + 1 < kV; ++i) key[i] = key[i + 1];
        key[kV - 1] = 0u;
      }
    }
    __syncwarp();
    unsure = unsure && valid;
    // every lane of the token has to agree; all tokens of the warp follow
    if (__any_sync(kFull, unsure)) {
      const uint32_t who = __ballot_sync(kFull, unsure);
      const bool mine = L == 32 ? who != 0 : ((who >> (tok * L)) & ((1u << (L & 31)) - 1u)) != 0;
      int keep[kMaxTopK];
#pragma unroll
      for (int j = 0; j < kMaxTopK; ++j) keep[j] = j < a.k ? pick[j] : 0;
      __syncwarp();
      route_exact<L>(a, l, sub, cs, gv, pick);
      if (!mine && sub == 0) {
#pragma unroll
        for (int j = 0; j < kMaxTopK; ++j)
          if (j < a.k) pick[j] = keep[j];
      }
      __syncwarp();
    }
    // weights of the chosen, from the logits again (cached): slot j in lane j
    // of the token, or two passes and more where L < k
    float den = 1.f;
    float top = -CUDART_INF_F;
    for (int j = sub; j < a.k; j += L) {
      const float x = valid ? a.logits[static_cast<int64_t>(t) * E + pick[j]] : 0.f;
      if (!masked(x)) top = fmaxf(top, x);
    }
    top = lanes_max<L>(top);
    // Renormalised weights are ratios: softmax scores are taken relative to
    // the largest chosen logit, and so are sigmoid scores far below zero
    // (where 1 + exp(l) is 1), which would underflow.
    const bool ratio = a.renormalize && (softmax || top < -40.f);
    auto score_of = [&](float x) {
      if (masked(x)) return 0.f;
      if (ratio) return expf(x - top);
      return softmax ? expf(x - m) / z : 1.f / (1.f + expf(-x));
    };
    if (a.renormalize) {
      float sum = 0.f;
      for (int j = sub; j < a.k; j += L)
        sum += score_of(valid ? a.logits[static_cast<int64_t>(t) * E + pick[j]] : 0.f);
      den = lanes_sum<L>(sum);
    }
    for (int j = sub; j < a.k; j += L) {
      if (valid) {
        const int e = pick[j];
        const float w = score_of(a.logits[static_cast<int64_t>(t) * E + e]);
        a.topk_idx[static_cast<int64_t>(t) * a.k + j] = e;
        a.topk_w[static_cast<int64_t>(t) * a.k + j] = den > 0.f ? a.scale * w / den : 0.f;
        if (stats) atomicAdd(&sh_cnt[e], 1);
      }
    }
    if (stats) {
      const float iz = softmax ? 1.f : (z > 0.f ? 1.f / z : 0.f);
#pragma unroll
      for (int i = 0; i < kV; ++i) psum[i] += valid ? s[i] * iz : 0.f;
    }
    __syncwarp();
  }
  if (bits) atomicOr(a.dev_status, bits);
  if (stats) {
#pragma unroll
    for (int i = 0; i < kV; ++i) sh_p[warp][tok][sub * kV + i] = psum[i];
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
__global__ void __launch_bounds__(kThreads) route_grouped_bwd_kernel(GroupedBwdArgs a) {
  constexpr int kTok = 32 / L;
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sub = lane & (L - 1), tok = lane / L;
  const int E = a.E;
  const bool softmax = a.score == MOE_SCORE_SOFTMAX, aux = a.grad_aux != nullptr;
  const bool need_p = aux || (softmax && !a.renormalize);  // the whole row's scores
  float h[kV];
  if (aux) {
    const float f = *a.grad_aux * (static_cast<float>(E) / (static_cast<float>(a.T) * static_cast<float>(a.T) * static_cast<float>(a.k)));
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int e = sub * kV + i;
      h[i] = e < E ? f * static_cast<float>(a.routed[e]) : 0.f;
    }
  }
  const int per_pass = gridDim.x * kWarps * kTok;
  for (int base = (blockIdx.x * kWarps + warp) * kTok; base < a.T; base += per_pass) {
    const int t = base + tok;
    const bool valid = t < a.T;
    float l[kV], s[kV], grad[kV];
    load_row<L>(a.logits, valid ? t : 0, valid, E, sub, l);
    float m = -CUDART_INF_F, z = 0.f;
    if (softmax) {
#pragma unroll
      for (int i = 0; i < kV; ++i)
        if (!masked(l[i])) m = fmaxf(m, l[i]);
      m = lanes_max<L>(m);
    }
    if (need_p) {
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        s[i] = masked(l[i]) ? 0.f
                            : softmax ? __expf(l[i] - m) : __fdividef(1.f, 1.f + __expf(-l[i]));
        z += s[i];
      }
      z = lanes_sum<L>(z);
    }
    const float iz = z > 0.f ? 1.f / z : 0.f;
    // the chosen slots, in lanes sub, sub + L, ...
    constexpr int kPer = (kMaxTopK + L - 1) / L;
    int ej[kPer];
    float sj[kPer], slope[kPer], gj[kPer];
    float top = -CUDART_INF_F;
    float x[kPer];
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int j = sub + q * L;
      ej[q] = -1;
      gj[q] = 0.f;
      x[q] = -CUDART_INF_F;
      if (valid && j < a.k) {
        ej[q] = a.topk_idx[static_cast<int64_t>(t) * a.k + j];
        gj[q] = a.grad_w[static_cast<int64_t>(t) * a.k + j];
        if (ej[q] < 0 || ej[q] >= E) ej[q] = -1;
        else x[q] = a.logits[static_cast<int64_t>(t) * E + ej[q]];
        if (masked(x[q])) ej[q] = -1;
        else top = fmaxf(top, x[q]);
      }
    }
    top = lanes_max<L>(top);
    const bool ratio = a.renormalize && (softmax || top < -40.f);
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      slope[q] = softmax ? 1.f : 1.f / (1.f + expf(x[q]));  // 1 - s
      sj[q] = ej[q] < 0 ? 0.f
                        : ratio ? expf(x[q] - top)
                                : softmax ? expf(x[q] - m) * iz : 1.f / (1.f + expf(-x[q]));
      sum += sj[q];
    }
    float dj[kPer];
    float dot = 0.f;
    if (a.renormalize) {
      sum = lanes_sum<L>(sum);
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        sj[q] *= inv;
        dot += sj[q] * gj[q];
      }
      dot = lanes_sum<L>(dot);
#pragma unroll
      for (int q = 0; q < kPer; ++q) dj[q] = a.scale * sj[q] * slope[q] * (gj[q] - dot);
      dot = 0.f;
    } else {
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        dj[q] = a.scale * sj[q] * slope[q] * gj[q];
        dot += softmax ? dj[q] : 0.f;
      }
      dot = lanes_sum<L>(dot);
    }
    // the whole row's part
    float ph = 0.f;
    if (aux) {
#pragma unroll
      for (int i = 0; i < kV; ++i) ph += s[i] * iz * h[i];
      ph = lanes_sum<L>(ph);
    }
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      grad[i] = 0.f;
      if (need_p) {
        const float p = s[i] * iz;
        if (softmax && !a.renormalize) grad[i] -= p * dot;
        if (aux) grad[i] += p * (softmax ? 1.f : 1.f - s[i]) * (h[i] - ph);
      }
    }
#pragma unroll
    for (int q = 0; q < kPer; ++q)
      for (int j = 0; j < L && q * L + j < a.k; ++j) {
        const int e = __shfl_sync(kFull, ej[q], tok * L + j);
        const float d = __shfl_sync(kFull, dj[q], tok * L + j);
#pragma unroll
        for (int i = 0; i < kV; ++i) grad[i] += e == sub * kV + i ? d : 0.f;
      }
    if (valid) {
      float* row = a.grad_logits + static_cast<int64_t>(t) * E;
      const int e0 = sub * kV;
      if ((E & 3) == 0) {
#pragma unroll
        for (int q = 0; q < 2; ++q)
          if (e0 + 4 * q < E)
            *reinterpret_cast<float4*>(row + e0 + 4 * q) =
                make_float4(grad[4 * q], grad[4 * q + 1], grad[4 * q + 2], grad[4 * q + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < kV; ++i)
          if (e0 + i < E) row[e0 + i] = grad[i];
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
