// What lies between two blocks of a model, in one pass over a token, and its
// gradient. With y_j the rows of the block's output that belong to a token
// (expert rows by dest_row, or the token's own), w_j their weights, N the width:
//
//   c   = sum_j w_j y_j                        (the combine)
//   n   = c r_c post,  r_c = 1 / sqrt(mean(c^2) + eps)   (post_norm; else n = c post)
//   out = s residual + gate n                  (gate: one value per token)
//   xn  = out r_h pre, r_h = 1 / sqrt(mean(out^2) + eps) (the next block's norm)
//
// out enters the second norm before it is rounded to bf16. The gradient takes
// the stream as it was stored, h:
//
//   v = pre g_xn,  G = g_out + r_h (v - h r_h^2 mean(v h)),  g_residual = s G
//   g_pre = sum_t g_xn h r_h,  g_gate = sum_i G post c r_c,  g_post = sum_t gate G c r_c
//   u = gate G post,  g_c = r_c (u - c r_c^2 mean(u c))   (post_norm; else g_c = u)
//   g_y[dest_j] = w_j g_c,  g_w_j = <g_c, y_j>
//
// All sums are fp32 in a fixed order; every value is rounded once, when it is
// stored. Both kernels read a token's rows once from HBM and are bound by their
// bytes, the gradient nearly so: 32768 tokens of 4096 with two rows each, a tenth of
// them dropped, take 197 us (6.3 TB/s of DRAM traffic; a copy has 6.7) and 356 us (5.6
// TB/s); 16383 of 2048 with six rows 98 and 200 us; one token 3.5 us. In
// the gradient 16 warps to an SM issue in half of the clocks; the rest is the
// latency of shared memory and of three sums over the block.
#include "moe_internal.h"
#include "moe_ptx.cuh"

namespace moe {

namespace {

// Values are worked on as pairs in 64-bit registers, one instruction for two.
using F2 = uint64_t;

__device__ __forceinline__ void unpack8(const uint4& v, F2 (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = f32x2(bf16_lo(w[i]), bf16_hi(w[i]));
}

__device__ __forceinline__ uint32_t pack2(F2 v) {
  float lo, hi;
  f32x2_get(v, lo, hi);
  return pack_bf16x2(lo, hi);
}

__device__ __forceinline__ uint4 pack8(const F2 (&f)[4]) {
  return make_uint4(pack2(f[0]), pack2(f[1]), pack2(f[2]), pack2(f[3]));
}

__device__ __forceinline__ float sum2(F2 v) {
  float lo, hi;
  f32x2_get(v, lo, hi);
  return lo + hi;
}

// 8 fp32 weights from column 8 * i, or ones.
__device__ __forceinline__ void weight8(const float* w, int i, F2 (&f)[4]) {
  if (w == nullptr) {
#pragma unroll
    for (int q = 0; q < 4; ++q) f[q] = f32x2(1.f, 1.f);
    return;
  }
  const float4 a = reinterpret_cast<const float4*>(w)[2 * i];
  const float4 b = reinterpret_cast<const float4*>(w)[2 * i + 1];
  f[0] = f32x2(a.x, a.y);
  f[1] = f32x2(a.z, a.w);
  f[2] = f32x2(b.x, b.y);
  f[3] = f32x2(b.z, b.w);
}

// A token's group is one warp (G = 32) or the whole block of G threads. Cross-warp
// scratch of such a block: three areas of 8 values a warp, taken in turn. A call's
// area is written again three calls later, after two barriers that every reader of
// the first has reached.
template <int G>
struct Scratch {
  static constexpr int W = G / 32;
  float v[3][8 * W];
  __device__ __forceinline__ static float warps(const float* r) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < W; w += 4) {
      const float4 q = *reinterpret_cast<const float4*>(r + w);
      s += (q.x + q.y) + (q.z + q.w);
    }
    return s;
  }
};

// Sums of M values over a token's group, in every thread.
template <int G, int M>
__device__ __forceinline__ void group_sum(float (&v)[M], Scratch<G>& red, int& turn) {
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[m] += __shfl_xor_sync(0xffffffffu, v[m], o);
  if constexpr (G > 32) {
    constexpr int W = G / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* r = red.v[turn];
    turn = turn == 2 ? 0 : turn + 1;
    if (lane == 0) {
#pragma unroll
      for (int m = 0; m < M; ++m) r[m * W + warp] = v[m];
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] = red.warps(r + m * W);
  }
}

// Sums of 8 values over the group, value j in thread j of it. A warp halves the
// values it still holds with each of the first three exchanges.
template <int G>
__device__ __forceinline__ float group_sum8(float (&v)[8], Scratch<G>& red, int& turn) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 4, o = 16; n > 0; n >>= 1, o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  float s = v[0];
  s += __shfl_xor_sync(0xffffffffu, s, 2);
  s += __shfl_xor_sync(0xffffffffu, s, 1);
  // lanes 4j .. 4j+3 hold value j
  if constexpr (G > 32) {
    constexpr int W = G / 32;
    const int warp = threadIdx.x >> 5;
    float* r = red.v[turn];
    turn = turn == 2 ? 0 : turn + 1;
    if ((lane & 3) == 0) r[(lane >> 2) * W + warp] = s;
    __syncthreads();
    return threadIdx.x < 8 ? red.warps(r + threadIdx.x * W) : 0.f;
  } else {
    return __shfl_sync(0xffffffffu, s, 4 * (lane & 7));
  }
}

// A lane's slot of a token: row of y (or -1) and weight, for lanes below k.
struct Slot {
  int row;
  float w;
};
__device__ __forceinline__ Slot load_slot(const BlockArgs& a, int64_t t, int lane) {
  Slot s{-1, 0.f};
  if (t < a.T && lane < a.k) {
    const int64_t i = t * a.k + lane;
    s.row = a.dest_row != nullptr ? a.dest_row[i] : static_cast<int>(t);
    s.w = a.topk_w != nullptr ? a.topk_w[i] : 1.f;
    if (s.row < 0 || s.row >= a.rows) s.row = -1;  // only rows of the buffer are touched
  }
  return s;
}

// Asks L2 to fetch a row of H bf16 values.
__device__ __forceinline__ void prefetch_row(const uint16_t* base, int64_t row, int H) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(base + row * H), "r"(2 * H)
               : "memory");
}

// c[v][8] = sum over the slots, ascending, of w_j y_j; KU rows in flight together.
template <int G, int NV, int KU>
__device__ __forceinline__ void combine_rows(const BlockArgs& a, const Slot& s, int gt, int nvec,
                                             F2 (&c)[NV][4]) {
  const uint4* yv = reinterpret_cast<const uint4*>(a.y);
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int q = 0; q < 4; ++q) c[v][q] = 0;
  for (int j0 = 0; j0 < a.k; j0 += KU) {
    uint4 b[KU][NV];
    int row[KU];
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      row[u] = __shfl_sync(0xffffffffu, s.row, j0 + u);  // lanes from k up hold no row
      if (row[u] >= 0) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int i = gt + G * v;
          b[u][v] = i < nvec ? __ldg(yv + static_cast<size_t>(row[u]) * nvec + i)
                             : make_uint4(0, 0, 0, 0);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      const float w = __shfl_sync(0xffffffffu, s.w, j0 + u);
      if (row[u] >= 0) {
        const F2 ww = f32x2(w, w);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          F2 f[4];
          unpack8(b[u][v], f);
#pragma unroll
          for (int q = 0; q < 4; ++q) c[v][q] = f32x2_fma(ww, f[q], c[v][q]);
        }
      }
    }
  }
}

template <int NV>
__device__ __forceinline__ float square_sum(const F2 (&h)[NV][4]) {
  F2 ss = 0;
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int q = 0; q < 4; ++q) ss = f32x2_fma(h[v][q], h[v][q], ss);
  return sum2(ss);
}

// G threads to a token, NV vectors of 8 columns to a thread (vector gt + G v):
// G * 8 * NV >= H. Blocks hold max(1, 128 / G) tokens. While a token is worked
// on, L2 is asked for the rows of the next one: without that a block's loads and
// its sums took turns (306 us for 32768 tokens of 4096 with two rows each, 207
// with it, 6.2 TB/s).
template <int G, int NV, int KU, int MB>
__global__ void __launch_bounds__(G == 32 ? 128 : G, MB) block_kernel(BlockArgs a) {
  constexpr int kPer = G == 32 ? 4 : 1;
  __shared__ __align__(16) Scratch<G> red;
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int gt = threadIdx.x % G;
  const int nvec = a.H >> 3;
  const float inv_h = 1.f / static_cast<float>(a.H);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kPer;
  int turn = 0;
  int64_t t = static_cast<int64_t>(blockIdx.x) * kPer + threadIdx.x / G;
  Slot s{-1, 0.f}, next{-1, 0.f}, next2{-1, 0.f};
  if (a.y != nullptr) {
    s = load_slot(a, t, lane);
    next = load_slot(a, t + step, lane);
  }
  for (; t < a.T; t += step, s = next, next = next2) {
    uint4 res[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = gt + G * v;
      // not by the read-only path: out may be the residual
      res[v] = i < nvec ? reinterpret_cast<const uint4*>(a.residual)[t * nvec + i]
                        : make_uint4(0, 0, 0, 0);
    }
    float gate = 1.f;
    if (a.gate != nullptr) gate = a.gate[t];
    F2 h[NV][4];
    if (gt < 32 && t + step < a.T) {
      if (next.row >= 0) prefetch_row(a.y, next.row, a.H);
      if (lane == 8) prefetch_row(a.residual, t + step, a.H);
    }
    const F2 scale = f32x2(a.scale, a.scale);
    if (a.y != nullptr) {
      next2 = load_slot(a, t + 2 * step, lane);
      combine_rows<G, NV, KU>(a, s, gt, nvec, h);
      float r = gate;
      if (a.post_norm) {
        float ss[1] = {square_sum<NV>(h)};
        group_sum<G, 1>(ss, red, turn);
        r *= rsqrtf(fmaf(ss[0], inv_h, a.eps));
      }
      const F2 rr = f32x2(r, r);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int i = gt + G * v;
        if (i < nvec) {
          F2 w[4], f[4];
          weight8(a.post_weight, i, w);
          unpack8(res[v], f);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            h[v][q] = f32x2_fma(scale, f[q], f32x2_mul(f32x2_mul(h[v][q], rr), w[q]));
        }
      }
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        unpack8(res[v], h[v]);
#pragma unroll
        for (int q = 0; q < 4; ++q) h[v][q] = f32x2_mul(scale, h[v][q]);
      }
    }
    if (a.out != nullptr) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int i = gt + G * v;
        if (i < nvec) reinterpret_cast<uint4*>(a.out)[t * nvec + i] = pack8(h[v]);
      }
    }
    if (a.xn != nullptr) {
      float ss[1] = {square_sum<NV>(h)};
      group_sum<G, 1>(ss, red, turn);
      const float r = rsqrtf(fmaf(ss[0], inv_h, a.eps));
      const F2 rr = f32x2(r, r);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int i = gt + G * v;
        if (i < nvec) {
          F2 w[4], f[4];
          weight8(a.pre_weight, i, w);
#pragma unroll
          for (int q = 0; q < 4; ++q) f[q] = f32x2_mul(f32x2_mul(h[v][q], rr), w[q]);
          reinterpret_cast<uint4*>(a.xn)[t * nvec + i] = pack8(f);
        }
      }
    }
  }
}

__device__ __forceinline__ void cp_async_16(uint4* dst, const uint4* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Layout as block_kernel's. A token's rows (g_out, g_xn, h and, kStageY, its y_j)
// are copied to shared memory by the threads that will read them, each its own
// columns: no barrier stands between a copy and its use, and with two stages the
// next token's rows arrive while this one is worked on. What this needs less of
// than loads into registers is registers, so that the three sums a token takes
// (each a barrier) and the second look at y_j wait on shared memory alone.
// Sums over tokens (g_post, g_pre) stay in registers, one column of a thread's
// each, until the block's last token; the groups' partial sums [groups][2][H]
// are added by column_sum_kernel.
template <int G, int NV, int KMAX, bool kStaged, bool kFull, int MB>
__global__ void __launch_bounds__(G == 32 ? 128 : G, MB)
    block_bwd_kernel(BlockArgs a, BlockGrads g, int stages) {
  constexpr int kPer = G == 32 ? 4 : 1;
  __shared__ __align__(16) Scratch<G> red;
  extern __shared__ uint4 dyn[];
  const int lane = threadIdx.x & 31;
  const int gt = threadIdx.x % G;
  const int nvec = kFull ? G * NV : a.H >> 3;
  const int stage_vecs = (3 + (kStaged ? a.k : 0)) * nvec;
  const float inv_h = 1.f / static_cast<float>(a.H);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kPer;
  int64_t t = static_cast<int64_t>(blockIdx.x) * kPer + threadIdx.x / G;
  uint4* const ring = dyn + (kStaged ? 4 * nvec : 0) +
                      static_cast<size_t>(threadIdx.x / G) * stages * stage_vecs;
  int turn = 0;
  grid_dependency_wait();
  grid_launch_dependents();
  auto weights = [&](bool pre, int i, F2 (&f)[4]) {
    if constexpr (kStaged) {
      const ulonglong2* w = reinterpret_cast<const ulonglong2*>(dyn) + (pre ? 2 * nvec : 0) + 2 * i;
      const ulonglong2 x = w[0], y = w[1];
      f[0] = x.x;
      f[1] = x.y;
      f[2] = y.x;
      f[3] = y.y;
    } else {
      weight8(pre ? a.pre_weight : a.post_weight, i, f);
    }
  };
  if (kStaged) {
    float* w = reinterpret_cast<float*>(dyn);
    for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
      w[i] = a.post_weight != nullptr ? a.post_weight[i] : 1.f;
      w[a.H + i] = a.pre_weight != nullptr ? a.pre_weight[i] : 1.f;
    }
    __syncthreads();
  }
  // this thread's columns of token t's rows into a stage, as one group
  auto fetch = [&](int64_t tok, const Slot& sl, uint4* st) {
    if (tok < a.T) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int i = gt + G * v;
        if (kFull || i < nvec) {
          const int64_t at = tok * nvec + i;
          if (g.out != nullptr) cp_async_16(st + i, reinterpret_cast<const uint4*>(g.out) + at);
          if (g.xn != nullptr) {
            cp_async_16(st + nvec + i, reinterpret_cast<const uint4*>(g.xn) + at);
            cp_async_16(st + 2 * nvec + i, reinterpret_cast<const uint4*>(g.h) + at);
          }
        }
      }
      if constexpr (kStaged) {
        if (a.y != nullptr) {
#pragma unroll
          for (int j = 0; j < KMAX; ++j) {
            const int row = __shfl_sync(0xffffffffu, sl.row, j);  // lanes from k up hold none
            if (row >= 0) {
#pragma unroll
              for (int v = 0; v < NV; ++v) {
                const int i = gt + G * v;
                if (kFull || i < nvec)
                  cp_async_16(st + (3 + j) * nvec + i, reinterpret_cast<const uint4*>(a.y) +
                                                           static_cast<size_t>(row) * nvec + i);
              }
            }
          }
        }
      }
    }
    cp_async_commit();
  };
  F2 s_post[NV][4], s_pre[NV][4];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int q = 0; q < 4; ++q) s_post[v][q] = s_pre[v][q] = 0;
  Slot s{-1, 0.f}, next{-1, 0.f}, next2{-1, 0.f};
  if (a.y != nullptr) {
    s = load_slot(a, t, lane);
    next = load_slot(a, t + step, lane);
  }
  fetch(t, s, ring);
  int cur = 0;
  for (; t < a.T; t += step, s = next, next = next2, cur = stages - 1 - cur) {
    const uint4* st = ring + cur * stage_vecs;
    float gate = 1.f;
    if (a.gate != nullptr) gate = a.gate[t];
    if (a.y != nullptr) next2 = load_slot(a, t + 2 * step, lane);
    if (stages == 2) {
      fetch(t + step, next, ring + (1 - cur) * stage_vecs);
      cp_async_wait<1>();
    } else {
      if (gt < 32 && t + step < a.T) {  // the next token's rows as far as L2
        if (next.row >= 0) prefetch_row(a.y, next.row, a.H);
        if (lane == 8 && g.out != nullptr) prefetch_row(g.out, t + step, a.H);
        if (lane == 9 && g.xn != nullptr) prefetch_row(g.xn, t + step, a.H);
        if (lane == 10 && g.xn != nullptr) prefetch_row(g.h, t + step, a.H);
      }
      cp_async_wait<0>();
    }
    // vector i of the token's row j of y
    auto y_vec = [&](int j, int row, int i) {
      return kStaged ? st[(3 + j) * nvec + i]
                     : __ldg(reinterpret_cast<const uint4*>(a.y) + static_cast<size_t>(row) * nvec + i);
    };
    // up to two rows stay in registers for the weights' gradient (362 -> 356 us)
    constexpr bool kKeep = kStaged && KMAX <= 2 && NV <= 2;
    uint4 kept[kKeep ? KMAX : 1][NV];
    F2 c[NV][4];
    float sums[3] = {0.f, 0.f, 0.f};  // h^2, pre g_xn h, c^2
    if (a.y != nullptr) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int q = 0; q < 4; ++q) c[v][q] = 0;
#pragma unroll
      for (int j = 0; j < KMAX; ++j) {
        const int row = __shfl_sync(0xffffffffu, s.row, j);
        const float w = __shfl_sync(0xffffffffu, s.w, j);
        if (row >= 0) {
          const F2 ww = f32x2(w, w);
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            const int i = gt + G * v;
            if (kFull || i < nvec) {
              F2 f[4];
              const uint4 yv = y_vec(j, row, i);
              if constexpr (kKeep) kept[j][v] = yv;
              unpack8(yv, f);
#pragma unroll
              for (int q = 0; q < 4; ++q) c[v][q] = f32x2_fma(ww, f[q], c[v][q]);
            }
          }
        }
      }
      sums[2] = square_sum<NV>(c);
    }
    if (g.xn != nullptr) {
      F2 hh = 0, vh = 0;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int i = gt + G * v;
        if (kFull || i < nvec) {
          F2 w[4], h[4], x[4];
          weights(true, i, w);
          unpack8(st[nvec + i], x);
          unpack8(st[2 * nvec + i], h);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            hh = f32x2_fma(h[q], h[q], hh);
            vh = f32x2_fma(f32x2_mul(w[q], x[q]), h[q], vh);
          }
        }
      }
      sums[0] = sum2(hh);
      sums[1] = sum2(vh);
    }
    group_sum<G, 3>(sums, red, turn);
    const float rh = rsqrtf(fmaf(sums[0], inv_h, a.eps));
    const float rc = a.post_norm ? rsqrtf(fmaf(sums[2], inv_h, a.eps)) : 1.f;
    const float along = -sums[1] * inv_h * rh * rh;  // -mean(v h) r_h^2
    const float gr = gate * rc;
    const F2 rh2 = f32x2(rh, rh), along2 = f32x2(along, along), gr2 = f32x2(gr, gr);
    const F2 scale = f32x2(a.scale, a.scale);
    F2 G8[NV][4];  // G, then G post, then g_c
    F2 uc2 = 0;    // sum of G post c
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = gt + G * v;
#pragma unroll
      for (int q = 0; q < 4; ++q) G8[v][q] = 0;
      if (kFull || i < nvec) {
        if (g.out != nullptr) unpack8(st[i], G8[v]);
        if (g.xn != nullptr) {
          F2 w[4], h[4], x[4];
          weights(true, i, w);
          unpack8(st[nvec + i], x);
          unpack8(st[2 * nvec + i], h);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const F2 d = f32x2_fma(h[q], along2, f32x2_mul(w[q], x[q]));
            G8[v][q] = f32x2_fma(rh2, d, G8[v][q]);
            s_pre[v][q] = f32x2_fma(f32x2_mul(x[q], rh2), h[q], s_pre[v][q]);
          }
        }
        if (g.residual != nullptr) {
          F2 f[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) f[q] = f32x2_mul(scale, G8[v][q]);
          st_global_cs_v4(reinterpret_cast<uint4*>(g.residual) + t * nvec + i, pack8(f));
        }
        if (a.y != nullptr) {
          F2 w[4];
          weights(false, i, w);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            s_post[v][q] = f32x2_fma(f32x2_mul(gr2, G8[v][q]), c[v][q], s_post[v][q]);
            G8[v][q] = f32x2_mul(G8[v][q], w[q]);
            uc2 = f32x2_fma(G8[v][q], c[v][q], uc2);
          }
        }
      }
    }
    if (a.y != nullptr) {
      float uc[1] = {sum2(uc2)};
      if (a.post_norm || g.gate != nullptr) group_sum<G, 1>(uc, red, turn);
      if (g.gate != nullptr && gt == 0) g.gate[t] = uc[0] * rc;
      const float back = a.post_norm ? -uc[0] * inv_h * rc * rc : 0.f;
      const F2 back2 = f32x2(back, back);
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          G8[v][q] = f32x2_mul(gr2, f32x2_fma(c[v][q], back2, G8[v][q]));
      float dots[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dots[j] = 0.f;
        if (j < KMAX) {
          const int row = __shfl_sync(0xffffffffu, s.row, j);
          const float w = __shfl_sync(0xffffffffu, s.w, j);
          if (row >= 0) {
            const F2 ww = f32x2(w, w);
            F2 d = 0;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              const int i = gt + G * v;
              if (kFull || i < nvec) {
                if (g.w != nullptr) {
                  F2 f[4];
                  if constexpr (kKeep) unpack8(kept[j & 1][v], f);
                  else unpack8(y_vec(j, row, i), f);
#pragma unroll
                  for (int q = 0; q < 4; ++q) d = f32x2_fma(G8[v][q], f[q], d);
                }
                if (g.y != nullptr) {
                  F2 f[4];
#pragma unroll
                  for (int q = 0; q < 4; ++q) f[q] = f32x2_mul(ww, G8[v][q]);
                  st_global_cs_v4(reinterpret_cast<uint4*>(g.y) + static_cast<size_t>(row) * nvec + i,
                                  pack8(f));
                }
              }
            }
            dots[j] = sum2(d);
          }
        }
      }
      if (g.w != nullptr) {
        float d;
        if constexpr (KMAX <= 2) {
          float two[2] = {dots[0], dots[1]};
          group_sum<G, 2>(two, red, turn);
          d = gt == 0 ? two[0] : two[1];
        } else {
          d = group_sum8<G>(dots, red, turn);
        }
        if (gt < a.k) g.w[t * a.k + gt] = d;
      }
    }
    // one stage: this thread has read all its columns of it
    if (stages == 1) fetch(t + step, next, ring);
  }
  cp_async_wait<0>();
  if (g.partial == nullptr) return;
  float* mine = g.partial + (static_cast<size_t>(blockIdx.x) * kPer + threadIdx.x / G) * 2 * a.H;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = gt + G * v;
    if (kFull || i < nvec) {
      ulonglong2* d = reinterpret_cast<ulonglong2*>(mine) + 2 * i;
      d[0] = make_ulonglong2(s_post[v][0], s_post[v][1]);
      d[1] = make_ulonglong2(s_post[v][2], s_post[v][3]);
      d = reinterpret_cast<ulonglong2*>(mine + a.H) + 2 * i;
      d[0] = make_ulonglong2(s_pre[v][0], s_pre[v][1]);
      d[1] = make_ulonglong2(s_pre[v][2], s_pre[v][3]);
    }
  }
}

// Sum of the partial rows: 32 columns x 8 slices of rows per block, each slice
// added in row order and the slices in theirs.
__global__ void __launch_bounds__(256) column_sum_kernel(const float* partial, int n, int H,
                                                         float* post, float* pre) {
  __shared__ float part[8][33];
  grid_dependency_wait();
  grid_launch_dependents();
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
  float* out = col < H ? post : pre;
  float s = 0.f;
  if (out != nullptr) {
#pragma unroll 8
    for (int i = slice; i < n; i += 8) s += partial[static_cast<size_t>(i) * 2 * H + col];
  }
  part[slice][threadIdx.x & 31] = s;
  __syncthreads();
  if (slice == 0 && out != nullptr) {
    for (int k = 1; k < 8; ++k) s += part[k][threadIdx.x & 31];
    out[col < H ? col : col - H] = s;
  }
}

// Blocks: no more than stay resident (MB to an SM), so that every SM has its share
// of the tokens in one round.
template <int G, int NV, int KU, int MB>
cudaError_t launch_fwd(const BlockArgs& a, int num_sms, cudaStream_t st) {
  constexpr int kPer = G == 32 ? 4 : 1;
  const int64_t need = (a.T + kPer - 1) / kPer;
  const int64_t cap = static_cast<int64_t>(num_sms) * MB;
  return launch_pdl(block_kernel<G, NV, KU, MB>, dim3(static_cast<unsigned>(need < cap ? need : cap)),
                    dim3(G == 32 ? 128 : G), 0, st, a);
}

constexpr int kSmSharedBytes = 228 * 1024;  // of an SM; 1 KB less for a block

template <int G, int NV, int KMAX, bool kStaged, bool kFull, int MB>
cudaError_t launch_bwd(const BlockArgs& a, const BlockGrads& g, int num_sms, cudaStream_t st,
                       int* groups) {
  constexpr int kPer = G == 32 ? 4 : 1;
  constexpr int kFixed = sizeof(Scratch<G>) + 1024;  // and what the system keeps of a block
  const int stage = (3 + (kStaged ? a.k : 0)) * a.H * 2 * kPer;
  const int weights = kStaged ? 8 * a.H : 0;
  const auto resident = [&](int stages) {
    const int n = kSmSharedBytes / (stages * stage + weights + kFixed);
    return n < MB ? n : MB;
  };
  // two stages, unless one lets twice as many blocks share an SM (5957 tokens of 2816
  // with eight rows: 206 us with two stages, 143 with one and two blocks)
  const int stages = resident(2) == 0 || 2 * resident(2) <= resident(1) ? 1 : 2;
  const int dyn = stages * stage + weights;
  const int per_sm = resident(stages);
  const auto kernel = block_bwd_kernel<G, NV, KMAX, kStaged, kFull, MB>;
  // the most a block may have, the same for every call: calls of other sizes on other
  // threads do not lower it before the launch
  const cudaError_t err =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kSmSharedBytes - 1024 - static_cast<int>(sizeof(Scratch<G>)));
  if (err != cudaSuccess) return err;
  const int64_t need = (a.T + kPer - 1) / kPer, cap = static_cast<int64_t>(num_sms) * per_sm;
  int blocks = static_cast<int>(need < cap ? need : cap);
  if (blocks * kPer > kBlockMaxGroups) blocks = kBlockMaxGroups / kPer;
  *groups = blocks * kPer;
  return launch_pdl(kernel, dim3(blocks), dim3(G == 32 ? 128 : G), dyn, st, a, g, stages);
}

// Whether a token's rows and the weights fit beside the block's other memory.
bool bwd_fits(int H, int k) {
  return (3 + k) * H * 2 + 8 * H + static_cast<int>(sizeof(Scratch<512>)) + 1024 <= kSmSharedBytes;
}

template <int G, int NV, int KMAX, int MB>
cudaError_t launch_bwd_k(const BlockArgs& a, const BlockGrads& g, int num_sms, cudaStream_t st,
                         int* groups) {
  if constexpr (G == 32) {
    return launch_bwd<G, NV, KMAX, true, false, MB>(a, g, num_sms, st, groups);
  } else {
    if constexpr (G == 512) {  // narrower rows fit with eight slots too
      if (!bwd_fits(a.H, a.k)) return launch_bwd<G, NV, 8, false, false, MB>(a, g, num_sms, st, groups);
    }
    if (a.H == 8 * G * NV) return launch_bwd<G, NV, KMAX, true, true, MB>(a, g, num_sms, st, groups);
    return launch_bwd<G, NV, KMAX, true, false, MB>(a, g, num_sms, st, groups);
  }
}

template <int G, int NV, int MB>
cudaError_t launch_bwd_any(const BlockArgs& a, const BlockGrads& g, int num_sms, cudaStream_t st,
                           int* groups) {
  if (a.k <= 2) return launch_bwd_k<G, NV, 2, MB>(a, g, num_sms, st, groups);
  if (a.k <= 4) return launch_bwd_k<G, NV, 4, MB>(a, g, num_sms, st, groups);
  return launch_bwd_k<G, NV, 8, MB>(a, g, num_sms, st, groups);
}

}  // namespace

// Partial rows of the gradient at most: one per token (or per four, rounded up
// to four), and kBlockMaxGroups.
int block_bwd_groups(int64_t T, int H) {
  const int64_t groups = H <= 512 ? (T + 3) / 4 * 4 : T;
  return static_cast<int>(groups < kBlockMaxGroups ? groups : kBlockMaxGroups);
}

// Threads, vectors to a thread, rows in flight and blocks to an SM by width. Few
// tokens at work at a time keep HBM's pages open: 4096 wide with 256 x 2, three blocks
// 197 us, four 224, five 364; 512 x 1, two blocks 271; 128 x 4, four blocks 229. 2048
// wide, six rows: 256 x 1, four blocks 98, six with two rows in flight 114; 128 x 2,
// five blocks 108.
cudaError_t launch_block(const BlockArgs& a, int num_sms, cudaStream_t st) {
  const bool few = a.k <= 2;
  if (a.H <= 256) return launch_fwd<32, 1, 4, 8>(a, num_sms, st);
  if (a.H <= 512) return launch_fwd<32, 2, 4, 4>(a, num_sms, st);
  if (a.H <= 1024)
    return few ? launch_fwd<128, 1, 2, 8>(a, num_sms, st) : launch_fwd<128, 1, 4, 8>(a, num_sms, st);
  if (a.H <= 2048)
    return few ? launch_fwd<256, 1, 2, 4>(a, num_sms, st) : launch_fwd<256, 1, 4, 4>(a, num_sms, st);
  if (a.H <= 4096)
    return few ? launch_fwd<256, 2, 2, 3>(a, num_sms, st) : launch_fwd<256, 2, 4, 2>(a, num_sms, st);
  if (a.H <= 8192)
    return few ? launch_fwd<256, 4, 2, 2>(a, num_sms, st) : launch_fwd<512, 2, 4, 1>(a, num_sms, st);
  return launch_fwd<512, 4, 2, 1>(a, num_sms, st);
}

// As above, for the gradient. 4096 wide, two rows: 256 x 2, two blocks 356 us (rows
// read again from shared memory 362; a loop over k that is not unrolled 391, three
// blocks' registers 483); 512 x 1, one block 643; 128 x 2 with rows in registers instead of shared memory 480. 2048 wide, six
// rows: 256 x 1, up to three blocks' registers 200, four 215; 128 x 2 218. 1024 wide,
// eight rows: 128 x 1 118, a warp with four vectors to a thread 204. Rows beyond 8192
// are left in L2 (29 to 45 % of the copy's rate; a block holds 1024 threads' sums).
cudaError_t launch_block_bwd(const BlockArgs& a, const BlockGrads& g, int num_sms, cudaStream_t st) {
  int groups = 0;
  cudaError_t err;
  if (a.H <= 256) err = launch_bwd_any<32, 1, 4>(a, g, num_sms, st, &groups);
  else if (a.H <= 512) err = launch_bwd_any<32, 2, 3>(a, g, num_sms, st, &groups);
  else if (a.H <= 1024) err = launch_bwd_any<128, 1, 6>(a, g, num_sms, st, &groups);
  else if (a.H <= 2048) err = launch_bwd_any<256, 1, 3>(a, g, num_sms, st, &groups);
  else if (a.H <= 4096) err = launch_bwd_any<256, 2, 2>(a, g, num_sms, st, &groups);
  else if (a.H <= 6144) err = launch_bwd_any<384, 2, 1>(a, g, num_sms, st, &groups);
  else if (a.H <= 8192) err = launch_bwd_any<512, 2, 1>(a, g, num_sms, st, &groups);
  else err = launch_bwd<1024, 2, 8, false, false, 1>(a, g, num_sms, st, &groups);
  if (err != cudaSuccess || g.partial == nullptr) return err;
  return launch_pdl(column_sum_kernel, dim3(a.H / 16), dim3(256), 0, st,
                    static_cast<const float*>(g.partial), groups, a.H, g.post, g.pre);
}

}  // namespace moe
