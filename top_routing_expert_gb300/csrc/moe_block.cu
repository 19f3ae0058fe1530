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
// stored. Both kernels are bound by their bytes: a token's rows are read once
// from HBM, the statistics come from registers, and the gradient's second look
// at y_j (for g_w) finds it in L1 or L2.
#include "moe_internal.h"
#include "moe_ptx.cuh"

namespace moe {

namespace {

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint4 v;
  v.x = pack_bf16x2(f[0], f[1]);
  v.y = pack_bf16x2(f[2], f[3]);
  v.z = pack_bf16x2(f[4], f[5]);
  v.w = pack_bf16x2(f[6], f[7]);
  return v;
}

// 8 fp32 weights from column 8 * i, or ones.
__device__ __forceinline__ void weight8(const float* w, int i, float (&f)[8]) {
  if (w == nullptr) {
#pragma unroll
    for (int q = 0; q < 8; ++q) f[q] = 1.f;
    return;
  }
  const float4 a = __ldg(reinterpret_cast<const float4*>(w) + 2 * i);
  const float4 b = __ldg(reinterpret_cast<const float4*>(w) + 2 * i + 1);
  f[0] = a.x;
  f[1] = a.y;
  f[2] = a.z;
  f[3] = a.w;
  f[4] = b.x;
  f[5] = b.y;
  f[6] = b.z;
  f[7] = b.w;
}

// Sums of M values over the G threads of a token's group, in every thread.
// G > 32: the group is the block; `red` holds M * G/32 values for each of two
// alternating calls, so one barrier a call is enough.
template <int G, int M>
__device__ __forceinline__ void group_sum(float (&v)[M], float* red, int& turn) {
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[m] += __shfl_xor_sync(0xffffffffu, v[m], o);
  if constexpr (G > 32) {
    constexpr int W = G / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* r = red + turn * (8 * W);
    turn ^= 1;
    if (lane == 0) {
#pragma unroll
      for (int m = 0; m < M; ++m) r[m * W + warp] = v[m];
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < M; ++m) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += r[m * W + w];
      v[m] = s;
    }
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

// c[v][8] = sum over the slots, ascending, of w_j y_j.
template <int G, int NV>
__device__ __forceinline__ void combine_rows(const BlockArgs& a, const Slot& s, int gt, int nvec,
                                             float (&c)[NV][8]) {
  constexpr int KU = NV <= 2 ? 4 : 2;  // rows in flight together
  const uint4* yv = reinterpret_cast<const uint4*>(a.y);
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int q = 0; q < 8; ++q) c[v][q] = 0.f;
  for (int j0 = 0; j0 < a.k; j0 += KU) {
    uint4 b[KU][NV];
    float w[KU];
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      const int j = j0 + u;
      const int row = __shfl_sync(0xffffffffu, s.row, j & 31);
      w[u] = __shfl_sync(0xffffffffu, s.w, j & 31);
      if (row < 0) w[u] = 0.f;  // lanes from k up hold no row
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int i = gt + G * v;
        b[u][v] = row >= 0 && i < nvec ? __ldg(yv + static_cast<size_t>(row) * nvec + i)
                                       : make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int u = 0; u < KU; ++u)
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float f[8];
        unpack8(b[u][v], f);
#pragma unroll
        for (int q = 0; q < 8; ++q) c[v][q] = fmaf(w[u], f[q], c[v][q]);
      }
  }
}

// G threads to a token, NV vectors of 8 columns to a thread (vector gt + G v):
// G * 8 * NV >= H. Blocks hold max(1, 128 / G) tokens.
template <int G, int NV>
__global__ void __launch_bounds__(G > 128 ? G : 128) block_kernel(BlockArgs a) {
  constexpr int kPer = G >= 128 ? 1 : 128 / G;
  __shared__ float red[2 * 8 * (G / 32)];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, gt = threadIdx.x % G;
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
      res[v] = i < nvec ? __ldg(reinterpret_cast<const uint4*>(a.residual) + t * nvec + i)
                        : make_uint4(0, 0, 0, 0);
    }
    float gate = 1.f;
    if (a.gate != nullptr) gate = a.gate[t];
    float h[NV][8];
    if (gt < 32 && t + step < a.T) {
      if (next.row >= 0) prefetch_row(a.y, next.row, a.H);
      if (lane == 8) prefetch_row(a.residual, t + step, a.H);
    }
    if (a.y != nullptr) {
      next2 = load_slot(a, t + 2 * step, lane);
      combine_rows<G, NV>(a, s, gt, nvec, h);
      float r = gate;
      if (a.post_norm) {
        float ss[1] = {0.f};
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int q = 0; q < 8; ++q) ss[0] = fmaf(h[v][q], h[v][q], ss[0]);
        group_sum<G, 1>(ss, red, turn);
        r *= rsqrtf(fmaf(ss[0], inv_h, a.eps));
      }
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int i = gt + G * v;
        if (i < nvec) {
          float w[8], f[8];
          weight8(a.post_weight, i, w);
          unpack8(res[v], f);
#pragma unroll
          for (int q = 0; q < 8; ++q) h[v][q] = fmaf(a.scale, f[q], h[v][q] * r * w[q]);
        }
      }
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float f[8];
        unpack8(res[v], f);
#pragma unroll
        for (int q = 0; q < 8; ++q) h[v][q] = a.scale * f[q];
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
      float ss[1] = {0.f};
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int q = 0; q < 8; ++q) ss[0] = fmaf(h[v][q], h[v][q], ss[0]);
      group_sum<G, 1>(ss, red, turn);
      const float r = rsqrtf(fmaf(ss[0], inv_h, a.eps));
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int i = gt + G * v;
        if (i < nvec) {
          float w[8], f[8];
          weight8(a.pre_weight, i, w);
#pragma unroll
          for (int q = 0; q < 8; ++q) f[q] = h[v][q] * r * w[q];
          reinterpret_cast<uint4*>(a.xn)[t * nvec + i] = pack8(f);
        }
      }
    }
  }
}

// As block_kernel's layout. Sums over tokens (g_post, g_pre) stay in registers,
// one column of a thread's each, until the block's last token; the blocks'
// partial sums [blocks][2][H] are added by column_sum_kernel.
template <int G, int NV>
__global__ void __launch_bounds__(G > 128 ? G : 128) block_bwd_kernel(BlockArgs a, BlockGrads g) {
  constexpr int kPer = G >= 128 ? 1 : 128 / G;
  __shared__ float red[2 * 8 * (G / 32)];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, gt = threadIdx.x % G;
  const int nvec = a.H >> 3;
  const float inv_h = 1.f / static_cast<float>(a.H);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kPer;
  int turn = 0;
  int64_t t = static_cast<int64_t>(blockIdx.x) * kPer + threadIdx.x / G;
  float s_post[NV][8], s_pre[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int q = 0; q < 8; ++q) s_post[v][q] = s_pre[v][q] = 0.f;
  Slot s{-1, 0.f}, next{-1, 0.f}, next2{-1, 0.f};
  if (a.y != nullptr) {
    s = load_slot(a, t, lane);
    next = load_slot(a, t + step, lane);
  }
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (; t < a.T; t += step, s = next, next = next2) {
    uint4 hv[NV], xv[NV], ov[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = gt + G * v;
      const bool in = i < nvec;
      ov[v] = in && g.out != nullptr ? ld_global_cs_v4(reinterpret_cast<const uint4*>(g.out) + t * nvec + i) : zero;
      xv[v] = in && g.xn != nullptr ? ld_global_cs_v4(reinterpret_cast<const uint4*>(g.xn) + t * nvec + i) : zero;
      hv[v] = in && g.xn != nullptr ? ld_global_cs_v4(reinterpret_cast<const uint4*>(g.h) + t * nvec + i) : zero;
    }
    float gate = 1.f;
    if (a.gate != nullptr) gate = a.gate[t];
    float c[NV][8];
    float sums[3] = {0.f, 0.f, 0.f};  // h^2, pre g_xn h, c^2
    if (gt < 32 && t + step < a.T) {
      if (next.row >= 0) prefetch_row(a.y, next.row, a.H);
      if (lane == 8 && g.out != nullptr) prefetch_row(g.out, t + step, a.H);
      if (lane == 9 && g.xn != nullptr) prefetch_row(g.xn, t + step, a.H);
      if (lane == 10 && g.xn != nullptr) prefetch_row(g.h, t + step, a.H);
    }
    if (a.y != nullptr) {
      next2 = load_slot(a, t + 2 * step, lane);
      combine_rows<G, NV>(a, s, gt, nvec, c);
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int q = 0; q < 8; ++q) sums[2] = fmaf(c[v][q], c[v][q], sums[2]);
    }
    if (g.xn != nullptr) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int i = gt + G * v;
        if (i < nvec) {
          float w[8], h[8], x[8];
          weight8(a.pre_weight, i, w);
          unpack8(hv[v], h);
          unpack8(xv[v], x);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            sums[0] = fmaf(h[q], h[q], sums[0]);
            sums[1] = fmaf(w[q] * x[q], h[q], sums[1]);
          }
        }
      }
    }
    group_sum<G, 3>(sums, red, turn);
    const float rh = rsqrtf(fmaf(sums[0], inv_h, a.eps));
    const float rc = a.post_norm ? rsqrtf(fmaf(sums[2], inv_h, a.eps)) : 1.f;
    const float along = sums[1] * inv_h * rh * rh;  // mean(v h) r_h^2
    float G8[NV][8];  // G, then g_c
    float uc[1] = {0.f};  // sum of G post c
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = gt + G * v;
      unpack8(ov[v], G8[v]);
      if (i < nvec) {
        if (g.xn != nullptr) {
          float w[8], h[8], x[8];
          weight8(a.pre_weight, i, w);
          unpack8(hv[v], h);
          unpack8(xv[v], x);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            G8[v][q] = fmaf(rh, fmaf(-h[q], along, w[q] * x[q]), G8[v][q]);
            s_pre[v][q] = fmaf(x[q] * rh, h[q], s_pre[v][q]);
          }
        }
        if (g.residual != nullptr) {
          float f[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) f[q] = a.scale * G8[v][q];
          st_global_cs_v4(reinterpret_cast<uint4*>(g.residual) + t * nvec + i, pack8(f));
        }
        if (a.y != nullptr) {
          float w[8];
          weight8(a.post_weight, i, w);
          const float gr = gate * rc;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            s_post[v][q] = fmaf(gr * G8[v][q], c[v][q], s_post[v][q]);
            G8[v][q] *= w[q];
            uc[0] = fmaf(G8[v][q], c[v][q], uc[0]);
          }
        }
      }
    }
    if (a.y == nullptr) continue;
    const bool need_uc = a.post_norm || g.gate != nullptr;
    if (need_uc) group_sum<G, 1>(uc, red, turn);
    if (g.gate != nullptr && gt == 0) g.gate[t] = uc[0] * rc;
    const float back = a.post_norm ? uc[0] * inv_h * rc * rc : 0.f;
    const float gr = gate * rc;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int q = 0; q < 8; ++q) G8[v][q] = gr * fmaf(-c[v][q], back, G8[v][q]);
    float dots[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dots[j] = 0.f;
      if (j < a.k) {
        const int row = __shfl_sync(0xffffffffu, s.row, j);
        const float w = __shfl_sync(0xffffffffu, s.w, j);
        if (row >= 0) {
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            const int i = gt + G * v;
            if (i < nvec) {
              const size_t at = static_cast<size_t>(row) * nvec + i;
              if (g.w != nullptr) {
                float f[8];
                unpack8(__ldg(reinterpret_cast<const uint4*>(a.y) + at), f);
#pragma unroll
                for (int q = 0; q < 8; ++q) dots[j] = fmaf(G8[v][q], f[q], dots[j]);
              }
              if (g.y != nullptr) {
                float f[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) f[q] = w * G8[v][q];
                st_global_cs_v4(reinterpret_cast<uint4*>(g.y) + at, pack8(f));
              }
            }
          }
        }
      }
    }
    if (g.w != nullptr) {
      if (a.k <= 2) {
        float d[2] = {dots[0], dots[1]};
        group_sum<G, 2>(d, red, turn);
        if (gt < a.k) g.w[t * a.k + gt] = gt == 0 ? d[0] : d[1];
      } else {
        group_sum<G, 8>(dots, red, turn);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < a.k && gt == j) g.w[t * a.k + j] = dots[j];
      }
    }
  }
  if (g.partial == nullptr) return;
  float* mine = g.partial + (static_cast<size_t>(blockIdx.x) * kPer + threadIdx.x / G) * 2 * a.H;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = gt + G * v;
    if (i < nvec) {
      float4* d = reinterpret_cast<float4*>(mine) + 2 * i;
      d[0] = make_float4(s_post[v][0], s_post[v][1], s_post[v][2], s_post[v][3]);
      d[1] = make_float4(s_post[v][4], s_post[v][5], s_post[v][6], s_post[v][7]);
      d = reinterpret_cast<float4*>(mine + a.H) + 2 * i;
      d[0] = make_float4(s_pre[v][0], s_pre[v][1], s_pre[v][2], s_pre[v][3]);
      d[1] = make_float4(s_pre[v][4], s_pre[v][5], s_pre[v][6], s_pre[v][7]);
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

template <int G, int NV>
cudaError_t launch_fwd(const BlockArgs& a, int num_sms, cudaStream_t st) {
  constexpr int kPer = G >= 128 ? 1 : 128 / G;
  const int64_t need = (a.T + kPer - 1) / kPer;
  const int cap = num_sms * (G > 128 ? 2048 / G : 16);
  return launch_pdl(block_kernel<G, NV>, dim3(static_cast<unsigned>(need < cap ? need : cap)),
                    dim3(G > 128 ? G : 128), 0, st, a);
}

template <int G, int NV>
cudaError_t launch_bwd(const BlockArgs& a, const BlockGrads& g, int blocks, cudaStream_t st) {
  return launch_pdl(block_bwd_kernel<G, NV>, dim3(blocks), dim3(G > 128 ? G : 128), 0, st, a, g);
}

// Threads of a token's group by width.
int group_threads(int H) { return H <= 1024 ? 32 : H <= 2048 ? 128 : H <= 8192 ? 256 : 512; }

}  // namespace

// Partial rows of the gradient: up to kBlockMaxGroups, a multiple of a block's
// groups.
int block_bwd_groups(int64_t T, int H) {
  const int per = group_threads(H) == 32 ? 4 : 1;
  const int64_t groups = (T + per - 1) / per * per;
  return static_cast<int>(groups < kBlockMaxGroups ? groups : kBlockMaxGroups);
}

cudaError_t launch_block(const BlockArgs& a, int num_sms, cudaStream_t st) {
  if (a.H <= 256) return launch_fwd<32, 1>(a, num_sms, st);
  if (a.H <= 512) return launch_fwd<32, 2>(a, num_sms, st);
  if (a.H <= 1024) return launch_fwd<32, 4>(a, num_sms, st);
  if (a.H <= 2048) return launch_fwd<128, 2>(a, num_sms, st);
  if (a.H <= 4096) return launch_fwd<256, 2>(a, num_sms, st);
  if (a.H <= 8192) return launch_fwd<256, 4>(a, num_sms, st);
  return launch_fwd<512, 4>(a, num_sms, st);
}

cudaError_t launch_block_bwd(const BlockArgs& a, const BlockGrads& g, cudaStream_t st) {
  const int groups = block_bwd_groups(a.T, a.H);
  const int blocks = group_threads(a.H) == 32 ? groups / 4 : groups;
  cudaError_t err;
  if (a.H <= 256) err = launch_bwd<32, 1>(a, g, blocks, st);
  else if (a.H <= 512) err = launch_bwd<32, 2>(a, g, blocks, st);
  else if (a.H <= 1024) err = launch_bwd<32, 4>(a, g, blocks, st);
  else if (a.H <= 2048) err = launch_bwd<128, 2>(a, g, blocks, st);
  else if (a.H <= 4096) err = launch_bwd<256, 2>(a, g, blocks, st);
  else if (a.H <= 8192) err = launch_bwd<256, 4>(a, g, blocks, st);
  else err = launch_bwd<512, 4>(a, g, blocks, st);
  if (err != cudaSuccess || g.partial == nullptr) return err;
  return launch_pdl(column_sum_kernel, dim3(a.H / 16), dim3(256), 0, st,
                    static_cast<const float*>(g.partial), groups, a.H, g.post, g.pre);
}

}  // namespace moe
