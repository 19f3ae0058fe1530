// The experts' grouped product on microscaled 4-bit operands:
//   D[r, n] = bf16(f(sum_k x[r, k] w[e(r)][n, k])),  f = identity or tanh GELU,
// over ragged expert segments of rows, by block-scaled UMMA (kind::mxf4: e2m1
// operands, one e8m0 scale per 32 along K applied by the tensor core, fp32
// accumulation in TMEM).
//
// The weights are the UMMA's A operand (M = 128 output columns) and the tokens
// its B operand (N = up to `tile_tokens` rows of one expert), so a tile's N
// follows the number of tokens it has, from 16 up: a decoding batch with a few
// rows per expert spends neither shared memory nor tensor time on rows that
// are not there, and its epilogue writes rows of D in 64-byte pieces.
//
// Scales reach TMEM by tcgen05.cp from shared memory, 128 rows x 4 scales (512
// bytes) at a time. Those of the weights lie in that order in memory and come
// by bulk copies; those of the tokens start at any row (a segment need not
// begin at a multiple of anything), so one warp copies them word by word
// (cp.async, 4 bytes, coalesced in memory) to their places.
//
// Roles (256 threads): warp 0 = TMA producer, warp 1 = UMMA issuer, warp 2 =
// token scales, warp 3 = TMEM allocation, warps 4-7 = epilogue.
#include "moe_internal.h"
#include "moe_ptx.cuh"

namespace moe {

namespace {

constexpr int kBM = 128;                 // output columns per tile
constexpr int kStageK = 256;             // K per stage: one 128-byte row of codes
constexpr int kMaxTokens = 240;          // two accumulators of 240 columns + scales in TMEM
constexpr uint32_t kWBytes = kBM * 128;  // 16 KB
constexpr uint32_t kWScaleBytes = 1024;  // 2 x 512
constexpr int kMaxStages = 10;
constexpr int kThreads = 256;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemSfW = 480;  // 2 x 4 columns
constexpr uint32_t kTmemSfX = 488;  // 2 x 8 columns

__host__ __device__ constexpr uint32_t x_scale_blocks(int nt) { return static_cast<uint32_t>(nt + 127) / 128; }
__host__ __device__ constexpr uint32_t stage_bytes(int nt) {
  return kWBytes + static_cast<uint32_t>(nt) * 128 + kWScaleBytes + 2 * 512 * x_scale_blocks(nt);
}

__device__ __forceinline__ float gelu_tanh_f(float u) {
  // 0.5 u (1 + tanh(z)) = u / (1 + exp(-2 z)),  z = sqrt(2/pi) (u + 0.044715 u^3)
  const float z2 = 1.5957691216057308f * fmaf(0.044715f * u, u * u, u);
  return __fdividef(u, 1.0f + __expf(-z2));
}

struct Tile {
  int e, row0, row_end, n0;
};

// Tile order: groups of 8 token tiles, all column tiles of a group before the
// next group, token tiles innermost (they share the weights in L2).
__device__ __forceinline__ Tile decode(int L, const int* prefix, const int* offs, int E, int total_t,
                                       int n_tiles_n, int nt) {
  constexpr int group = 8;
  const int per_group = group * n_tiles_n;
  const int g = L / per_group;
  const int first = g * group;
  const int gsz = min(group, total_t - first);
  const int r = L - g * per_group;
  const int tt = first + r % gsz;
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= tt) lo = mid; else hi = mid - 1;
  }
  Tile t;
  t.e = lo;
  t.row0 = offs[lo] + (tt - prefix[lo]) * nt;
  t.row_end = offs[lo + 1];
  t.n0 = (r / gsz) * kBM;
  return t;
}

__global__ void __launch_bounds__(kThreads, 1)
    expert_gemm_mx4_kernel(const __grid_constant__ CUtensorMap tm_w,
                           const __grid_constant__ CUtensorMap tm_x, Mx4GemmArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_up_1024(smem_raw);
  const int nst = p.stages, NT = p.tile_tokens;
  const uint32_t sb = stage_bytes(NT);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + static_cast<size_t>(nst) * sb);
  uint64_t* empty = full + nst;
  uint64_t* tfull = empty + nst;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  uint32_t* abort_flag = tmem_slot + 1;
  int* offs = reinterpret_cast<int*>(abort_flag + 1);  // [E+1]
  int* prefix = offs + (p.E + 1);                      // [E+1]

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int E = p.E;
  if (warp == 3) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  if (warp == 2 && lane == 0) {
    for (int s = 0; s < nst; ++s) {
      mbar_init(&full[s], 1 + 32);  // the producer's bytes and the scale warp's lanes
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 128);
    }
    mbar_init(drain, 1);
    *abort_flag = 0u;
    fence_barrier_init();
  }
  if (warp == 1 && lane == 0) {
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
  }
  grid_dependency_wait();
  grid_launch_dependents();
  for (int i = tid; i <= E; i += kThreads) {
    const int v = p.offsets[i];
    offs[i] = v < 0 ? 0 : (v > p.rows ? p.rows : v);  // rows outside the buffer are never touched
  }
  __syncthreads();
  if (tid == 0)
    for (int i = 1; i <= E; ++i) offs[i] = offs[i] < offs[i - 1] ? offs[i - 1] : offs[i];
  __syncthreads();
  if (warp == 0) {
    int carry = 0;
    for (int b = 0; b < E; b += 32) {
      const int e = b + lane;
      const int n = e < E ? (offs[e + 1] - offs[e] + NT - 1) / NT : 0;
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (e < E) prefix[e] = carry + incl - n;
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) prefix[E] = carry;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const uint32_t tmem_base = *tmem_slot;
  const int total_t = prefix[E];
  const int n_tiles_n = (p.N + kBM - 1) / kBM;
  const int total = total_t * n_tiles_n;
  const int nk = (p.K + kStageK - 1) / kStageK;   // stages per tile
  const int nkb = (p.K + 127) / 128;              // 128-deep scale blocks
  const WaitCtl wc{abort_flag, p.dev_status, p.timeout_ns};

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------ TMA producer ----
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0;
      bool aborted = false;
      for (int L = blockIdx.x; L < total && !aborted; L += gridDim.x) {
        const Tile c = decode(L, prefix, offs, E, total_t, n_tiles_n, NT);
        const uint8_t* ws = p.w_scale +
            (static_cast<size_t>(c.e) * n_tiles_n + c.n0 / kBM) * nkb * 512;
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, wc)) {
            aborted = true;
            break;
          }
          uint8_t* sw = smem + static_cast<size_t>(stage) * sb;
          uint8_t* sx = sw + kWBytes;
          uint8_t* ssw = sx + NT * 128;
          const uint32_t sc = 512u * static_cast<uint32_t>(min(2, nkb - 2 * kb));
          mbar_arrive_expect_tx(&full[stage], kWBytes + static_cast<uint32_t>(NT) * 128 + sc);
          tma_load_2d(sw, &tm_w, &full[stage], kb * 128, c.e * p.N + c.n0);
          tma_load_2d(sx, &tm_x, &full[stage], kb * 128, c.row0);
          bulk_load(ssw, ws + static_cast<size_t>(kb) * 1024, sc, &full[stage]);
          ++issued;
          if (++stage == nst) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (aborted) {
        // copies in flight land before the CTA exits
        int s = stage;
        uint32_t ph = phase;
        for (int d = 0; d < nst && d < issued; ++d) {
          if (--s < 0) {
            s = nst - 1;
            ph ^= 1u;
          }
          mbar_wait_drain(&full[s], ph, kDrainLimitNs);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ------------------------------------------------- UMMA issuer ----
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool aborted = false;
      for (int L = blockIdx.x; L < total && !aborted; L += gridDim.x) {
        const Tile c = decode(L, prefix, offs, E, total_t, n_tiles_n, NT);
        const int n_tok = min(NT, c.row_end - c.row0);
        const uint32_t idesc = idesc_mxf4_e8m0(kBM, static_cast<uint32_t>((n_tok + 15) & ~15));
        if (!mbar_wait(&tempty[acc], acc_phase ^ 1u, wc)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kMaxTokens);
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait(&full[stage], phase, wc)) {
            aborted = true;
            break;
          }
          fence_proxy_async();  // the scale warp's copies, before tcgen05.cp reads them
          tc_fence_after();
          const uint32_t aw = smem_u32(smem + static_cast<size_t>(stage) * sb);
          const uint32_t ax = aw + kWBytes;
          const uint32_t asw = ax + static_cast<uint32_t>(NT) * 128;
          const uint32_t asx = asw + kWScaleBytes;
          const uint32_t xb = x_scale_blocks(NT);
          const int steps = min(4, (p.K - kb * kStageK) / 64);
          for (int h = 0; 2 * h < steps; ++h) {
            tmem_cp_32x128b(tmem_base + kTmemSfW + 4u * h, smem_desc_plain(asw + 512u * h, 128u));
            for (uint32_t q = 0; q < xb; ++q)
              tmem_cp_32x128b(tmem_base + kTmemSfX + 8u * h + 4u * q,
                              smem_desc_plain(asx + 512u * (xb * h + q), 128u));
          }
          for (int s = 0; s < steps; ++s) {
            const uint32_t h = static_cast<uint32_t>(s >> 1);
            const uint32_t id = static_cast<uint32_t>(s & 1) * 2u;  // scale bytes 0-1 or 2-3
            umma_mxf4(d_tmem, smem_desc_sw128(aw + 32u * s, 16u, 1024u),
                      smem_desc_sw128(ax + 32u * s, 16u, 1024u), idesc | (id << 4) | (id << 29),
                      tmem_base + kTmemSfW + 4u * h, tmem_base + kTmemSfX + 8u * h,
                      (kb | s) != 0 ? 1u : 0u);
          }
          umma_commit(&empty[stage]);
          if (++stage == nst) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (aborted) break;
        umma_commit(&tfull[acc]);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      // every UMMA issued must finish before TMEM is released
      umma_commit(drain);
      mbar_wait_drain(drain, 0, kDrainLimitNs);
    }
  } else if (warp == 2) {
    // ---------------------------------------------------- token scales ----
    int stage = 0;
    uint32_t phase = 0;
    bool aborted = false;
    const uint32_t* xs = reinterpret_cast<const uint32_t*>(p.x_scale);
    const uint32_t xb = x_scale_blocks(NT);
    for (int L = blockIdx.x; L < total && !aborted; L += gridDim.x) {
      const Tile c = decode(L, prefix, offs, E, total_t, n_tiles_n, NT);
      const int n_tok = min(NT, c.row_end - c.row0);
      for (int kb = 0; kb < nk; ++kb) {
        if (!mbar_wait(&empty[stage], phase ^ 1u, wc)) {
          aborted = true;
          break;
        }
        const uint32_t dst = smem_u32(smem + static_cast<size_t>(stage) * sb) + kWBytes +
                             static_cast<uint32_t>(NT) * 128 + kWScaleBytes;
        for (int h = 0; h < 2 && 2 * kb + h < nkb; ++h) {
          const uint32_t* src = xs + static_cast<size_t>(2 * kb + h) * p.rows + c.row0;
          // token i of a block of 128: lane i % 32 of TMEM, word i / 32
          for (int i = lane; i < n_tok; i += 32)
            cp_async_4(dst + 512u * (xb * h + static_cast<uint32_t>(i >> 7)) + 16u * (i & 31) +
                           4u * ((i >> 5) & 3),
                       src + i);
        }
        cp_async_arrive(&full[stage]);
        if (++stage == nst) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    cp_async_wait_all();
  } else if (warp >= 4) {
    // ------------------------------------------------------ epilogue ----
    // warp w reads TMEM lanes 32 (w % 4) .. + 31: output columns
    const int q = warp & 3;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int L = blockIdx.x; L < total; L += gridDim.x) {
      const Tile c = decode(L, prefix, offs, E, total_t, n_tiles_n, NT);
      const int n_tok = min(NT, c.row_end - c.row0);
      if (!mbar_wait(&tfull[acc], acc_phase, wc)) break;
      tc_fence_after();
      const int n = c.n0 + 32 * q + lane;
      const uint32_t t_base = tmem_base + (static_cast<uint32_t>(32 * q) << 16) +
                              static_cast<uint32_t>(acc * kMaxTokens);
      if (c.n0 + 32 * q < p.N) {
        uint16_t* d = p.D + static_cast<size_t>(c.row0) * p.N + n;
        for (int j = 0; j < n_tok; j += 16) {
          uint32_t r[16];
          tmem_ld_32x32b_x16(t_base + static_cast<uint32_t>(j), r);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (j + i < n_tok) {
              float v = __uint_as_float(r[i]);
              if (p.gelu) v = gelu_tanh_f(v);
              d[static_cast<size_t>(j + i) * p.N] =
                  __bfloat16_as_ushort(__float2bfloat16_rn(v));
            }
        }
      }
      tc_fence_before();
      mbar_arrive(&tempty[acc]);
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 3) tmem_dealloc(tmem_base, kTmemCols);
}

size_t smem_bytes(int E, int stages, int nt) {
  return 1024 + static_cast<size_t>(stages) * stage_bytes(nt) + 8 * (2 * stages + 5) + 8 +
         8 * static_cast<size_t>(E + 1);
}

}  // namespace

// Twice the average rows of an expert plus 8 hold almost any decoding batch's
// segments in one tile; larger averages take the widest tile.
int mx4_tile_tokens(int64_t rows, int E) {
  const int64_t want = (2 * rows / E + 8 + 15) / 16 * 16;
  return want < kMaxTokens ? static_cast<int>(want) : kMaxTokens;
}

cudaError_t launch_expert_gemm_mx4(const CUtensorMap& tm_w, const CUtensorMap& tm_x,
                                   const Mx4GemmArgs& a, int num_sms, cudaStream_t st) {
  int dev = 0, optin = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  err = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  if (err != cudaSuccess) return err;
  Mx4GemmArgs args = a;
  args.stages = kMaxStages;
  while (args.stages > 2 && smem_bytes(a.E, args.stages, a.tile_tokens) > static_cast<size_t>(optin))
    --args.stages;
  const size_t smem = smem_bytes(a.E, args.stages, a.tile_tokens);
  err = cudaFuncSetAttribute(expert_gemm_mx4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem));
  if (err != cudaSuccess) return err;
  return launch_pdl(expert_gemm_mx4_kernel, dim3(num_sms), dim3(kThreads), smem, st, tm_w, tm_x, args);
}

}  // namespace moe
