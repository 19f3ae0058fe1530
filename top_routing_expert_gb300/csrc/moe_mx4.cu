// Microscaled 4-bit floating point: blocks of 32 consecutive values along K
// share one power-of-two scale (e8m0: 2^(byte - 127), byte 255 = NaN) and are
// held as e2m1 codes (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives).
//
// For a block with largest magnitude amax: scale exponent
// E = max(floor(log2(amax)) - 2, -127), q = e2m1(x * 2^-E), round to nearest
// even, magnitudes above 6 held at 6. Multiplying by a power of two is exact,
// so the one rounding is that to e2m1. A block of zeros has byte 0; a block
// with a NaN or an infinity has byte 255 and codes 0.
//
// Layouts: codes two to a byte, the even element in the low half; scales of
// rows as [ceil(K/128)][rows][4] (the four scales of 128 consecutive k form a
// word, and the words of consecutive rows are consecutive, so a tile of rows
// reads and writes whole cache lines of them); scales of weights as 512-byte
// blocks of 128 output columns x 4 scales in the order the tensor core's scale
// copy reads: column n at (n % 32) * 16 + (n / 32) * 4.
#include <cuda_fp4.h>

#include "moe_internal.h"
#include "moe_ptx.cuh"

namespace moe {

namespace {

constexpr unsigned kFull = 0xffffffffu;

// Scale byte of a block from the bits of its largest magnitude (a bf16 value
// as fp32 bits). The biased exponent of amax is floor(log2) + 127; subnormal
// amax gives at most byte 0 either way.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  if (e == 255u) return 255u;
  return e > 2u ? e - 2u : 0u;
}
// 2^-(byte - 127), exact: byte <= 252 for finite blocks, so the biased
// exponent 254 - byte is at least 2.
__device__ __forceinline__ float scale_inverse(uint32_t byte) {
  return byte == 255u ? 0.f : __uint_as_float((254u - byte) << 23);
}
// Two values to e2m1 codes, `lo` in the low half of the byte.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp4x2(make_float2(lo, hi), __NV_E2M1, cudaRoundNearest);
}

__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t w) {
  const uint32_t lo = (w << 16) & 0x7fff0000u, hi = w & 0x7fff0000u;
  return max(m, max(lo, hi));
}

// 8 bf16 (one 16-byte vector) times a power of two to 8 codes.
__device__ __forceinline__ uint32_t codes8(const uint4& v, float inv, bool bad) {
  if (bad) return 0u;
  uint32_t r = e2m1x2(bf16_lo(v.x) * inv, bf16_hi(v.x) * inv);
  r |= e2m1x2(bf16_lo(v.y) * inv, bf16_hi(v.y) * inv) << 8;
  r |= e2m1x2(bf16_lo(v.z) * inv, bf16_hi(v.z) * inv) << 16;
  r |= e2m1x2(bf16_lo(v.w) * inv, bf16_hi(v.w) * inv) << 24;
  return r;
}

// A warp takes 4 rows x 256 values: all its loads go out before the first is
// used, and the scale words of the four rows, which are neighbours in memory,
// leave together. A lane holds 8 consecutive values of each row, four lanes a
// block of 32. HBM bounds both directions: 65536 x 4096 there and back, 1.36 GB,
// take 238 us, 5.7 TB/s.
constexpr int kRows = 4;

__device__ __forceinline__ uint4 ld_stream(const uint4* p) {  // read once
  uint4 v;
  asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__global__ void __launch_bounds__(256) quantize_rows_kernel(const uint16_t* __restrict__ x,
                                                            uint8_t* __restrict__ q,
                                                            uint8_t* __restrict__ scale,
                                                            const int32_t* __restrict__ n_rows,
                                                            int64_t rows, int K) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  int64_t n = rows;
  if (n_rows != nullptr) {
    const int64_t v = *n_rows;
    n = v < 0 ? 0 : (v < rows ? v : rows);
  }
  const int chunks = (K + 255) >> 8;
  const int64_t tasks = (n + kRows - 1) / kRows * chunks;
  const int64_t warps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
  for (int64_t task = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; task < tasks;
       task += warps) {
    const int64_t r0 = task / chunks * kRows;
    const int i = static_cast<int>(task % chunks) * 32 + lane;  // 8 values of the row
    const bool in = 8 * i < K;
    const int m = static_cast<int>(n - r0 < kRows ? n - r0 : kRows);
    uint4 v[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j)
      v[j] = in && j < m ? ld_stream(reinterpret_cast<const uint4*>(x + (r0 + j) * K) + i)
                         : make_uint4(0, 0, 0, 0);
    uint32_t word[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      uint32_t a = abs_max2(abs_max2(abs_max2(abs_max2(0u, v[j].x), v[j].y), v[j].z), v[j].w);
      a = max(a, __shfl_xor_sync(kFull, a, 1));
      a = max(a, __shfl_xor_sync(kFull, a, 2));
      const uint32_t byte = scale_byte(a);
      if (in && j < m)
        *reinterpret_cast<uint32_t*>(q + (r0 + j) * (K >> 1) + 4 * static_cast<int64_t>(i)) =
            codes8(v[j], scale_inverse(byte), byte == 255u);
      // the word of 128 values: four blocks' bytes, from lanes 0, 4, 8, 12 of 16
      uint32_t w = byte << (8 * ((lane >> 2) & 3));
      w |= __shfl_xor_sync(kFull, w, 4);
      w |= __shfl_xor_sync(kFull, w, 8);
      word[j] = w;
    }
    if ((lane & 15) == 0 && in) {
      uint32_t* s = reinterpret_cast<uint32_t*>(scale) + static_cast<int64_t>(i >> 4) * rows + r0;
      if (m == kRows && (rows & 3) == 0) {
        *reinterpret_cast<uint4*>(s) = make_uint4(word[0], word[1], word[2], word[3]);
      } else {
#pragma unroll
        for (int j = 0; j < kRows; ++j)
          if (j < m) s[j] = word[j];
      }
    }
  }
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
  // 2^-127 is a subnormal; 255 stands for NaN
  return byte == 255u ? __uint_as_float(0x7fc00000u)
                      : byte == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}

__device__ __forceinline__ uint32_t dequant2(uint32_t code2, float s) {
  const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(code2), __NV_E2M1);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16x2(f.x * s, f.y * s);
}

__global__ void __launch_bounds__(256) dequantize_rows_kernel(const uint8_t* __restrict__ q,
                                                              const uint8_t* __restrict__ scale,
                                                              uint16_t* __restrict__ x,
                                                              int64_t rows, int K) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int chunks = (K + 255) >> 8;
  const int64_t tasks = (rows + kRows - 1) / kRows * chunks;
  const int64_t warps = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5;
  for (int64_t task = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; task < tasks;
       task += warps) {
    const int64_t r0 = task / chunks * kRows;
    const int i = static_cast<int>(task % chunks) * 32 + lane;
    if (8 * i >= K) continue;
    const int m = static_cast<int>(rows - r0 < kRows ? rows - r0 : kRows);
    uint32_t c[kRows], w[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j)
      c[j] = j < m ? __ldcs(reinterpret_cast<const uint32_t*>(q + (r0 + j) * (K >> 1)) + i) : 0u;
    const uint32_t* s = reinterpret_cast<const uint32_t*>(scale) + static_cast<int64_t>(i >> 4) * rows + r0;
    if (m == kRows && (rows & 3) == 0) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(s));
      w[0] = u.x;
      w[1] = u.y;
      w[2] = u.z;
      w[3] = u.w;
    } else {
#pragma unroll
      for (int j = 0; j < kRows; ++j) w[j] = j < m ? __ldg(s + j) : 0u;
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const float f = scale_value((w[j] >> (8 * ((lane >> 2) & 3))) & 255u);
      if (j < m)
        st_global_cs_v4(reinterpret_cast<uint4*>(x + (r0 + j) * K) + i,
                        make_uint4(dequant2(c[j] & 255u, f), dequant2((c[j] >> 8) & 255u, f),
                                   dequant2((c[j] >> 16) & 255u, f), dequant2(c[j] >> 24, f)));
    }
  }
}

// Enough warps for every task, or 64 to an SM.
unsigned rows_grid(int64_t rows, int K, int num_sms) {
  const int64_t tasks = (rows + kRows - 1) / kRows * ((K + 255) / 256);
  const int64_t blocks = (tasks + 7) / 8;
  return static_cast<unsigned>(blocks < num_sms * 8 ? blocks : num_sms * 8);
}

// Weights W [E, K, N] -> Wq [E, N, K/2]: a block takes 64 columns x 128 k
// through shared memory; a thread then holds one column's 32 consecutive k.
__global__ void __launch_bounds__(256) quantize_weights_kernel(const uint16_t* __restrict__ W,
                                                               uint8_t* __restrict__ Wq,
                                                               uint8_t* __restrict__ w_scale,
                                                               int K, int N) {
  __shared__ uint16_t tile[128][64 + 2];
  const int e = blockIdx.z, n0 = blockIdx.x * 64, k0 = blockIdx.y * 128;
  const int tid = threadIdx.x;
  const int kn = min(128, K - k0);
  for (int i = tid; i < 128 * 32; i += 256) {
    const int r = i >> 5, c = (i & 31) * 2;
    uint32_t v = 0u;
    if (r < kn)
      v = *reinterpret_cast<const uint32_t*>(W + (static_cast<size_t>(e) * K + k0 + r) * N + n0 + c);
    *reinterpret_cast<uint32_t*>(&tile[r][c]) = v;
  }
  __syncthreads();
  const int c = tid >> 2, blk = tid & 3;
  const int n = n0 + c;
  uint32_t byte = 0u;
  if (blk * 32 < kn) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      m = max(m, (static_cast<uint32_t>(tile[blk * 32 + i][c]) << 16) & 0x7fff0000u);
    byte = scale_byte(m);
    const float inv = scale_inverse(byte);
    uint32_t w[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      uint4 v;
      const uint16_t(*t)[66] = &tile[blk * 32 + 8 * g];
      v.x = t[0][c] | (static_cast<uint32_t>(t[1][c]) << 16);
      v.y = t[2][c] | (static_cast<uint32_t>(t[3][c]) << 16);
      v.z = t[4][c] | (static_cast<uint32_t>(t[5][c]) << 16);
      v.w = t[6][c] | (static_cast<uint32_t>(t[7][c]) << 16);
      w[g] = codes8(v, inv, byte == 255u);
    }
    *reinterpret_cast<uint4*>(Wq + (static_cast<size_t>(e) * N + n) * (K >> 1) + (k0 >> 1) + blk * 16) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
  const size_t atom = (static_cast<size_t>(e) * ((N + 127) / 128) + n / 128) * ((K + 127) / 128) + k0 / 128;
  w_scale[atom * 512 + (n & 31) * 16 + ((n >> 5) & 3) * 4 + blk] = static_cast<uint8_t>(byte);
}

}  // namespace

cudaError_t launch_quantize_rows_mx4(const uint16_t* x, uint8_t* q, uint8_t* scale,
                                     const int32_t* n_rows, int64_t rows, int K, int num_sms,
                                     cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  return launch_pdl(quantize_rows_kernel, dim3(rows_grid(rows, K, num_sms)), dim3(256), 0, st, x, q,
                    scale, n_rows, rows, K);
}

cudaError_t launch_dequantize_rows_mx4(const uint8_t* q, const uint8_t* scale, uint16_t* x,
                                       int64_t rows, int K, int num_sms, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  return launch_pdl(dequantize_rows_kernel, dim3(rows_grid(rows, K, num_sms)), dim3(256), 0, st, q,
                    scale, x, rows, K);
}

cudaError_t launch_quantize_weights_mx4(const uint16_t* W, uint8_t* Wq, uint8_t* w_scale, int E,
                                        int K, int N, cudaStream_t st) {
  const size_t bytes = static_cast<size_t>(E) * ((N + 127) / 128) * ((K + 127) / 128) * 512;
  cudaError_t err = cudaMemsetAsync(w_scale, 0, bytes, st);  // columns past N, blocks past K
  if (err != cudaSuccess) return err;
  quantize_weights_kernel<<<dim3(N / 64, (K + 127) / 128, E), 256, 0, st>>>(W, Wq, w_scale, K, N);
  return cudaGetLastError();
}

}  // namespace moe
