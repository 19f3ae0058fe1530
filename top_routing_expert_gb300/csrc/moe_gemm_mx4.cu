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
// by TMA; those of the tokens start at any row (a segment need not begin at a
// multiple of anything), so two warps fetch them into registers, coalesced and
// stages ahead, and store them word by word in their places.
//
// Roles (640 threads): warp 0 = TMA producer, warp 1 = UMMA issuer and TMEM
// allocation, warps 2-3 = token scales, warps 4-19 = epilogue (four to a TMEM
// lane quadrant, taking chunks of 32 tokens in turn).
//
// CTA pairs (cta_group::2, M = 256) do the work, or single CTAs (M = 128) where
// there are too few columns for the pairs.
//
// Measured with a cold L2, and what bounds it: 65536 rows x 4096 x 14336 over 8
// experts 1.17 to 1.21 ms, 6.4 to 6.6 PFLOP/s, at 1.76 GHz under the power limit of
// 1373 W (1.07 and 7.2 in short runs); the tensor pipe works in 77 % of the clocks,
// the issuer waits for stages in 12 % and for accumulators in 5. 98304 x 1408 x 2048
// over 64 experts 137 to 140 us: tensor 44 %, waits 11 and 4 %, and the ends of tiles
// of 5.5 stages. 16 rows over 8 experts of 4096 x 14336 40 to 44 us, 5.0 to 5.5 TB/s of
// weights; 96 over 64 of 2048 x 1408 with GELU 22 to 23 us, 3.4 TB/s, and 8191 over 16
// of 1024 x 2816 with GELU 29 us: a start and an end of some 7 us around two to four
// rounds of tiles. Replayed from a graph, with weights left in L2, these three took
// 35, 16 and 26 us; the comparisons below are such replays.
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
constexpr int kScaleWarps = 2;
constexpr int kTokenWords = (kMaxTokens + 31) / 32;  // scale words per lane, block and tile
constexpr int kEpiWarps = 16;                        // four to a TMEM lane quadrant
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr uint32_t kChunkBytes = 1024;   // epilogue staging per warp: 16 tokens x 32 columns
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemSfX = 480;  // scales of a K block: the tokens', 2 x 8 columns,
constexpr uint32_t kTmemSfW = 496;  // and the weights', 2 x 4 columns per sub-tile

__host__ __device__ constexpr uint32_t x_scale_blocks(int nt) { return static_cast<uint32_t>(nt + 127) / 128; }
// A stage: the weights' codes (128 rows, twice in a pair), the tokens' (half of
// them in a pair), the weights' scales, the tokens' scales; every part is a
// multiple of 1024 bytes.
__host__ __device__ constexpr uint32_t stage_bytes(int nt, bool pair) {
  return (kWBytes + kWScaleBytes) * (pair ? 2 : 1) + static_cast<uint32_t>(nt) * (pair ? 64 : 128) +
         2 * 512 * x_scale_blocks(nt);
}

// The epilogue's two halves, for one warp's 32 output columns x 32 tokens. The
// accumulator has output columns in lanes and tokens in columns; it is read as
// 8x8 fragments and rounded to bf16, two tokens to a register (m[4g + c]: tokens
// 8g .. 8g + 7, columns 8c .. 8c + 7).
__device__ __forceinline__ void load_chunk(uint32_t taddr, int gelu, uint32_t (&m)[16]) {
  uint32_t a[16], b[16];
  tmem_ld_16x256b_x4(taddr, a);
  tmem_ld_16x256b_x4(taddr + (16u << 16), b);
  tmem_ld_wait();
  if (gelu) {
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      gelu_tanh_x2(a[i], a[i + 1]);
      gelu_tanh_x2(b[i], b[i + 1]);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m[(i >> 1) * 4 + (i & 1)] = pack_bf16x2(__uint_as_float(a[2 * i]), __uint_as_float(a[2 * i + 1]));
    m[(i >> 1) * 4 + 2 + (i & 1)] = pack_bf16x2(__uint_as_float(b[2 * i]), __uint_as_float(b[2 * i + 1]));
  }
}

// Half a chunk (h) to shared memory, transposed: [16 tokens][32 columns], 64-byte
// rows in TMA's 64-byte swizzle, which also keeps the 16-byte pieces of eight
// tokens in different banks.
__device__ __forceinline__ void stage_half(const uint32_t (&m)[16], int h, uint32_t buf, int lane) {
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const uint32_t t = 8u * g + (lane & 7), c = static_cast<uint32_t>(lane) >> 3;
    const int f = 4 * (2 * h + g);
    stmatrix_x4_trans(buf + 64u * t + 16u * (c ^ ((t >> 1) & 3u)), m[f], m[f + 1], m[f + 2], m[f + 3]);
  }
}

// The first n (under 16) tokens of a staged half to D.
__device__ __forceinline__ void store_rows(uint32_t buf, uint16_t* d, int pitch, int n, int lane) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t t = 8u * i + (static_cast<uint32_t>(lane) >> 2), c = lane & 3;
    const uint4 v = ld_shared_v4(buf + 64u * t + 16u * (c ^ ((t >> 1) & 3u)));
    if (static_cast<int>(t) < n) st_global_cs_v4(d + static_cast<size_t>(t) * pitch + 8 * c, v);
  }
}

// A value that is the same in all lanes of the warp, made known as such: it and
// what is computed from it stay in uniform registers, which tcgen05
// instructions take their operands from.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

struct Tile {
  int e, row0, row_end, n0;  // at most tile_tokens rows, at least one
};

// Tile order: groups of 8 token tiles, all column tiles of a group before the
// next group, token tiles innermost (they share the weights in L2).
__device__ __forceinline__ Tile decode(int L, const int* prefix, const int* offs, int E, int total_t,
                                       int n_tiles_n, int nt, int bm = kBM) {
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
  // the expert's rows go evenly over its tiles, in 16s: the last is shorter by the
  // roundings alone (8192 rows: 34 tiles of 240 and one of 32)
  const int rows = offs[lo + 1] - offs[lo], tiles = prefix[lo + 1] - prefix[lo];
  const int each = ((rows + tiles - 1) / tiles + 15) & ~15;
  Tile t;
  t.e = lo;
  t.row0 = offs[lo] + (tt - prefix[lo]) * each;
  t.row_end = min(t.row0 + each, offs[lo + 1]);
  t.n0 = (r / gsz) * bm;
  return t;
}

// The tiles unit, unit + units, ... of one warp, in order. Decoding one takes
// several hundred clocks (divisions, a search): the lanes decode 32 at a time.
struct Tiles {
  const int *prefix, *offs;
  int E, total_t, total, n_tiles_n, nt, bm, unit, units;
  int i = 0;      // the next tile is unit + i * units
  Tile mine;
  // Called by the whole warp; false after the last tile. The result is uniform.
  __device__ __forceinline__ bool next(Tile& t) {
    if (unit + i * units >= total) return false;
    if ((i & 31) == 0) {
      const int L = unit + (i + static_cast<int>(threadIdx.x & 31)) * units;
      if (L < total) mine = decode(L, prefix, offs, E, total_t, n_tiles_n, nt, bm);
    }
    t.e = __shfl_sync(0xffffffffu, mine.e, i & 31);
    t.row0 = __shfl_sync(0xffffffffu, mine.row0, i & 31);
    t.row_end = __shfl_sync(0xffffffffu, mine.row_end, i & 31);
    t.n0 = __shfl_sync(0xffffffffu, mine.n0, i & 31);
    ++i;
    return true;
  }
};

// Segment offsets, held to the buffer and non-decreasing, and the prefix of the
// experts' token tiles, by one warp; followed by a barrier of the caller's. (One
// thread going through 64 offsets in shared memory took 2 us.)
__device__ __forceinline__ void prefix_tiles(const int* offs, int* prefix, int E, int nt) {
  const int lane = threadIdx.x & 31;
  int tiles = 0;
  for (int b = 0; b <= E; b += 32) {
    const int i = b + lane;  // the tiles of expert i - 1, and through it
    int n = i > 0 && i <= E ? (offs[i] - offs[i - 1] + nt - 1) / nt : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) n += u;
    }
    if (i <= E) prefix[i] = tiles + n;
    tiles += __shfl_sync(0xffffffffu, n, 31);
  }
  __syncwarp();
}

// Tile size where the tiles are so few that the last round of them over the
// units counts: lane c tries 16 c tokens less than the widest, at the cost of its
// rounds times its size and 300 tokens' worth, which a round of tiles of any size
// costs about. With this and without, in us: 2048 rows of 8 experts (4096 x 1024)
// 13.6, 15.2; 8191 skewed rows of 16 (1024 x 2816, GELU) 25.9, 27.4; 4096 rows of
// 4 (2048 x 2048, GELU) 17.0, 19.7; but 8191 rows of 8 16.7, 16.3. Shorter
// segments lose by it (2048 rows of 64 experts 27.1, 25.1) and keep the widest.
__device__ __forceinline__ int choose_tile(const int* offs, int E, int nt, int n_tiles_n, int units) {
  const int lane = threadIdx.x & 31;
  const int cand = nt - 16 * (lane & 15);
  int tiles = 0;
  if (cand >= 64) {
    const float inv = 1.0f / static_cast<float>(cand);
    for (int e = 0; e < E; ++e)  // a ceiling to within a rounding: an estimate
      tiles += static_cast<int>(ceilf(static_cast<float>(offs[e + 1] - offs[e]) * inv));
  }
  const int rounds = (tiles * n_tiles_n + units - 1) / units;
  uint32_t key = cand >= 64 ? (static_cast<uint32_t>(rounds) * static_cast<uint32_t>(cand + 300)) << 4 | (lane & 15u)
                            : 0xffffffffu;
  key = __reduce_min_sync(0xffffffffu, key);
  return nt - 16 * static_cast<int>(key & 15u);
}

__device__ __forceinline__ void load_offsets(const Mx4GemmArgs& p, int* offs, int* prefix, int nt,
                                             int n_tiles_n, int units) {
  const int lane = threadIdx.x & 31, E = p.E;
  int last = 0;  // offs[b - 1]
  for (int b = 0; b <= E; b += 32) {
    const int i = b + lane;
    int v = i <= E ? p.offsets[i] : 0;
    v = v < 0 ? 0 : (v > p.rows ? p.rows : v);  // rows outside the buffer are never touched
    v = max(v, last);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = max(v, u);
    }
    if (i <= E) offs[i] = v;
    last = __shfl_sync(0xffffffffu, v, 31);
  }
  __syncwarp();
  prefix_tiles(offs, prefix, E, nt);
  if (p.rows >= 256 * E && E <= 64 && prefix[E] * n_tiles_n <= 8 * units) {
    const int fit = choose_tile(offs, E, nt, n_tiles_n, units);
    if (fit != nt) prefix_tiles(offs, prefix, E, fit);
  }
}

// What the UMMAs of one K block of a sub-tile read; all uniform.
struct Block {
  uint64_t w, x, ws, xs;    // descriptors: codes and scales, of the weights and the tokens
  uint32_t d;               // accumulator
  uint32_t sf_w, sf_x;      // scales in TMEM
  uint32_t idesc0, idesc1;  // for scale bytes 0-1 and 2-3 of a word
  uint32_t add;             // 0: the accumulator starts here
};

// Issues a K block of 256: its scales to TMEM, then four UMMAs of 64 (which wait
// for them in order). Called by the whole warp; straight-line code, so that one
// elected lane issues an instruction about every 20 clocks (with the branches on
// sizes inside, about 36, too slow for 120-clock UMMAs with their scales).
template <bool kPair, bool kWide>
__device__ __forceinline__ void issue_block(const Block& b, uint64_t* release) {
  if (elect_one()) {
    tmem_cp<kPair>(b.sf_w, b.ws);
    tmem_cp<kPair>(b.sf_x, b.xs);
    if constexpr (kWide) {  // more than 128 tokens: two blocks of scales
      tmem_cp<kPair>(b.sf_x + 4u, b.xs + 32u);
      tmem_cp<kPair>(b.sf_x + 8u, b.xs + 64u);
      tmem_cp<kPair>(b.sf_x + 12u, b.xs + 96u);
    } else {
      tmem_cp<kPair>(b.sf_x + 8u, b.xs + 32u);
    }
    tmem_cp<kPair>(b.sf_w + 4u, b.ws + 32u);
    umma_mxf4<kPair>(b.d, b.w, b.x, b.idesc0, b.sf_w, b.sf_x, b.add);
    umma_mxf4<kPair>(b.d, b.w + 2u, b.x + 2u, b.idesc1, b.sf_w, b.sf_x, 1u);
    umma_mxf4<kPair>(b.d, b.w + 4u, b.x + 4u, b.idesc0, b.sf_w + 4u, b.sf_x + 8u, 1u);
    umma_mxf4<kPair>(b.d, b.w + 6u, b.x + 6u, b.idesc1, b.sf_w + 4u, b.sf_x + 8u, 1u);
    if (release != nullptr) {
      if constexpr (kPair) umma_commit_pair_multicast(release, 0x3);
      else umma_commit(release);
    }
  }
  __syncwarp();
}

// A K block of both sub-tiles (b: sub-tile A's, whose descriptors and addresses
// lead to B's), with the tokens' scales copied once.
template <bool kWide>
__device__ __forceinline__ void issue_block_ab(const Block& b, uint32_t d_b, uint64_t* release) {
  constexpr uint32_t kW = kWBytes >> 4, kS = kWScaleBytes >> 4;
  if (elect_one()) {
    tmem_cp<true>(b.sf_w, b.ws);
    tmem_cp<true>(b.sf_x, b.xs);
    if constexpr (kWide) {
      tmem_cp<true>(b.sf_x + 4u, b.xs + 32u);
      tmem_cp<true>(b.sf_x + 8u, b.xs + 64u);
      tmem_cp<true>(b.sf_x + 12u, b.xs + 96u);
    } else {
      tmem_cp<true>(b.sf_x + 8u, b.xs + 32u);
    }
    tmem_cp<true>(b.sf_w + 4u, b.ws + 32u);
    tmem_cp<true>(b.sf_w + 8u, b.ws + kS);
    tmem_cp<true>(b.sf_w + 12u, b.ws + kS + 32u);
    umma_mxf4<true>(b.d, b.w, b.x, b.idesc0, b.sf_w, b.sf_x, b.add);
    umma_mxf4<true>(b.d, b.w + 2u, b.x + 2u, b.idesc1, b.sf_w, b.sf_x, 1u);
    umma_mxf4<true>(b.d, b.w + 4u, b.x + 4u, b.idesc0, b.sf_w + 4u, b.sf_x + 8u, 1u);
    umma_mxf4<true>(b.d, b.w + 6u, b.x + 6u, b.idesc1, b.sf_w + 4u, b.sf_x + 8u, 1u);
    umma_mxf4<true>(d_b, b.w + kW, b.x, b.idesc0, b.sf_w + 8u, b.sf_x, b.add);
    umma_mxf4<true>(d_b, b.w + kW + 2u, b.x + 2u, b.idesc1, b.sf_w + 8u, b.sf_x, 1u);
    umma_mxf4<true>(d_b, b.w + kW + 4u, b.x + 4u, b.idesc0, b.sf_w + 12u, b.sf_x + 8u, 1u);
    umma_mxf4<true>(d_b, b.w + kW + 6u, b.x + 6u, b.idesc1, b.sf_w + 12u, b.sf_x + 8u, 1u);
    umma_commit_pair_multicast(release, 0x3);
  }
  __syncwarp();
}

// The last K block of a tile when it is 64, 128 or 192 deep.
template <bool kPair>
__device__ __noinline__ void issue_tail(const Block& b, int steps, bool wide, uint64_t* release) {
  if (elect_one()) {
    for (uint32_t h = 0; 2 * h < static_cast<uint32_t>(steps); ++h) {
      tmem_cp<kPair>(b.sf_w + 4u * h, b.ws + 32u * h);
      tmem_cp<kPair>(b.sf_x + 8u * h, b.xs + (wide ? 64u : 32u) * h);
      if (wide) tmem_cp<kPair>(b.sf_x + 8u * h + 4u, b.xs + 64u * h + 32u);
    }
    for (uint32_t q = 0; q < static_cast<uint32_t>(steps); ++q)
      umma_mxf4<kPair>(b.d, b.w + 2u * q, b.x + 2u * q, (q & 1u) ? b.idesc1 : b.idesc0,
                       b.sf_w + 4u * (q >> 1), b.sf_x + 8u * (q >> 1), q == 0 ? b.add : 1u);
    if (release != nullptr) {
      if constexpr (kPair) umma_commit_pair_multicast(release, 0x3);
      else umma_commit(release);
    }
  }
  __syncwarp();
}

// kPair: a tile is 512 output columns x up to tile_tokens tokens on a cluster
// pair, as two sub-tiles A and B of 256 columns (128 per CTA) that share the
// tokens of a stage, each with an accumulator of its own. Per CTA a stage then
// brings 49 KB for 960 clocks of UMMAs, 51 bytes a clock at the full rate (40 at the
// large product's) of the 64 or so that an SM takes in from L2 (one 256-column
// sub-tile alone: 34 KB for 480, 71).
// Each CTA loads half of the tokens' codes and all of their scales, and the
// leader (rank 0) issues the UMMAs, so stage barriers of both CTAs' copies live
// there.
// Otherwise a tile is 128 columns of one CTA, its accumulators used in turn.
template <bool kPair>
__global__ void __launch_bounds__(kThreads, 1)
    expert_gemm_mx4_kernel(const __grid_constant__ CUtensorMap tm_w,
                           const __grid_constant__ CUtensorMap tm_x,
                           const __grid_constant__ CUtensorMap tm_ws,
                           const __grid_constant__ CUtensorMap tm_d, Mx4GemmArgs p) {
  constexpr int kCtas = kPair ? 2 : 1;
  constexpr int kSubs = kPair ? 2 : 1;           // sub-tiles per tile
  constexpr int kSubN = kBM * kCtas;             // columns of a sub-tile, M of the UMMA
  constexpr int kTileN = kSubN * kSubs;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_up_1024(smem_raw);
  const int nst = p.stages, NT = p.tile_tokens;
  const uint32_t sb = stage_bytes(NT, kPair);
  const uint32_t xbytes = static_cast<uint32_t>(NT) * 128 / kCtas;  // a multiple of 1024
  uint8_t* staging = smem + static_cast<size_t>(nst) * sb;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kEpiWarps * kChunkBytes);
  uint64_t* empty = full + nst;
  uint64_t* tfull = empty + nst;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint64_t* xbar = drain + 1;  // pair leader: the peer's count of loaded stages has arrived
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(xbar + 1);
  uint32_t* abort_flag = tmem_slot + 1;
  uint32_t* peer_issued = abort_flag + 1;
  int* offs = reinterpret_cast<int*>(peer_issued + 1);  // [E+1]
  int* prefix = offs + (p.E + 1);                       // [E+1]

  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  const int E = p.E;
  const uint32_t rank = kPair ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  const int unit = blockIdx.x / kCtas, units = gridDim.x / kCtas;
  if (warp == 1) {
    if constexpr (kPair) {
      tmem_alloc_pair(tmem_slot, kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, kTmemCols);
      tmem_relinquish();
    }
  }
  if (warp == 2 && lane == 0) {
    for (int s = 0; s < nst; ++s) {
      mbar_init(&full[s], 1 + kCtas * kScaleWarps);  // the bytes, and the scale warps
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], kCtas * 32 * kEpiWarps);
    }
    mbar_init(drain, 1);
    mbar_init(xbar, 1);
    *abort_flag = 0u;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_ws);
    tma_prefetch_desc(&tm_d);
  }
  grid_dependency_wait();
  grid_launch_dependents();
  const int n_tiles_n = (p.N + kTileN - 1) / kTileN;
  if (warp == 0) load_offsets(p, offs, prefix, NT, n_tiles_n, units);
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) cluster_sync();  // barriers initialised before any remote use
  tc_fence_after();

  const uint32_t tmem_base = static_cast<uint32_t>(uniform(static_cast<int>(*tmem_slot)));
  const int total_t = uniform(prefix[E]);
  const int total = total_t * n_tiles_n;
  const int nk = (p.K + kStageK - 1) / kStageK;   // stages per tile
  const int nkb = (p.K + 127) / 128;              // 128-deep scale blocks
  Tiles tiles{prefix, offs, E, total_t, total, n_tiles_n, NT, kTileN, unit, units};
  Tile c;
  const WaitCtl wc{abort_flag, p.dev_status, p.timeout_ns};
  // A wait that gives up stops the peer CTA too.
  const uint32_t peer_abort = kPair ? mapa_shared(smem_u32(abort_flag), rank ^ 1u) : 0u;
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (mbar_wait(bar, parity, wc)) return true;
    if constexpr (kPair) st_u32_cluster(peer_abort, 1u);
    return false;
  };
  const uint32_t full0 = kPair ? mapa_shared(smem_u32(full), 0) : smem_u32(full);

  if (warp == 0) {
    // ------------------------------------------------ TMA producer ----
    int stage = 0;
    uint32_t phase = 0;
    int issued = 0;
    bool aborted = false;
    const uint32_t bytes = kSubs * (kWBytes + kWScaleBytes) + xbytes;  // per CTA and stage
    const int s_none = E * ((p.N + kBM - 1) / kBM) * nkb;  // past the end: reads as zeros
    while (!aborted && tiles.next(c)) {
      const int half = ((c.row_end - c.row0 + 15) & ~15) >> 1;
      const int n0 = c.n0 + static_cast<int>(rank) * kBM;
      const int x_row = c.row0 + (kPair ? static_cast<int>(rank) * half : 0);
      // scale blocks of this CTA's 128 columns (past N or K: others', unused)
      const int s_row = (c.e * ((p.N + kBM - 1) / kBM) + n0 / kBM) * nkb;
      for (int kb = 0; kb < nk; ++kb) {
        if (!__all_sync(0xffffffffu, wait(&empty[stage], phase ^ 1u))) {
          aborted = true;
          break;
        }
        if (elect_one()) {
          uint8_t* sw = smem + static_cast<size_t>(stage) * sb;
          uint8_t* sx = sw + kSubs * kWBytes;
          if (leader) mbar_arrive_expect_tx(&full[stage], kCtas * bytes);
          if constexpr (kPair) {
            const uint32_t bar = full0 + 8u * static_cast<uint32_t>(stage);
            tma_load_2d_pair(sw, &tm_w, bar, kb * 128, c.e * p.N + n0);
            tma_load_2d_pair(sx, &tm_x, bar, kb * 128, x_row);
            tma_load_2d_pair(sx + xbytes, &tm_ws, bar, 0, s_row + 2 * kb);
            // sub-tile B, if N reaches that far (else zeros, without memory traffic)
            const bool b = c.n0 + kSubN < p.N;
            tma_load_2d_pair(sw + kWBytes, &tm_w, bar, kb * 128, b ? c.e * p.N + n0 + kSubN : E * p.N);
            tma_load_2d_pair(sx + xbytes + kWScaleBytes, &tm_ws, bar, 0,
                             b ? s_row + (kSubN / kBM) * nkb + 2 * kb : s_none);
          } else {
            tma_load_2d(sw, &tm_w, &full[stage], kb * 128, c.e * p.N + n0);
            tma_load_2d(sx, &tm_x, &full[stage], kb * 128, x_row);
            tma_load_2d(sx + xbytes, &tm_ws, &full[stage], 0, s_row + 2 * kb);
          }
        }
        __syncwarp();
        ++issued;
        if (++stage == nst) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (lane == 0) {
      // Every load issued lands before any CTA can exit. In a pair the peer
      // reports how many stages it loaded, and the leader makes the byte
      // accounting of each stage still in flight whole before it waits for it
      // (after an abort one CTA may have loaded stages that the other did not).
      if (kPair && !leader) {
        st_async_u32_cluster(mapa_shared(smem_u32(peer_issued), 0), static_cast<uint32_t>(issued),
                             mapa_shared(smem_u32(xbar), 0));
      } else {
        int theirs = issued;
        if constexpr (kPair) {
          mbar_arrive_expect_tx(xbar, 4);
          if (mbar_wait_drain(xbar, 0, p.timeout_ns + kDrainLimitNs)) {
            // the peer cannot load more than a ring ahead of what this CTA armed
            theirs = min(static_cast<int>(*reinterpret_cast<volatile uint32_t*>(peer_issued)),
                         issued + nst);
          } else {
            atomicOr(p.dev_status, MOE_DEV_TIMEOUT);
          }
        }
        const int hi = max(issued, theirs);
        for (int i = max(0, hi - nst); i < hi; ++i) {
          uint64_t* b = &full[i % nst];
          if (i >= issued)
            mbar_arrive_expect_tx(b, bytes);  // armed here for the peer's half alone
          else if (i >= theirs)
            mbar_complete_tx(b, bytes);       // the peer's half will never come
          mbar_wait_drain(b, static_cast<uint32_t>(i / nst) & 1u, kDrainLimitNs);
        }
      }
    }
  } else if (warp == 1) {
    if (leader) {
      // ------------------------------------------------- UMMA issuer ----
      // The whole warp runs this converged and one elected lane issues: the
      // descriptors then stay in uniform registers. From a branch on lane 0
      // each tcgen05 instruction took about 44 clocks to issue, ten a stage
      // against the 480 clocks of its four UMMAs; elected, about 10.
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;             // the accumulator of sub-tile A
      uint32_t acc_phase = 0;  // bit a: parity of accumulator a's next use
      bool aborted = false;
      const uint32_t s0 = smem_u32(smem);
      const uint64_t w_desc = smem_desc_sw128(s0, 16u, 1024u);
      const uint64_t x_desc = smem_desc_sw128(s0 + kSubs * kWBytes, 16u, 1024u);
      const uint64_t ws_desc = smem_desc_plain(s0 + kSubs * kWBytes + xbytes, 128u);
      const uint64_t xs_desc =
          smem_desc_plain(s0 + kSubs * (kWBytes + kWScaleBytes) + xbytes, 128u);
      const uint32_t sf_w = tmem_base + kTmemSfW, sf_x = tmem_base + kTmemSfX;
      const bool wide = NT > 128;  // two blocks of token scales
      uint32_t idesc = 0;
      // the UMMAs of sub-tile `sub` for K block kb, which lies in ring slot `st`,
      // into accumulator `a`; `release`: the slot is free once they are done
      auto block = [&](int st, int kb, uint32_t sub, int a) {
        const uint64_t so = static_cast<uint64_t>(static_cast<uint32_t>(st) * (sb >> 4));
        Block k;
        k.w = w_desc + so + sub * (kWBytes >> 4);
        k.x = x_desc + so;
        k.ws = ws_desc + so + sub * (kWScaleBytes >> 4);
        k.xs = xs_desc + so;
        k.d = tmem_base + static_cast<uint32_t>(a * kMaxTokens);
        k.sf_w = sf_w + 8u * sub;
        k.sf_x = sf_x;
        k.idesc0 = idesc;
        k.idesc1 = idesc | (2u << 4) | (2u << 29);
        k.add = kb != 0 ? 1u : 0u;
        return k;
      };
      auto issue = [&](int st, int kb, uint32_t sub, int a, bool release) {
        const Block k = block(st, kb, sub, a);
        uint64_t* bar = release ? &empty[st] : nullptr;
        const int steps = (p.K - kb * kStageK) / 64;
        if (steps >= 4) {
          if (wide) issue_block<kPair, true>(k, bar);
          else issue_block<kPair, false>(k, bar);
        } else {
          issue_tail<kPair>(k, steps, wide, bar);
        }
      };
      auto finish = [&](int a) {  // accumulator a is complete
        if (elect_one()) {
          if constexpr (kPair) umma_commit_pair_multicast(&tfull[a], 0x3);
          else umma_commit(&tfull[a]);
        }
        __syncwarp();
      };
      auto acquire = [&](int a) -> bool {  // accumulator a has been drained
        const bool ok = __all_sync(0xffffffffu, wait(&tempty[a], ((acc_phase >> a) & 1u) ^ 1u));
        acc_phase ^= 1u << a;
        tc_fence_after();
        return ok;
      };
      while (!aborted && tiles.next(c)) {
        const int n_tok = c.row_end - c.row0;
        idesc = idesc_mxf4_e8m0(kSubN, static_cast<uint32_t>((n_tok + 15) & ~15));
        const bool b = kPair && c.n0 + kSubN < p.N;
        if (!acquire(acc)) break;
        int b_kb = 0, b_stage = stage;  // the next K block of B
        for (int kb = 0; kb < nk; ++kb) {
          // cluster scope: the peer's scale warps arrive here too
          if (!__all_sync(0xffffffffu, mbar_wait<kPair>(&full[stage], phase, wc))) {
            if constexpr (kPair) st_u32_cluster(peer_abort, 1u);
            aborted = true;
            break;
          }
          fence_proxy_async();  // the scale warps' stores, before tcgen05.cp reads them
          tc_fence_after();
          // B goes with A, block by block. While B's accumulator is still being drained
          // A goes on alone, as far as the ring holds the blocks that B has to come
          // back to. (Letting A run ahead at a tile's end too cost more in issue than
          // it hid: 6 us more on 98304 x 1408 x 2048.)
          bool hold = false;
          if (b && b_kb == 0 && kb < nk - 1 && kb + 2 <= nst)
            hold = !__all_sync(0xffffffffu, mbar_try_wait(&tempty[1], ((acc_phase >> 1) & 1u) ^ 1u));
          if (kPair && b && !hold && b_kb == kb && kb != nk - 1) {
            if (kb == 0 && !acquire(1)) {
              aborted = true;
              break;
            }
            const Block k = block(stage, kb, 0u, 0);
            if (wide) issue_block_ab<true>(k, k.d + kMaxTokens, &empty[stage]);
            else issue_block_ab<false>(k, k.d + kMaxTokens, &empty[stage]);
            ++b_kb;
            if (++stage == nst) {
              stage = 0;
              phase ^= 1u;
            }
            b_stage = stage;
            continue;
          }
          issue(stage, kb, 0u, acc, !b);
          if (kb == nk - 1) finish(acc);
          if (++stage == nst) {
            stage = 0;
            phase ^= 1u;
          }
          if (b && !hold) {
            if (b_kb == 0 && !acquire(1)) {
              aborted = true;
              break;
            }
            for (; b_kb <= kb; ++b_kb) {
              issue(b_stage, b_kb, 1u, 1, true);
              if (++b_stage == nst) b_stage = 0;
            }
          }
        }
        if (aborted) break;
        if (b) finish(1);
        if constexpr (!kPair) acc ^= 1;
      }
      // every UMMA issued must finish before TMEM is released
      if (elect_one()) {
        if constexpr (kPair) umma_commit_pair(drain);
        else umma_commit(drain);
      }
      __syncwarp();
      mbar_wait_drain(drain, 0, kDrainLimitNs);
    }
  } else if (warp < 2 + kScaleWarps) {
    // ---------------------------------------------------- token scales ----
    // Each of the two warps has one of a stage's two 128-deep blocks. Words are
    // fetched kAhead stages before their place in shared memory is free (the
    // loads' latency passes meanwhile), then stored and released.
    constexpr int kAhead = 4;
    const int h = warp - 2;
    const uint32_t* xs = reinterpret_cast<const uint32_t*>(p.x_scale);
    const uint32_t dst0 = smem_u32(smem) + kSubs * (kWBytes + kWScaleBytes) + xbytes +
                          512u * x_scale_blocks(NT) * static_cast<uint32_t>(h) + 16u * lane;
    const int n_stages = (total > unit ? (total - 1 - unit) / units + 1 : 0) * nk;
    int fkb = 0;  // the next K block to fetch, of the current tile
    bool f_more = true;
    const uint32_t* f_src = nullptr;
    int f_tok = 0;
    auto fetch = [&](uint32_t(&v)[kTokenWords]) {
      if (fkb == 0 && f_more) {
        f_more = tiles.next(c);
        f_tok = c.row_end - c.row0;
        f_src = xs + static_cast<size_t>(h) * p.rows + c.row0;
      }
      if (!f_more) return;
      const bool in = 2 * fkb + h < nkb;
#pragma unroll
      for (int m = 0; m < kTokenWords; ++m)
        v[m] = in && 32 * m + lane < f_tok ? __ldg(f_src + 32 * m + lane) : 0u;
      f_src += 2 * static_cast<size_t>(p.rows);
      if (++fkb == nk) fkb = 0;
    };
    uint32_t v[kAhead][kTokenWords];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) fetch(v[a]);
    int stage = 0;
    uint32_t phase = 0;
    bool aborted = false;
    for (int i = 0; i < n_stages && !aborted; i += kAhead) {
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        if (i + a < n_stages && !aborted) {
          if (!__all_sync(0xffffffffu, wait(&empty[stage], phase ^ 1u))) {
            aborted = true;
          } else {
            // token t of a block of 128: TMEM lane t % 32, word t / 32
            const uint32_t dst = dst0 + static_cast<uint32_t>(stage) * sb;
#pragma unroll
            for (int m = 0; m < kTokenWords; ++m)
              if (32 * m < NT) st_shared_u32(dst + 512u * (m >> 2) + 4u * (m & 3), v[a][m]);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
              // The leader's UMMA issuer has the tensor cores of both CTAs read them, so it
              // acquires at cluster scope, and they are released there. (A release of all
              // memory would wait for the loads in flight: 3.56 ms instead of 1.40 on
              // 65536 x 4096 x 14336, in an early form. By a warp without loads it still
              // takes 1250 to 3850 clocks under the copies' traffic: 1.34 instead of 1.20.)
              if constexpr (kPair) mbar_arrive_release_shared(full0 + 8u * static_cast<uint32_t>(stage));
              else mbar_arrive(&full[stage]);
            }
            fetch(v[a]);
            if (++stage == nst) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------ epilogue ----
    // warp w reads TMEM lanes 32 (w % 4) .. + 31, i.e. 32 output columns, and every
    // fourth chunk of 32 tokens, which it stages 16 at a time for TMA to store
    // (stores of 16 bytes a lane made the large product 14 % slower; 64 columns of
    // two warps at a time cost more in their barriers than longer rows gained).
    // With 8 warps instead of 16 the ragged product with GELU took 4 us more.
    const int q = warp & 3, part = (warp - 4) >> 2;
    const uint32_t buf = smem_u32(staging + (warp - 4) * kChunkBytes);
    const uint32_t tempty0 = kPair ? mapa_shared(smem_u32(tempty), 0) : 0u;
    int acc = 0;
    uint32_t acc_phase = 0;  // bit a: parity of accumulator a's next use
    bool aborted = false;
    while (!aborted && tiles.next(c)) {
      const int n_tok = c.row_end - c.row0;
      for (int sub = 0; sub < kSubs; ++sub) {
        if (sub > 0 && c.n0 + kSubN >= p.N) break;
        const int a = kPair ? sub : acc;
        if (!__all_sync(0xffffffffu, wait(&tfull[a], (acc_phase >> a) & 1u))) {
          aborted = true;
          break;
        }
        acc_phase ^= 1u << a;
        __syncwarp();
        tc_fence_after();
        const int n = c.n0 + sub * kSubN + static_cast<int>(rank) * kBM + 32 * q;
        const uint32_t t_base = tmem_base + (static_cast<uint32_t>(32 * q) << 16) +
                                static_cast<uint32_t>(a * kMaxTokens);
        // Everything is read out of TMEM and the accumulator handed back before
        // anything is stored: its next use waits for the reads alone.
        constexpr int kChunks = (kMaxTokens + 127) / 128;
        uint32_t m[kChunks][16];
        const bool any = n < p.N;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const int j = 128 * i + 32 * part;
          if (any && j < n_tok) load_chunk(t_base + static_cast<uint32_t>(j), p.gelu, m[i]);
        }
        tc_fence_before();
        if constexpr (kPair) mbar_arrive_cluster(tempty0 + 8u * static_cast<uint32_t>(a));
        else mbar_arrive(&tempty[a]);
#pragma unroll
        for (int i = 0; i < 2 * kChunks; ++i) {
          const int j = 128 * (i >> 1) + 32 * part + 16 * (i & 1);
          if (any && j < n_tok) {
            if (lane == 0) tma_store_wait_read();
            __syncwarp();
            stage_half(m[i >> 1], i & 1, buf, lane);
            fence_proxy_async();
            __syncwarp();
            if (n_tok - j >= 16) {
              if (lane == 0) tma_store_2d(&tm_d, buf, n, c.row0 + j);
            } else {  // rows past the segment belong to the next expert
              store_rows(buf, p.D + static_cast<size_t>(c.row0 + j) * p.N + n, p.N, n_tok - j, lane);
            }
          }
        }
      }
      if constexpr (!kPair) acc ^= 1;
    }
    if (lane == 0) tma_store_wait();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) cluster_sync();  // neither CTA leaves while the peer may still signal it
  tc_fence_after();
  if (warp == 1) {
    if constexpr (kPair) tmem_dealloc_pair(tmem_base, kTmemCols);
    else tmem_dealloc(tmem_base, kTmemCols);
  }
}

size_t smem_bytes(int E, int stages, int nt, bool pair) {
  return 1024 + static_cast<size_t>(stages) * stage_bytes(nt, pair) + kEpiWarps * kChunkBytes +
         8 * (2 * stages + 6) + 16 + 8 * static_cast<size_t>(E + 1);
}

}  // namespace

// Twice the average rows of an expert plus 8 hold almost any decoding batch's
// segments in one tile; larger averages take the widest tile.
int mx4_tile_tokens(int64_t rows, int E) {
  const int64_t want = (2 * rows / E + 8 + 15) / 16 * 16;
  return want < kMaxTokens ? static_cast<int>(want) : kMaxTokens;
}

// A pair of CTAs reads each tile's tokens once for 512 columns and has the better
// rate, unless there are so few columns that the pairs get less than 1.5 tiles
// each. In us, pairs against single CTAs: 64 experts of 2048 x 1408 (2.3 tiles)
// 15.8, 18.0 at 96 rows and 22.5, 24.8 at 1024; 16 of 4096 x 4096 (1.7 tiles) 28.4,
// 31.7 at 128 rows; 16 of 1024 x 2816 (1.2) 10.4, 9.4 at 128 rows and 11.8, 10.8
// at 1024. Long segments are what the pair is made for.
bool mx4_use_pair(int64_t rows, int E, int64_t N, int num_sms) {
  return rows >= 64 * static_cast<int64_t>(E) || 2 * E * N >= 3 * 512 * (num_sms / 2);
}

template <bool kPair>
static cudaError_t launch_mx4(const CUtensorMap& tm_w, const CUtensorMap& tm_x,
                              const CUtensorMap& tm_ws, const CUtensorMap& tm_d,
                              const Mx4GemmArgs& a, int num_sms, cudaStream_t st) {
  int dev = 0, optin = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  err = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  if (err != cudaSuccess) return err;
  Mx4GemmArgs args = a;
  args.stages = kMaxStages;
  while (args.stages > 3 &&  // the pair holds up to three slots at a tile's end
         smem_bytes(a.E, args.stages, a.tile_tokens, kPair) > static_cast<size_t>(optin))
    --args.stages;
  const size_t smem = smem_bytes(a.E, args.stages, a.tile_tokens, kPair);
  err = cudaFuncSetAttribute(expert_gemm_mx4_kernel<kPair>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(kPair ? 2 * (num_sms / 2) : num_sms), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kPair ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, expert_gemm_mx4_kernel<kPair>, tm_w, tm_x, tm_ws, tm_d, args);
}

cudaError_t launch_expert_gemm_mx4(const CUtensorMap& tm_w, const CUtensorMap& tm_x,
                                   const CUtensorMap& tm_ws, const CUtensorMap& tm_d,
                                   const Mx4GemmArgs& a, bool pair, int num_sms, cudaStream_t st) {
  return pair ? launch_mx4<true>(tm_w, tm_x, tm_ws, tm_d, a, num_sms, st)
              : launch_mx4<false>(tm_w, tm_x, tm_ws, tm_d, a, num_sms, st);
}

}  // namespace moe
