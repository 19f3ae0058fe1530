// Gradient of the experts' grouped product to the weights:
//   dW[e] = sum over the rows r of expert e's segment of x[r]^T g[r],
// a product of [K x n_e] by [n_e x N] per expert whose contraction runs over a
// ragged segment of rows.
//
// Both operands lie with the contraction as their outer dimension, so both are
// MN-major UMMA operands: a TMA box of 64 rows x 2 blocks of 64 columns (16 KB)
// is a CTA's share of one operand in a stage, as memory has it. A CTA pair
// computes 256 x 256 of dW[e] (cta_group::2, M = 256, N = 256): each CTA holds
// 128 columns of x and 128 of g, and its own 128 rows of the result.
//
// A segment starts at any row and its length is no multiple of anything, while
// a box always has 64 rows: those behind the segment belong to the next expert
// or to nothing, and may hold infinities or NaN. Only ceil(n / 16) of a stage's
// four K steps are issued, and where the last one has rows of both kinds the
// stage takes a longer way: its loads count on barriers of their own CTA, a
// warp waits for them, writes zeros over the rows behind the segment in both
// operands, and hands the stage to the issuer.
//
// Roles per CTA (352 threads): warp 0 TMA producer; warp 1 UMMA issuer (leader)
// and TMEM allocation; warp 2 the zeros behind a segment; warps 3-10 the
// epilogue, each 32 rows x 128 columns of the CTA's 128 x 256: TMEM is added to
// registers piece by piece, and a finished tile goes through 4 KB of swizzled
// shared memory a warp and out by TMA (which cuts the tile at K and N, and with
// `accumulate` adds in the fp32 gradient's place).
//
// 65536 rows over 8 experts of 4096 x 14336, fp32: 4.25 to 4.7 ms, 1.7 to 1.8 PFLOP/s
// at the power limit (tensor pipe 93 % of the clocks); 65535 over 128 of 4096 x 2048,
// bf16: 742 us (67 %). What bounds it is the way into shared memory: a stage is 32 KB
// for 512 clocks of UMMAs, and all SMs together take in about 14 TB/s from L2 (47 to
// 55 bytes a clock each), whichever the product.
//
// Tiles of one expert cost as many stages as its segment has; experts are taken
// from the longest segment down, so that the round-robin over pairs ends with
// the cheapest tiles.
#include "moe_internal.h"
#include "moe_ptx.cuh"

namespace moe {

namespace {

constexpr int kTile = 256;          // rows and columns of dW per pair
constexpr int kDepth = 64;          // rows of x and g per stage
constexpr int kStages = 6;
constexpr int kEpiWarps = 8;
constexpr int kFirstEpi = 3;
constexpr int kThreads = 32 * (kFirstEpi + kEpiWarps);
constexpr uint32_t kOpBytes = kDepth * 128 * 2;      // 16 KB: 64 rows x 128 columns
constexpr uint32_t kBlockBytes = kDepth * 128;       // 8 KB: one block of 64 columns
constexpr uint32_t kStageBytes = 2 * kOpBytes;
constexpr uint32_t kOutBytes = 32 * 128;             // one warp's 32 rows x 128 bytes
constexpr uint32_t kTmemCols = 2 * kTile;
constexpr int kGroup = 8;           // m-tiles per raster group
// Stages summed in TMEM before the sum moves to registers. The tensor core's
// fp32 additions cut towards zero, a bias of about 2^-25 of the sum each, which
// adds up over a long segment: 9e-6 of the result after 8192 rows. The epilogue
// adds the pieces with rounding.
constexpr int kPiece = 8;
// Segments of this many rows on average are split over pairs where their tiles are
// too few for all: over four where there is one tile for eight pairs, over two where
// there is one for two (clusters of eight CTAs do not pack as well: 16 tiles of 2048
// rows took 22.7 us in them, two rounds). Unsplit and split: 1 tile of 1024 rows
// 10.9, 11.8 us, of 2048 15.1, 12.8, of 8192 40.8, 19.5; 30 tiles of 8192 rows 42.4,
// 30.5; 16 of 32768 (a router's gradient, 4096 x 64) 138, 75.
constexpr int kSplitRows = 2048;

struct WgTile {
  int lo, len, m0, n0, e;
  int empty;  // the whole segment is
};

__device__ __forceinline__ WgTile decode_wg(int L, const int* offs, const uint8_t* order, int mt,
                                            int nt) {
  const int per_e = mt * nt;
  WgTile t;
  t.e = order[L / per_e];
  t.lo = offs[t.e];
  t.len = offs[t.e + 1] - t.lo;
  t.empty = t.len == 0;
  const int r = L % per_e;
  const int g = r / (kGroup * nt);
  const int gsz = min(kGroup, mt - g * kGroup);
  const int q = r - g * kGroup * nt;
  t.m0 = (g * kGroup + q % gsz) * kTile;
  t.n0 = q / gsz * kTile;
  return t;
}

// A warp's walk over its pair's tiles. Each lane decodes one of the next 32 (the
// divisions would otherwise stand between every two tiles of the issuer); called
// by the whole warp.
struct TileWalk {
  const int* offs;
  const uint8_t* order;
  int mt, nt, total, stride, L, at;
  int part, parts;  // which of how many pieces of a segment's stages
  WgTile mine;

  __device__ __forceinline__ TileWalk(const int* offs_, const uint8_t* order_, int mt_, int nt_,
                                      int total_, int first, int stride_, int part_, int parts_)
      : offs(offs_), order(order_), mt(mt_), nt(nt_), total(total_), stride(stride_), L(first), at(32),
        part(part_), parts(parts_) {}

  __device__ __forceinline__ bool next(WgTile& t) {
    if (L >= total) return false;
    if (at == 32) {
      const int l = min(L + static_cast<int>(threadIdx.x & 31) * stride, total - 1);
      mine = decode_wg(l, offs, order, mt, nt);
      if (parts > 1) {
        const int nk = (mine.len + kDepth - 1) / kDepth;
        const int first = static_cast<int>(static_cast<int64_t>(nk) * part / parts) * kDepth;
        const int last = static_cast<int>(static_cast<int64_t>(nk) * (part + 1) / parts) * kDepth;
        mine.lo += first;
        mine.len = min(mine.len, last) - first;
      }
      at = 0;
    }
    t.lo = __shfl_sync(0xffffffffu, mine.lo, at);
    t.len = __shfl_sync(0xffffffffu, mine.len, at);
    t.m0 = __shfl_sync(0xffffffffu, mine.m0, at);
    t.n0 = __shfl_sync(0xffffffffu, mine.n0, at);
    t.e = __shfl_sync(0xffffffffu, mine.e, at);
    t.empty = __shfl_sync(0xffffffffu, mine.empty, at);
    ++at;
    L += stride;
    return true;
  }
};

// Whether stage kb of a segment of len rows has a K step with rows behind it.
__device__ __forceinline__ bool is_tail(int len, int kb) {
  const int left = len - kb * kDepth;
  return left < kDepth && (left & 15) != 0;
}

// Issues a stage's K steps of 16 rows and releases it. One 128-byte row per k: a
// step is 2 KB on in both operands (128 in a descriptor); the blocks of 64
// columns are 8 KB apart, g's behind x's. Called by the whole warp, straight on
// for a full stage, so that an elected lane keeps the tensor core's queue filled
// (a lane that issued alone in a diverged warp, its descriptors built on the way,
// took 185 clocks per UMMA of 128: 852 us instead of 788 for 128 experts).
__device__ __forceinline__ void issue_stage(uint32_t d_tmem, uint64_t xd, uint32_t idesc, bool add,
                                            int steps, uint64_t* release, uint64_t* done,
                                            uint16_t pair_mask) {
  constexpr uint64_t kG = kOpBytes >> 4;
  if (elect_one()) {
    umma_bf16_pair(d_tmem, xd, xd + kG, idesc, add ? 1u : 0u);
    if (steps == kDepth / 16) {
#pragma unroll
      for (uint32_t k = 1; k < kDepth / 16; ++k)
        umma_bf16_pair(d_tmem, xd + 128u * k, xd + kG + 128u * k, idesc, 1u);
    } else {
      for (uint32_t k = 1; k < static_cast<uint32_t>(steps); ++k)
        umma_bf16_pair(d_tmem, xd + 128u * k, xd + kG + 128u * k, idesc, 1u);
    }
    umma_commit_pair_multicast(release, pair_mask);
    if (done != nullptr) umma_commit_pair_multicast(done, pair_mask);
  }
  __syncwarp();
}

// kSplit: a cluster of kSplit pairs works on one tile, each on a part of the
// segment's stages. The parts' sums then lie in shared memory (the ring's, by then
// idle) as [column / 4][row] of four, and each pair adds up, in the pairs' order,
// the columns that it stores. One tile to a cluster at most.
template <int kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    wgrad_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_g,
                 const __grid_constant__ CUtensorMap tm_d, WgradArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_up_1024(smem_raw);
  uint8_t* out_buf = smem + kStages * kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(out_buf + kEpiWarps * kOutBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tail_ld = empty + kStages;  // own CTA's loads of a stage with a cut K step
  uint64_t* tail_ok = tail_ld + kStages;  // leader: such a stage has its zeros in both CTAs
  uint64_t* tfull = tail_ok + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint64_t* xbar = drain + 1;  // leader: the peer's count of loaded stages has arrived
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(xbar + 1);
  uint32_t* abort_flag = tmem_slot + 1;
  uint32_t* peer_issued = abort_flag + 1;
  volatile uint32_t* loaded = peer_issued + 1;  // stages this CTA's producer has issued
  int* offs = reinterpret_cast<int*>(peer_issued + 2);        // [E+1]
  uint8_t* order = reinterpret_cast<uint8_t*>(offs + p.E + 1);  // [E] longest segment first

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int E = p.E;
  const uint32_t cta = cluster_ctarank();
  const uint32_t rank = cta & 1u, lead = cta & ~1u;  // in the pair; the pair's leader
  const bool leader = rank == 0;
  const uint16_t pair_mask = static_cast<uint16_t>(3u << lead);
  const int part = static_cast<int>(cta >> 1);
  const int cluster = blockIdx.x / (2 * kSplit), n_clusters = gridDim.x / (2 * kSplit);

  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  if (warp == 2 && lane == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&tail_ld[s], 1);
      mbar_init(&tail_ok[s], 2);  // a warp of each CTA
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * kEpiWarps * 32);
    }
    mbar_init(drain, 1);
    mbar_init(xbar, 1);
    *abort_flag = 0u;
    *loaded = 0u;
    fence_barrier_init();
  }
  if (warp == kFirstEpi && lane == 0) {
    tma_prefetch_desc(&tm_x);
    tma_prefetch_desc(&tm_g);
    tma_prefetch_desc(&tm_d);
  }
  grid_dependency_wait();
  grid_launch_dependents();
  for (int i = tid; i <= E; i += kThreads) {
    const int v = p.offsets[i];
    offs[i] = v < 0 ? 0 : (v > p.rows ? p.rows : v);
  }
  __syncthreads();
  if (tid == 0)
    for (int i = 1; i <= E; ++i) offs[i] = offs[i] < offs[i - 1] ? offs[i - 1] : offs[i];
  __syncthreads();
  for (int e = tid; e < E; e += kThreads) {
    const int n = offs[e + 1] - offs[e];
    int before = 0;
    for (int i = 0; i < E; ++i) {
      const int m = offs[i + 1] - offs[i];
      before += m > n || (m == n && i < e);
    }
    order[before] = static_cast<uint8_t>(e);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // barrier initialisation visible to the peer before any remote use
  tc_fence_after();

  const uint32_t tmem_base = *tmem_slot;
  const int mt = (p.K + kTile - 1) / kTile, nt = (p.N + kTile - 1) / kTile;
  const int total = E * mt * nt;
  const WaitCtl wc{abort_flag, p.dev_status, p.timeout_ns};
  const uint32_t peer_abort = mapa_shared(smem_u32(abort_flag), cta ^ 1u);
  auto pair_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (mbar_wait(bar, parity, wc)) return true;
    st_u32_cluster(peer_abort, 1u);
    return false;
  };

  TileWalk tiles(offs, order, mt, nt, total, cluster, n_clusters, part, kSplit);
  WgTile c;
  if (warp == 0) {
    {
      // ------------------------------------------------------ TMA producer ----
      int stage = 0;
      uint32_t phase = 0;
      // per stage, as bits: parity of the next use of full and of tail_ld, and
      // whether the last use was a tail
      uint32_t full_par = 0, tail_par = 0, was_tail = 0;
      int issued = 0;
      bool aborted = false;
      while (!aborted && tiles.next(c)) {
        const int nk = (c.len + kDepth - 1) / kDepth;
        const bool half_n = p.N - c.n0 <= kTile / 2;
        const int xb = (c.m0 + static_cast<int>(rank) * (kTile / 2)) / 64;
        const int gb = (c.n0 + static_cast<int>(rank) * (half_n ? kTile / 4 : kTile / 2)) / 64;
        for (int kb = 0; kb < nk; ++kb) {
          if (!__all_sync(0xffffffffu, pair_wait(&empty[stage], phase ^ 1u))) {
            aborted = true;
            break;
          }
          const uint32_t bit = 1u << stage;
          const bool tail = is_tail(c.len, kb);
          if (tail) {
            tail_par ^= bit;
            was_tail |= bit;
          } else {
            full_par ^= bit;
            was_tail &= ~bit;
          }
          if (elect_one()) {
            uint32_t bar;
            if (tail) {
              mbar_arrive_expect_tx(&tail_ld[stage], kStageBytes);
              bar = mapa_shared(smem_u32(&tail_ld[stage]), cta);
            } else {
              if (leader) mbar_arrive_expect_tx(&full[stage], 2 * kStageBytes);
              bar = mapa_shared(smem_u32(&full[stage]), lead);
            }
            uint8_t* sx = smem + stage * kStageBytes;
            const int row = c.lo + kb * kDepth;
            tma_load_3d_pair(sx, &tm_x, bar, 0, row, xb);
            tma_load_3d_pair(sx + kOpBytes, &tm_g, bar, 0, row, gb);
            *loaded = static_cast<uint32_t>(issued + 1);
          }
          __syncwarp();
          ++issued;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // No CTA exits before its loads have landed (the kernel ends with a
      // cluster barrier). Loads of a tail count on their own CTA's barrier; the
      // others of both CTAs on the leader's. After an abort the two may have
      // stopped at different stages: the peer reports how many it loaded, and
      // the leader makes the accounting of each stage in flight whole before it
      // waits. (Both walk the same tiles, so stage i is of one kind in both;
      // where the leader never reached it, waiting for a tail as for another
      // stage only runs into the limit.)
      if (lane != 0) {
        // lane 0 does the rest
      } else if (!leader) {
        st_async_u32_cluster(mapa_shared(smem_u32(peer_issued), lead), static_cast<uint32_t>(issued),
                             mapa_shared(smem_u32(xbar), lead));
        for (int i = max(0, issued - kStages); i < issued; ++i) {
          const int s = i % kStages;
          if (was_tail >> s & 1u) mbar_wait_drain(&tail_ld[s], (tail_par >> s & 1u) ^ 1u, kDrainLimitNs);
        }
      } else {
        mbar_arrive_expect_tx(xbar, 4);
        int theirs = issued;
        if (mbar_wait_drain(xbar, 0, p.timeout_ns + kDrainLimitNs)) {
          theirs = min(static_cast<int>(*reinterpret_cast<volatile uint32_t*>(peer_issued)),
                       issued + kStages);
        } else {
          atomicOr(p.dev_status, MOE_DEV_TIMEOUT);
        }
        const int hi = max(issued, theirs);
        for (int i = max(0, hi - kStages); i < hi; ++i) {
          const int s = i % kStages;
          if (i >= issued) {
            mbar_arrive_expect_tx(&full[s], kStageBytes);  // the peer's half alone
            mbar_wait_drain(&full[s], full_par >> s & 1u, kDrainLimitNs);
          } else if (was_tail >> s & 1u) {
            mbar_wait_drain(&tail_ld[s], (tail_par >> s & 1u) ^ 1u, kDrainLimitNs);
          } else {
            if (i >= theirs) mbar_complete_tx(&full[s], kStageBytes);  // will never come
            mbar_wait_drain(&full[s], (full_par >> s & 1u) ^ 1u, kDrainLimitNs);
          }
        }
      }
    }
  } else if (warp == 1) {
    if (leader) {
      // ------------------------------------------- UMMA issuer (leader) ----
      // the whole warp walks, an elected lane issues
      int stage = 0;
      uint32_t full_par = 0, tail_par = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool aborted = false;
      const uint64_t desc0 = smem_desc_sw128(smem_u32(smem), kBlockBytes, 1024u);
      while (!aborted && tiles.next(c)) {
        const uint32_t idesc = idesc_bf16_f32(kTile, p.N - c.n0 <= kTile / 2 ? kTile / 2 : kTile,
                                              true, true);
        const int nk = (c.len + kDepth - 1) / kDepth;
        for (int kb = 0; kb < nk; ++kb) {
          const int in_piece = kb % kPiece;
          bool ok = true;
          if (in_piece == 0) ok = pair_wait(&tempty[acc], acc_phase ^ 1u);
          if (ok) {
            if (is_tail(c.len, kb)) {
              ok = mbar_wait<true>(&tail_ok[stage], tail_par >> stage & 1u, wc);
              if (!ok) st_u32_cluster(peer_abort, 1u);
              tail_par ^= 1u << stage;
            } else {
              ok = pair_wait(&full[stage], full_par >> stage & 1u);
              full_par ^= 1u << stage;
            }
          }
          if (!__all_sync(0xffffffffu, ok)) {
            aborted = true;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kTile);
          const uint64_t xd = desc0 + ((stage * kStageBytes) >> 4);
          const int steps = min(kDepth / 16, (c.len - kb * kDepth + 15) / 16);
          const bool piece_end = in_piece == kPiece - 1 || kb == nk - 1;
          issue_stage(d_tmem, xd, idesc, in_piece != 0, steps, &empty[stage],
                      piece_end ? &tfull[acc] : nullptr, pair_mask);
          if (++stage == kStages) stage = 0;
          if (piece_end && ++acc == 2) {
            acc = 0;
            acc_phase ^= 1u;
          }
        }
      }
      // every UMMA issued must finish before TMEM is released
      if (elect_one()) umma_commit_pair(drain);
      __syncwarp();
      mbar_wait_drain(drain, 0, kDrainLimitNs);
    }
  } else if (warp < kFirstEpi) {
    // ------------------------------------- zeros behind a segment's end ----
    // whole 128-byte rows, which the swizzle keeps together, in the four
    // 64-column blocks (two of each operand) of each tail stage. Between two tails
    // there may be whole segments without one, most of the kernel's time, so the limit
    // of this wait counts from the producer's last stage.
    int stage = 0;
    uint32_t tail_par = 0;
    bool aborted = false;
    while (!aborted && tiles.next(c)) {
      const int nk = (c.len + kDepth - 1) / kDepth;
      if (nk == 0) continue;
      const int s = (stage + nk - 1) % kStages;
      stage = (stage + nk) % kStages;
      if (!is_tail(c.len, nk - 1)) continue;
      const bool ok = mbar_wait_progress(&tail_ld[s], tail_par >> s & 1u, wc, loaded);
      if (!ok) st_u32_cluster(peer_abort, 1u);
      if (!__all_sync(0xffffffffu, ok)) {
        aborted = true;
        break;
      }
      tail_par ^= 1u << s;
      const int left = c.len - (nk - 1) * kDepth;
      const int words = (((left + 15) & ~15) - left) * 8;  // 16-byte words per block
      const uint32_t at = smem_u32(smem) + s * kStageBytes + 128u * left;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        for (int i = lane; i < words; i += 32)
          st_shared_v4(at + b * kBlockBytes + 16u * i, make_uint4(0, 0, 0, 0));
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive_release_shared(mapa_shared(smem_u32(&tail_ok[s]), lead));
    }
  } else {
    // ------------------------------------------------------ epilogue ----
    const int q = warp & 3;
    const int half = (warp - kFirstEpi) >> 2;
    const uint32_t buf = smem_u32(out_buf) + static_cast<uint32_t>(warp - kFirstEpi) * kOutBytes;
    // this lane's row of the buffer: 128 bytes in eight 16-byte words, word w at
    // w ^ (row & 7) as the 128-byte swizzle of the store has it
    const uint32_t my = buf + 128u * lane;
    const uint32_t tempty_leader[2] = {mapa_shared(smem_u32(&tempty[0]), lead),
                                       mapa_shared(smem_u32(&tempty[1]), lead)};
    int acc = 0;
    uint32_t acc_phase = 0;
    bool aborted = false;
    while (!aborted && tiles.next(c)) {
      if (c.empty && p.accumulate) continue;
      const int row = c.m0 + static_cast<int>(rank) * (kTile / 2) + 32 * q;
      const int col0 = c.n0 + half * (kTile / 2);
      // whole 32-column chunks: N and K are multiples of 64
      const int n_chunks = col0 >= p.N || row >= p.K ? 0 : min(4, (p.N - col0) / 32);
      float sum[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) sum[i] = 0.f;
      for (int left = c.len; left > 0; left -= kPiece * kDepth) {
        if (!__all_sync(0xffffffffu, pair_wait(&tfull[acc], acc_phase))) {
          aborted = true;
          break;
        }
        tc_fence_after();
        const uint32_t t_base = tmem_base + (static_cast<uint32_t>(32 * q) << 16) +
                                static_cast<uint32_t>(acc * kTile + half * (kTile / 2));
#pragma unroll
        for (int cc = 0; cc < 8; ++cc) {
          if (cc < 2 * n_chunks) {
            uint32_t r[16];
            tmem_ld_32x32b_x16(t_base + 16u * cc, r);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[16 * cc + i] += __uint_as_float(r[i]);
          }
        }
        tc_fence_before();
        mbar_arrive_cluster(tempty_leader[acc]);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (aborted) break;
      if constexpr (kSplit > 1) {
        const uint32_t at = smem_u32(smem) + 16u * (128 * 32 * half + 32 * q + lane);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          st_shared_v4(at + 16u * 128 * i,
                       make_uint4(__float_as_uint(sum[4 * i]), __float_as_uint(sum[4 * i + 1]),
                                  __float_as_uint(sum[4 * i + 2]), __float_as_uint(sum[4 * i + 3])));
        continue;
      }
#pragma unroll
      for (int cc = 0; cc < 4; ++cc) {
        if (cc < n_chunks) {
          const int col = col0 + 32 * cc;
          if (p.bf16_out) {
            // two chunks share a buffer of 64 columns
            if ((cc & 1) == 0) {
              if (lane == 0) tma_store_wait_read();
              __syncwarp();
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float* v = sum + 32 * cc + 8 * i;
              st_shared_v4(my + 16u * ((4 * (cc & 1) + i) ^ (lane & 7)),
                           make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                      pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
            }
            if ((cc & 1) == 1) {
              fence_proxy_async();
              __syncwarp();
              if (lane == 0) tma_store_3d(&tm_d, buf, col - 32, row, c.e);
            }
          } else {
            if (lane == 0) tma_store_wait_read();
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float* v = sum + 32 * cc + 4 * i;
              st_shared_v4(my + 16u * (i ^ (lane & 7)),
                           make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]),
                                      __float_as_uint(v[2]), __float_as_uint(v[3])));
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
              if (p.accumulate) tma_reduce_add_3d(&tm_d, buf, col, row, c.e);
              else tma_store_3d(&tm_d, buf, col, row, c.e);
            }
          }
        }
      }
    }
    if (lane == 0) tma_store_wait();
  }

  if constexpr (kSplit > 1) {
    __syncwarp();
    cluster_sync();  // every pair's sums are in place
    TileWalk again(offs, order, mt, nt, total, cluster, n_clusters, part, kSplit);
    if (warp >= kFirstEpi && again.next(c) && !(c.empty && p.accumulate)) {
      constexpr int kCols = kTile / kSplit / 2;  // of each warp
      const int local = 32 * (warp & 3) + lane;
      const int row = c.m0 + static_cast<int>(rank) * (kTile / 2) + local;
      const int first = part * (kTile / kSplit) + ((warp - kFirstEpi) >> 2) * kCols;
#pragma unroll 1
      for (int cc = 0; cc < kCols && c.n0 + first + cc < p.N && row < p.K; cc += 32) {
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0.f;
        for (uint32_t pair = 0; pair < kSplit; ++pair) {
          const uint32_t at = mapa_shared(
              smem_u32(smem) + 16u * (128 * ((first + cc) / 4) + local), 2 * pair + rank);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 f = ld_shared_cluster_v4(at + 16u * 128 * i);
            v[4 * i] += f.x;
            v[4 * i + 1] += f.y;
            v[4 * i + 2] += f.z;
            v[4 * i + 3] += f.w;
          }
        }
        const size_t at = (static_cast<size_t>(c.e) * p.K + row) * p.N + c.n0 + first + cc;
        if (p.bf16_out) {
          uint4* d = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.dW) + at);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            d[i] = make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                              pack_bf16x2(v[8 * i + 4], v[8 * i + 5]),
                              pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
        } else {
          float4* d = reinterpret_cast<float4*>(static_cast<float*>(p.dW) + at);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float4 f = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            if (p.accumulate) {
              const float4 o = d[i];
              f = make_float4(f.x + o.x, f.y + o.y, f.z + o.z, f.w + o.w);
            }
            d[i] = f;
          }
        }
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the peer may still signal it
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, kTmemCols);
}

size_t wgrad_smem_bytes(int E) {
  return 1024 + kStages * kStageBytes + kEpiWarps * kOutBytes + 8 * (4 * kStages + 6) + 16 +
         4 * static_cast<size_t>(E + 1) + static_cast<size_t>(E);
}

}  // namespace

namespace {

template <int kSplit>
cudaError_t launch_split(const CUtensorMap& tm_x, const CUtensorMap& tm_g, const CUtensorMap& tm_d,
                         const WgradArgs& a, int num_sms, cudaStream_t st) {
  const size_t smem = wgrad_smem_bytes(a.E);
  // for every expert count: calls on other threads do not lower it before the launch
  cudaError_t err = cudaFuncSetAttribute(wgrad_kernel<kSplit>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(wgrad_smem_bytes(kMaxExperts)));
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  constexpr int kCluster = 2 * kSplit;
  cfg.gridDim = dim3(static_cast<unsigned>(num_sms / kCluster * kCluster), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  err = cudaLaunchKernelEx(&cfg, wgrad_kernel<kSplit>, tm_x, tm_g, tm_d, a);
  return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace

cudaError_t launch_wgrad(const CUtensorMap& tm_x, const CUtensorMap& tm_g, const CUtensorMap& tm_d,
                         const WgradArgs& a, int num_sms, cudaStream_t st) {
  const int64_t tiles = static_cast<int64_t>(a.E) * ((a.K + kTile - 1) / kTile) * ((a.N + kTile - 1) / kTile);
  const int64_t rows = a.rows / a.E;
  if (rows >= kSplitRows && tiles <= num_sms / 16) return launch_split<4>(tm_x, tm_g, tm_d, a, num_sms, st);
  if (rows >= kSplitRows && tiles <= num_sms / 4) return launch_split<2>(tm_x, tm_g, tm_d, a, num_sms, st);
  return launch_split<1>(tm_x, tm_g, tm_d, a, num_sms, st);
}

}  // namespace moe
