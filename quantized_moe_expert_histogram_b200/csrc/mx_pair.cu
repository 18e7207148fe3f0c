// Grouped product of MXFP4 rows and matrices, two SMs to a tile: the larger
// batches of mx_gemm.cu, where the one-SM kernel waits for L2.
//
// A thread-block cluster of two CTAs computes 256 rows x 256 outputs with
// instructions of both SMs' tensor cores: each CTA holds its 128 rows, half of
// the tile's weight rows and, in its tensor memory, its rows' accumulators.
// Per 256 K an SM loads 32 KB of codes for products that take 48 KB with one
// SM (measured there: 50 bytes a cycle and SM is what arrives, 1000 cycles a
// stage whose products take 512), and six stages fit instead of four.
//
// The even CTA leads: its warp 1 issues scale copies and products for both;
// the loads of both complete on the leader's barriers, the leader's commits
// arrive in both.  Otherwise the roles, the overlapping accumulators and the
// two sets of scale columns are those of mx_gemm.cu.  The scales of all 256
// weight rows go into both tensor memories, and all scales come as TMA boxes
// of scale tiles, so that they too complete on the leader's barrier: written
// by threads, as in mx_gemm.cu, each stage waited for a proxy fence and an
// arrival at cluster scope of about 650 cycles each.  The rows' scales are
// therefore put into tiles first (k_mx_tile_scales, 2 us), h's by the
// epilogue that forms them.  Nothing touches the other CTA after the cluster
// barrier that ends the kernel.
#include <atomic>
#include <type_traits>

#include "mx_gemm.cuh"

namespace moeq {
namespace {

using namespace ptx;

constexpr int kThreads = 384;
constexpr int kM = 256, kMc = 128;  // rows of a tile, of one CTA
constexpr int kNT = 256;
constexpr int kKS = 256;  // K of a stage
constexpr int kStages = 6;
constexpr int kSets = 2;  // sets of scale columns
constexpr int kA = kMc * 128, kB = kNT / 2 * 128, kSA = 1024, kSB = 2048;
constexpr int kOffB = kStages * kA;
constexpr int kOffSA = kOffB + kStages * kB;
constexpr int kOffSB = kOffSA + kStages * kSA;
constexpr int kOffOut = kOffSB + kStages * kSB;
constexpr int kOffTile = kOffOut + kEpiWarps * kStageOut;
constexpr int kOffBar = kOffTile + 3 * (kMxMaxExperts + 1) * 4 + 4;
constexpr int kBars = 2 * kStages + 4 + 1;  // (three tables of E + 1 ints before them)
constexpr int kOffMisc = kOffBar + kBars * 8;
constexpr int kSmem = kOffMisc + 16;
static_assert(kSmem <= 232448, "shared memory");
constexpr int kAcc1 = 208, kSF0 = kAcc1 + kNT, kSFCols = 24;
static_assert(kSF0 + kSets * kSFCols <= 512, "tensor memory");

struct Params {
  CUtensorMap a, a_all;  // codes of the rows: boxes of 32, of 128 rows
  CUtensorMap b;         // codes of the matrices, boxes of 128 rows
  CUtensorMap sa;        // scale tiles of the rows: 32-bit words [tiles][128], boxes of two
  CUtensorMap sb;        // of the matrices: [E][tiles][128]
  const int32_t* offsets;
  int rows, E, N, K;
  int row_tiles;  // scale tiles of the rows that the buffers hold
  void* out;
  uint8_t* out_scales;
  int32_t* status;
};

// First 128-row scale tile of each expert's rows, by one warp.
__device__ __forceinline__ void scan_row_tiles(const int* off, int E, int* row_tile, int lane) {
  const int per = (E + 31) / 32, b0 = lane * per;
  int run = 0;
  for (int i = 0; i < per; ++i)
    if (b0 + i < E) {
      row_tile[b0 + i] = run;
      run += (max(0, off[b0 + i + 1] - off[b0 + i]) + kMc - 1) / kMc;
    }
  int incl = run;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  for (int i = 0; i < per; ++i)
    if (b0 + i < E) row_tile[b0 + i] += incl - run;
  if (lane == 31) row_tile[E] = incl;
}

// Row scales [rows][K/32] into tiles, an expert's rows starting a new one: a
// CTA per row tile, a thread per row (rows past the expert's: zeros).
__global__ void __launch_bounds__(kMc) k_mx_tile_scales(const uint32_t* __restrict__ scales,
                                                        const int32_t* __restrict__ offsets, int rows, int E, int KT,
                                                        int tiles, uint32_t* __restrict__ out) {
  __shared__ int off[kMxMaxExperts + 1], row_tile[kMxMaxExperts + 1];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, r = tid;
  for (int b = tid; b <= E; b += kMc) off[b] = min(max(offsets[b], 0), rows);
  __syncthreads();
  if (tid < 32) scan_row_tiles(off, E, row_tile, tid);
  __syncthreads();
  const int tile = blockIdx.x;
  if (tile >= min(row_tile[E], tiles)) return;
  int lo = 0, hi = E;  // largest e with row_tile[e] <= tile
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (row_tile[mid] <= tile) lo = mid; else hi = mid;
  }
  const int row = off[lo] + (tile - row_tile[lo]) * kMc + r;
  const bool live = row < off[lo + 1];
  const uint32_t* src = scales + static_cast<size_t>(row) * KT;
  uint32_t* dst = out + static_cast<size_t>(tile) * KT * 128 + (r & 31) * 4 + (r >> 5);
#pragma unroll 4
  for (int k = blockIdx.y; k < KT; k += gridDim.y) dst[static_cast<size_t>(k) * 128] = live ? src[k] : 0u;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void arrive_at(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// Bounded wait by a whole warp for arrivals from either CTA.
__device__ __forceinline__ bool warp_wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                                  int32_t* status) {
  auto attempt = [&]() -> bool {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred P;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 P, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, P;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
  };
  bool ok = attempt();
  if (__all_sync(0xffffffffu, ok)) return true;
  uint64_t t0 = 0;
  for (uint32_t i = 1; !ok; ++i) {
    ok = attempt();
    if (!ok && (i & 7) == 0) {
      const uint64_t now = global_ns();  // (read only here: see mbar_wait)
      if (t0 == 0) t0 = now;
      if (*abort_flag) break;
      if (now - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        flag_status(status, MOE_DEV_TIMEOUT);
        break;
      }
    }
  }
  __syncwarp();
  return __all_sync(0xffffffffu, ok);
}

// Loads into this CTA's shared memory that complete on a barrier of either
// CTA of the pair.
__device__ __forceinline__ void pair_load_2d(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], "
      "[%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void pair_load_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2,
                                             uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], "
      "[%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void pair_copy_scales(uint32_t taddr, uint64_t sdesc) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
      "l"(sdesc)
      : "memory");
}
// Arrives at this address in both CTAs once the leader's copies and products
// so far are complete.
__device__ __forceinline__ void pair_commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(
          bar)
      : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

template <int OUT>
__global__ void __launch_bounds__(kThreads, 1) k_mx_pair(const __grid_constant__ Params P) {
  extern __shared__ __align__(1024) uint8_t smem[];
  int* tile_start = reinterpret_cast<int*>(smem + kOffTile);
  int* off_s = tile_start + (kMxMaxExperts + 1);
  int* row_tile = off_s + (kMxMaxExperts + 1);  // first scale tile of an expert's rows
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  const uint32_t bar0 = smem_u32(smem + kOffBar);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const uint32_t lead0 = cluster_map_shared(smem + kOffBar, 0);  // the leader's barriers
  auto full = [&](int i) { return bar0 + 8u * i; };         // leader: a stage of both CTAs is loaded
  auto lead_full = [&](int i) { return lead0 + 8u * i; };
  auto empty = [&](int i) { return bar0 + 8u * (kStages + i); };
  // the pair's tile i: its sums are complete; its columns that the next tile overwrites are read
  auto acc_full = [&](int i) { return bar0 + 8u * (2 * kStages + (i & 1)); };
  auto acc_free = [&](int i) { return bar0 + 8u * (2 * kStages + 2 + (i & 1)); };  // leader
  auto lead_free = [&](int i) { return lead0 + 8u * (2 * kStages + 2 + (i & 1)); };
  const uint32_t drain_bar = bar0 + 8u * (2 * kStages + 4);
  const int E = P.E, NB = (P.N + kNT - 1) / kNT;
  const int KB = (P.K + kKS - 1) / kKS;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full(i), 1);
      mbar_init(acc_free(i), 2 * kEpiWarps);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 3) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  pdl_trigger();
  build_tiles<kM>(P.offsets, E, P.rows, NB, P.status, tile_start, off_s);
  if (warp == 1) scan_row_tiles(off_s, E, row_tile, lane);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_publish();  // both CTAs' barriers exist
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const int tiles = __shfl_sync(0xffffffffu, tile_start[E], 0);
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;  // clusters

  if (warp == 0 || warp == 2) {
    // ---- weights (warp 0), rows (warp 2), with their scales ----------------------------
    int s = 0, ph = 0;
    bool ok = true;
    for (int t = first; t < tiles && ok; t += step) {
      const Tile T = decode_tile<kM, kNT>(t, tile_start, off_s, E, P.N);
      auto boxes_of = [&](int r) { return (min(max(T.nrows - r * kMc, 0), kMc) + kABox - 1) / kABox; };
      const int boxes = boxes_of(rank), row0 = T.row0 + static_cast<int>(rank) * kMc;
      const int rts = T.nn > 128 ? 2 : 1;
      const uint32_t bytes = (boxes_of(0) + boxes_of(1)) * (kABox * 128) + 2 * (kB + kSA + rts * 1024);
      for (int kb = 0; kb < KB; ++kb) {
        ok = warp_wait(empty(s), ph ^ 1, abort_flag, P.status);
        if (!ok) break;
        if (warp == 0) {
          if (rank == 0) elect_expect_tx(full(s), bytes);
          pair_load_3d(smem_u32(smem + kOffB + s * kB), &P.b, kb * 128, T.n0 + static_cast<int>(rank) * (T.nn / 2), T.e,
                       lead_full(s));
          for (int r = 0; r < rts; ++r)
            pair_load_3d(smem_u32(smem + kOffSB + s * kSB + r * 1024), &P.sb, 0,
                         ((T.n0 >> 7) + r) * (P.K / 128) + 2 * kb, T.e, lead_full(s));
        } else {
          pair_load_2d(smem_u32(smem + kOffSA + s * kSA), &P.sa, 0,
                       (row_tile[T.e] + T.at / kMc + static_cast<int>(rank)) * (P.K / 128) + 2 * kb, lead_full(s));
          const uint32_t adst = smem_u32(smem + s * kA);
          if (boxes == kMc / kABox) {
            pair_load_2d(adst, &P.a_all, kb * 128, row0, lead_full(s));
          } else {
            for (int i = 0; i < boxes; ++i)
              pair_load_2d(adst + i * (kABox * 128), &P.a, kb * 128, row0 + i * kABox, lead_full(s));
          }
        }
        if (++s == kStages) { s = 0; ph ^= 1; }
      }
    }
    if (!ok && rank == 0 && warp == 0) {  // both CTAs' copies in flight land before the cluster goes
      const uint64_t t0 = global_ns();
      for (int i = 0; i < kStages; ++i) {
        const int p = i < s ? ph : ph ^ 1;
        while (!mbar_try(full(i), p) && global_ns() - t0 < kWaitLimitNs) {}
      }
      __syncwarp();
    }
  } else if (warp == 1) {
    // ---- products, issued by the leader ----------------------------------------------
    if (rank == 0) {
      int s = 0, ph = 0, n = 0, tile = 0;
      bool ok = true;
      const uint64_t da0 = desc_sw128(smem_u32(smem)), db0 = desc_sw128(smem_u32(smem + kOffB));
      const uint64_t dsa0 = desc_plain(smem_u32(smem + kOffSA)), dsb0 = desc_plain(smem_u32(smem + kOffSB));
      for (int t = first; t < tiles && ok; t += step, ++tile) {
        const Tile T = decode_tile<kM, kNT>(t, tile_start, off_s, E, P.N);
        // M = 256 across the pair
        const uint32_t id0 = idesc_mxf4(T.nn, 0) + (8u << 24), id1 = idesc_mxf4(T.nn, 1) + (8u << 24);
        if (tile >= 1) {
          ok = warp_wait_cluster(acc_free(tile - 1), ((tile - 1) >> 1) & 1, abort_flag, P.status);
          if (!ok) break;
        }
        tc_fence_after();
        const uint32_t d = tmem + (tile & 1) * kAcc1;
        // (a stage's copies and products in one straight line, as in mx_gemm.cu)
        auto stage = [&](auto two, uint32_t later) {
          if (!warp_wait_cluster(full(s), ph, abort_flag, P.status)) return false;
          // the products of kSets stages ago, which read this set of scale columns
          if (n >= kSets && !warp_wait(empty((n - kSets) % kStages), ((n - kSets) / kStages) & 1, abort_flag, P.status))
            return false;
          tc_fence_after();
          const uint32_t sfa = tmem + kSF0 + (n % kSets) * kSFCols, sfb = sfa + 8;
          const uint64_t da = da0 + s * (kA >> 4), db = db0 + s * (kB >> 4);
          const uint64_t dsa = dsa0 + s * (kSA >> 4), dsb = dsb0 + s * (kSB >> 4);
          // (a tile of 128 of 256 outputs: the second tile of scales is stale and unused)
          pair_copy_scales(sfa, dsa);
          pair_copy_scales(sfb, dsb);
          pair_copy_scales(sfb + 4, dsb + 64);
          if constexpr (two.value) {
            pair_copy_scales(sfa + 4, dsa + 32);
            pair_copy_scales(sfb + 8, dsb + 32);
            pair_copy_scales(sfb + 12, dsb + 96);
          }
          pair_mma(d, da, db, id0, sfa, sfb, later);
          pair_mma(d, da + 2, db + 2, id1, sfa, sfb, 1u);
          if constexpr (two.value) {
            pair_mma(d, da + 4, db + 4, id0, sfa + 4, sfb + 8, 1u);
            pair_mma(d, da + 6, db + 6, id1, sfa + 4, sfb + 8, 1u);
          }
          pair_commit(empty(s));
          if (++s == kStages) { s = 0; ph ^= 1; }
          ++n;
          return true;
        };
        for (int kb = 0; kb < P.K / kKS && ok; ++kb) ok = stage(std::true_type{}, kb != 0);
        if (ok && P.K % kKS) ok = stage(std::false_type{}, P.K > kKS);
        if (!ok) break;
        pair_commit(acc_full(tile));
      }
      // every product completes before the cluster goes
      pair_commit(drain_bar);
      const uint64_t t0 = global_ns();
      while (!mbar_try(drain_bar, 0) && global_ns() - t0 < kWaitLimitNs) {}
      __syncwarp();
    }
  } else if (warp >= 4) {
    // ---- epilogue: lane = row of the CTA's half, quadrant = warp % 4; the quadrant's
    // two warps take the even and the odd groups of 64 columns ------------------------
    const int q = warp & 3, half = (warp - 4) >> 2;
    uint8_t* st = smem + kOffOut + (warp - 4) * kStageOut;
    int tile = 0;
    bool ok = true;
    for (int t = first; t < tiles && ok; t += step, ++tile) {
      const Tile T = decode_tile<kM, kNT>(t, tile_start, off_s, E, P.N);
      ok = warp_wait(acc_full(tile), (tile >> 1) & 1, abort_flag, P.status);
      if (!ok) break;
      tc_fence_after();
      const uint32_t tb = tmem + (static_cast<uint32_t>(32 * q) << 16) + (tile & 1) * kAcc1;
      const int r0 = static_cast<int>(rank) * kMc + 32 * q, live = T.nrows - r0;
      bool bad = false;
      // the group in the shared columns (the last of the first accumulator, the
      // first of the second) is taken first by the warp that has it, which then
      // frees the columns; the other frees them at once
      const bool last_first = (tile & 1) == 0;
      auto freed = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_at(lead_free(tile));
      };
      if (half != (last_first ? 1 : 0)) freed();
#pragma unroll 1
      for (int i = half; i < 4; i += 2) {
        const int grp = last_first && half == 1 ? 4 - i : i;
        if (grp < T.nn / 64 && live > 0)
          bad |= store_group<OUT>(
              P.out,
              [&](int blk) {
                return P.out_scales +
                       // (a table whose experts overlap has more tiles than the rows)
                       (static_cast<size_t>(min(row_tile[T.e] + T.at / kMc + static_cast<int>(rank), P.row_tiles - 1)) *
                            (P.N / 256) +
                        blk / 4) *
                           512 +
                       lane * 16 + q * 4 + (blk & 3);
              },
              tb + grp * 64, st, lane, T.row0 + r0, live, T.n0 + grp * 64, P.N);
        if (i == half && half == (last_first ? 1 : 0)) freed();
      }
      if (bad) flag_status(P.status, MOE_DEV_RANGE);
    }
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync_publish();  // every role of both CTAs is done
  if (warp == 3) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

template <int OUT>
moe_status_t launch(const MxGemmArgs& a, cudaStream_t s) {
  Params P{};
  const cuuint64_t half_k = static_cast<cuuint64_t>(a.K / 2);
  const cuuint64_t da[2] = {half_k, static_cast<cuuint64_t>(a.rows)}, sa[1] = {half_k};
  const cuuint32_t ba[2] = {128, kABox}, ba_all[2] = {128, kMc};
  const cuuint64_t db[3] = {half_k, static_cast<cuuint64_t>(a.N), static_cast<cuuint64_t>(a.E)};
  const cuuint64_t sb[2] = {half_k, static_cast<cuuint64_t>(a.mat_stride)};
  const cuuint32_t bb[3] = {128, kNT / 2, 1};
  const cuuint64_t ds[3] = {128, static_cast<cuuint64_t>(a.N / 128) * (a.K / 128), static_cast<cuuint64_t>(a.E)};
  const cuuint64_t ss[2] = {512, static_cast<cuuint64_t>(a.mat_stride)};
  const cuuint32_t bs[3] = {128, 2, 1}, es[3] = {1, 1, 1};
  const cuuint64_t dt[2] = {128, static_cast<cuuint64_t>(mx_row_tiles(a.rows, a.E)) * (a.K / 128)}, stt[1] = {512};
  auto fn = get_encode();
  auto words = [&](CUtensorMap* m, int rank, const uint8_t* base, const cuuint64_t* dims, const cuuint64_t* strides) {
    return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, rank, const_cast<uint8_t*>(base), dims, strides, bs, es,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (!encode_bytes(&P.a, 2, a.a_codes, da, sa, ba) || !encode_bytes(&P.a_all, 2, a.a_codes, da, sa, ba_all) ||
      !encode_bytes(&P.b, 3, a.mats, db, sb, bb) ||
      !words(&P.sa, 2, a.a_tiles, dt, stt) || !words(&P.sb, 3, a.mats + static_cast<size_t>(a.N) * (a.K / 2), ds, ss)) {
    set_error("tensor map (MXFP4 codes) could not be encoded");
    return MOE_ERR_CUDA;
  }
  P.offsets = a.offsets;
  P.rows = a.rows;
  P.row_tiles = static_cast<int>(mx_row_tiles(a.rows, a.E));
  P.E = a.E;
  P.N = a.N;
  P.K = a.K;
  P.out = a.out;
  P.out_scales = a.out_scales;
  P.status = a.status;
  static std::atomic<uint64_t> attr_set{0};  // per device, as in mx_gemm.cu
  static std::atomic<int> sms[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_check(e, "MXFP4 product: cudaGetDevice");
  if (dev < 0 || dev >= 64) {
    set_error("MXFP4 product: device %d beyond the supported 64", dev);
    return MOE_ERR_UNSUPPORTED_SHAPE;
  }
  auto kern = k_mx_pair<OUT>;
  if (!(attr_set.load() & (1ull << dev))) {
    int n = 0;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_check(e, "MXFP4 product: shared-memory attribute");
    sms[dev].store(n);
    attr_set.fetch_or(1ull << dev);
  }
  const long most = (static_cast<long>(a.rows) / kM + std::min(a.E, a.rows)) * ceil_div(a.N, kNT);
  const int clusters = static_cast<int>(std::min<long>(most, sms[dev].load() / 2));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * clusters);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_for(a.rows) ? 2 : 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, kern, P), "MXFP4 product launch");
}

}  // namespace

moe_status_t launch_mx_tile_scales(const uint8_t* scales, const int32_t* offsets, int rows, int E, int K,
                                   uint8_t* tiles, cudaStream_t s) {
  const int n = static_cast<int>(mx_row_tiles(rows, E)), kt = K / 128;
  return cuda_check(launch_pdl(pdl_for(rows), k_mx_tile_scales, dim3(n, ceil_div(kt, 16)), dim3(kMc), 0, s,
                               reinterpret_cast<const uint32_t*>(scales), offsets, rows, E, kt, n,
                               reinterpret_cast<uint32_t*>(tiles)),
                    "MXFP4 product: scale tiles launch");
}

moe_status_t launch_mx_pair(const MxGemmArgs& a, cudaStream_t s) {
  switch (a.out_kind) {
    case kMxOutF16: return launch<kMxOutF16>(a, s);
    case kMxOutBf16: return launch<kMxOutBf16>(a, s);
    case kMxOutF32: return launch<kMxOutF32>(a, s);
    default: return launch<kMxOutSwiglu>(a, s);
  }
}

}  // namespace moeq
