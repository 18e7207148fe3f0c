// Grouped product of MXFP4 rows and MXFP4 expert matrices on the block-scaled
// tensor-core instruction, y[p] = W_e xq[p] for the rows p of each expert e,
// and the expert SwiGLU FFN built from two of them.
//
// An instruction multiplies e2m1 codes and applies both operands' scales
// (one per 32 K) itself, accumulating in fp32 in tensor memory: nothing is
// dequantised, so the kernel only has to move bytes.  The rows of an expert
// are the M side (128 to a tile) and its weight rows the N side, so that a
// thread of the epilogue holds consecutive outputs of one row: a block of 32
// hidden values and its scale are formed in one thread's registers when the
// SwiGLU output is quantised again for the second product.  (With few rows
// the M side is mostly empty; the tensor cores then do up to 128 times the
// work asked for, but at 17/32 byte per weight the weight stream, not the
// tensor pipe, is the bound: a stage of 256 weight rows x 256 K takes four
// instructions of about 128 cycles and 34 KB, which at the memory's share
// per SM of about 23 bytes a cycle arrive in 1500.)
//
// Warps: 0 loads the weights' codes (TMA, 128B swizzle) and scales (bulk
// copies of scale tiles); 2 the rows' codes (one box of 128 rows, or boxes of
// 32 for a short tile); 3 the rows' scales, which lie row by row (row offsets
// of a bin are arbitrary, so they cannot come as tiles), and writes them in
// tile order; 1 issues the scale copies into tensor memory and the products;
// 4-11 are the epilogue, two warps to a lane quadrant, each with every other
// group of 64 columns.
//
// Tensor memory (512 columns) at 256 outputs a tile: two accumulators of 256
// that share 48 columns, and two sets of scale columns.  The epilogue takes
// the shared group of a tile's columns first, and the next tile's products
// start as soon as that group is read, so they hide the rest of the
// epilogue.  A set of scale columns is written again only after the products
// that read it have completed (the commit of their stage).
//
// The tiles of the last round over the SMs are cut into halves of 128 outputs
// where that lets more SMs share them (a small call is all last round): FFN of
// 64 experts, 1 token 23.8 -> 20.1 us, product of 512 x 4096 x 4096 14.1 ->
// 13.1 us.
//
// Where experts have many rows the bound is not established.  A stage is 52 KB
// for 512 cycles of products; 32768 rows of 64 experts, 2048 x 2048 and 2048 x
// 1024 (an FFN: 160 us in a short run, 2.6 PFLOP/s; 182 in a long one) load
// and store 1.6 GB between L2 and the SMs, 16384 rows of 8 experts at d =
// 4096, F = 14336 (1.46 ms in a short run, 4.0 PFLOP/s; 1.60 in a long one,
// under the power cap) 17.5 GB: 10 and 12 TB/s, with the tensor pipe 32 to
// 43 % busy.  Pairs of SMs that share a weight tile (two thirds of a stage's
// bytes) were 5 % faster at 2048 rows an expert and up to 18 % slower below,
// so bytes are not all of it; a stage's six scale copies and four products
// wait for the products of two stages before (two sets of scale columns),
// which was not timed apart.  Sixteen epilogue warps in place of eight took 182
// us for the first.
//
// Every wait is bounded; on a timeout the CTA raises MOE_DEV_TIMEOUT, lets its
// copies land, frees tensor memory and returns.
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>
#include <type_traits>

#include "mx.cuh"
#include "ptx.cuh"

namespace moeq {
namespace {

using namespace ptx;

constexpr int kThreads = 384;
constexpr int kM = 128;       // rows of a tile
constexpr int kKS = 256;      // K of a stage (128 bytes of codes)
constexpr int kABox = 32;     // rows of one activation box
constexpr int kEpiWarps = 8;
constexpr int kStageOut = 2048;  // staging bytes of an epilogue warp: 32 rows x 64 bytes

constexpr int kNT = 256;      // outputs of a tile (half tiles: 128)
constexpr int kStages = 4;
constexpr int kSets = 2;      // sets of scale columns
constexpr int kA = kM * 128, kB = kNT * 128;  // bytes of a stage: codes of the rows, of the weights,
constexpr int kSA = 1024, kSB = 2048;         // their scales
constexpr int kOffB = kStages * kA;
constexpr int kOffSA = kOffB + kStages * kB;
constexpr int kOffSB = kOffSA + kStages * kSA;
constexpr int kOffOut = kOffSB + kStages * kSB;
constexpr int kOffTile = kOffOut + kEpiWarps * kStageOut;  // int tile_start[E + 1], off[E + 1]
constexpr int kOffBar = kOffTile + 2 * (kMxMaxExperts + 1) * 4;
constexpr int kOffMisc = kOffBar + (2 * kStages + 4 + 2) * 8;
constexpr int kSmem = kOffMisc + 16;
static_assert(kSmem <= 232448, "shared memory");
constexpr int kAcc1 = 208;  // first column of the second accumulator
constexpr int kSF0 = kAcc1 + kNT, kSFCols = 24;
static_assert(kSF0 + kSets * kSFCols <= 512, "tensor memory");

struct Params {
  CUtensorMap a;      // codes of the rows: bytes [rows][K/2], boxes of 32 rows
  CUtensorMap a_all;  // the same, boxes of 128 rows
  CUtensorMap b;       // codes of the matrices: bytes [E][N][K/2], boxes of 256 rows
  CUtensorMap b_half;  // the same, boxes of 128 rows
  const uint8_t* a_scales;
  const uint8_t* b_scales;  // scale section of matrix 0
  size_t mat_stride;
  const int32_t* offsets;
  int rows, E, N, K;
  void* out;
  uint8_t* out_scales;
  int32_t* status;
  uint64_t wait_ns;  // limit of a wait
  int stall;         // test hook: CTA 0 does not say that its first tile's sums are complete
};

struct Tile {
  int e, row0, nrows, n0, nn;
};

// Tile t of the list.  From `cut` on the tiles are cut in two (128 outputs
// each): the last round's, where that lets twice as many SMs share them.
__device__ __forceinline__ Tile decode_tile(int t, int cut, const int* tile_start, const int* off, int E, int N) {
  int half = 0, nn = kNT;
  if (t >= cut) {
    half = (t - cut) & 1;
    nn = kNT / 2;
    t = cut + ((t - cut) >> 1);
  }
  int lo = 0, hi = E;  // largest e with tile_start[e] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tile_start[mid] <= t) lo = mid; else hi = mid;
  }
  Tile T;
  T.e = lo;
  const int o0 = off[lo], n = off[lo + 1] - o0;
  const int mt = (n + kM - 1) / kM;
  const int local = t - tile_start[lo];
  // row tiles inside a weight tile: CTAs that run together share its codes
  const int nb = local / mt, mb = local - nb * mt;
  T.row0 = o0 + mb * kM;
  T.nrows = min(kM, n - mb * kM);
  T.n0 = nb * kNT + half * (kNT / 2);
  T.nn = min(nn, N - T.n0);
  return T;
}

// Tiles of 128 rows per expert -> exclusive scan over the experts, by all
// threads; ends with warp 0 having written tile_start (the caller
// synchronises).  Offsets are clamped into [0, rows]: no table can send a tile
// outside.  One that does not rise from 0 to rows is flagged.
__device__ __forceinline__ void build_tiles(const int32_t* offsets, int E, int rows, int NB, int32_t* status,
                                            int* tile_start, int* off_s) {
  const int tid = threadIdx.x, lane = tid & 31;
  for (int b = tid; b <= E; b += blockDim.x) {
    const int v = offsets[b];
    const int c = min(max(v, 0), rows);
    if (c != v || (b == 0 && v != 0) || (b == E ? v != rows : offsets[b + 1] < v)) flag_status(status, MOE_DEV_BAD_INDEX);
    off_s[b] = c;
  }
  __syncwarp();
  __syncthreads();
  if (tid < 32) {  // a run of experts per lane
    const int per = (E + 31) / 32, b0 = lane * per;
    int run = 0;
    for (int i = 0; i < per; ++i) {
      const int b = b0 + i;
      if (b < E) {
        const int n = max(0, off_s[b + 1] - off_s[b]);
        tile_start[b] = run;
        run += (n + kM - 1) / kM * NB;
      }
    }
    int incl = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    for (int i = 0; i < per; ++i)
      if (b0 + i < E) tile_start[b0 + i] += incl - run;
    if (lane == 31) tile_start[E] = incl;
  }
}

// 64 columns (outputs n0 .. n0 + 63) of a warp's 32 rows (row0 .., the first
// `live` of them exist) from tensor memory at taddr to the output; whether a
// value left the range.
template <int OUT>
__device__ __forceinline__ bool store_group(void* out_v, uint8_t* out_scales, uint32_t taddr, uint8_t* st, int lane, int row0,
                                            int live, int n0, int N) {
  bool bad = false;
  if (OUT == kMxOutSwiglu) {
    // 32 gate columns and the 32 up columns of the same features: one 32-block of h
    uint32_t g[32], u[32];
    tmem_ld32(taddr, g);
    tmem_ld32(taddr + 32, u);
    tmem_ld_wait();
    float h[32];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      // (a fast division, 2 ulp: the exact one's path for tiny operands, which the rows
      // past the tile's hold, took 4 times as long as all the rest of the kernel.  For g
      // below -87.3, where |silu(g)| < 2^-119, it gives 0.)
      const float gv = __uint_as_float(g[j]);
      h[j] = __fdividef(gv, 1.0f + __expf(-gv)) * __uint_as_float(u[j]);
      m = max(m, __float_as_uint(h[j]) & 0x7FFFFFFFu);
    }
    const uint32_t byte = mx_scale_byte(m);
    uint32_t w[4] = {0, 0, 0, 0};
    if (byte != 255u) {
      const float inv = mx_inv_scale(byte);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = h[8 * k + j] * inv;
        w[k] = mx_encode8(v);
      }
    }
    if (lane < live) {
      bad = byte == 255u;
      const size_t row = static_cast<size_t>(row0 + lane);
      *reinterpret_cast<uint4*>(static_cast<uint8_t*>(out_v) + row * (N / 4) + n0 / 4) =
          make_uint4(w[0], w[1], w[2], w[3]);
      out_scales[row * (N / 64) + n0 / 64] = static_cast<uint8_t>(byte);
    }
    return bad;
  }
  // 64 bytes of every row at a time through the warp's staging rows (16-byte
  // pieces swizzled by row), so that a store instruction covers whole 64-byte
  // runs
  constexpr int ES = OUT == kMxOutF32 ? 4 : 2, CW = 64 / ES;
  uint8_t* out = static_cast<uint8_t*>(out_v) + (static_cast<size_t>(row0 + (lane >> 2)) * N + n0) * ES + (lane & 3) * 16;
  uint32_t v[64];
  tmem_ld32(taddr, *reinterpret_cast<uint32_t(*)[32]>(v));
  tmem_ld32(taddr + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
  tmem_ld_wait();
#pragma unroll
  for (int c = 0; c < 64; c += CW) {
    __syncwarp();  // the rows staged before have been read
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (OUT == kMxOutF32) {
          w[k] = v[c + 4 * j + k];
        } else {
          const float y0 = __uint_as_float(v[c + 8 * j + 2 * k]), y1 = __uint_as_float(v[c + 8 * j + 2 * k + 1]);
          if (OUT == kMxOutF16) {
            bad |= !(fabsf(y0) <= 65504.0f) || !(fabsf(y1) <= 65504.0f);
            const __half2 h = __floats2half2_rn(y0, y1);
            w[k] = *reinterpret_cast<const uint32_t*>(&h);
          } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(y0, y1);
            w[k] = *reinterpret_cast<const uint32_t*>(&h);
          }
        }
      }
      *reinterpret_cast<uint4*>(st + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
    uint4 t[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = 8 * k + (lane >> 2);
      t[k] = *reinterpret_cast<const uint4*>(st + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) << 4));
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (8 * k + (lane >> 2) < live)
        *reinterpret_cast<uint4*>(out + (static_cast<size_t>(8 * k) * N + c) * ES) = t[k];
  }
  return bad && lane < live;
}

template <int OUT>
__global__ void __launch_bounds__(kThreads, 1) k_mx_gemm(const __grid_constant__ Params P) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  int* tile_start = reinterpret_cast<int*>(smem + kOffTile);
  int* off_s = tile_start + (kMxMaxExperts + 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  const uint32_t bar0 = smem_u32(smem + kOffBar);
  auto full = [&](int i) { return bar0 + 8u * i; };
  auto empty = [&](int i) { return bar0 + 8u * (kStages + i); };
  // the CTA's tile i: its sums are complete; its columns that a later tile overwrites first are read
  auto acc_full = [&](int i) { return bar0 + 8u * (2 * kStages + (i & 1)); };
  auto acc_free = [&](int i) { return bar0 + 8u * (2 * kStages + 2 + (i & 1)); };
  const uint32_t drain_bar = bar0 + 8u * (2 * kStages + 4);
  const uint32_t exit_bar = drain_bar + 8u;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int E = P.E, NB = (P.N + kNT - 1) / kNT;
  const int KB = (P.K + kKS - 1) / kKS;  // stages of a tile; the last may hold 128 K

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full(i), 3);  // warps 0, 2 and 3
      mbar_init(empty(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full(i), 1);
      mbar_init(acc_free(i), kEpiWarps);
    }
    mbar_init(drain_bar, 1);
    mbar_init(exit_bar, kThreads / 32);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 3) tmem_alloc(smem_u32(tmem_slot), 512);
  pdl_wait();
  pdl_trigger();
  build_tiles(P.offsets, E, P.rows, NB, P.status, tile_start, off_s);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int tiles = tile_start[E], cut = tiles;
  if (P.N % kNT == 0) {
    const int last = tiles % static_cast<int>(gridDim.x);
    if (2 * last <= static_cast<int>(gridDim.x)) cut -= last;
    tiles += tiles - cut;
  }

  if (warp == 0 || warp == 2) {
    // ---- weights (warp 0), codes of the rows (warp 2) ------------------------
    int s = 0, ph = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const Tile T = decode_tile(t, cut, tile_start, off_s, E, P.N);
      const int boxes = (T.nrows + kABox - 1) / kABox;
      const bool two_rt = T.nn > 128;
      const uint8_t* sc = P.b_scales + static_cast<size_t>(T.e) * P.mat_stride +
                          static_cast<size_t>(T.n0 >> 7) * (P.K / 128) * 512;
      for (int kb = 0; kb < KB; ++kb) {
        ok = warp_wait(empty(s), ph ^ 1, abort_flag, P.status, P.wait_ns);
        if (!ok) break;
        if (warp == 0) {
          const uint32_t sb = P.K - kb * kKS > 128 ? 1024 : 512;
          const uint32_t sdst = smem_u32(smem + kOffSB + s * kSB);
          elect_expect_tx(full(s), two_rt ? kB + 2 * sb : kB / 2 + sb);
          tma_load_3d(smem_u32(smem + kOffB + s * kB), two_rt ? &P.b : &P.b_half, kb * 128, T.n0, T.e, full(s));
          bulk_load(sdst, sc + static_cast<size_t>(kb) * 1024, sb, full(s));
          if (two_rt)
            bulk_load(sdst + 1024, sc + (static_cast<size_t>(P.K / 128) + 2 * kb) * 512, sb, full(s));
        } else {
          const uint32_t adst = smem_u32(smem + s * kA);
          elect_expect_tx(full(s), boxes * (kABox * 128));
          if (boxes == kM / kABox) {
            tma_load_2d(adst, &P.a_all, kb * 128, T.row0, full(s));
          } else {
            for (int i = 0; i < boxes; ++i)
              tma_load_2d(adst + i * (kABox * 128), &P.a, kb * 128, T.row0 + i * kABox, full(s));
          }
        }
        if (++s == kStages) { s = 0; ph ^= 1; }
      }
    }
    // The copies issued here land before the CTA goes, also where another warp
    // gives up after the last of them was issued (a slot never used is complete).
    uint64_t t0 = 0;
    for (int i = 0; i < kStages; ++i) mbar_drain(full(i), i < s ? ph : ph ^ 1, P.wait_ns, t0);
    __syncwarp();
  } else if (warp == 3) {
    // ---- row scales: four rows a lane, two 128-K words a stage --------------
    constexpr int G = 4;  // stages loaded ahead of the ones being written
    int s = 0, ph = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const Tile T = decode_tile(t, cut, tile_start, off_s, E, P.N);
      const uint8_t* base = P.a_scales + static_cast<size_t>(T.row0 + lane) * (P.K / 32);
      auto fetch = [&](int kb0, uint4 (&w)[G][2]) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int k = (kb0 + g) * kKS + h * 128;
            uint32_t v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              v[j] = k < P.K && lane + 32 * j < T.nrows
                         ? *reinterpret_cast<const uint32_t*>(base + static_cast<size_t>(32 * j) * (P.K / 32) + k / 32)
                         : 0u;
            w[g][h] = make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
      };
      uint4 cur[G][2], nxt[G][2];
      fetch(0, cur);
      for (int kb0 = 0; kb0 < KB && ok; kb0 += G) {
        if (kb0 + G < KB) fetch(kb0 + G, nxt);
#pragma unroll
        for (int g = 0; g < G; ++g) {
          if (kb0 + g < KB && ok) {
            ok = warp_wait(empty(s), ph ^ 1, abort_flag, P.status, P.wait_ns);
            if (ok) {
              uint8_t* dst = smem + kOffSA + s * kSA + lane * 16;
              *reinterpret_cast<uint4*>(dst) = cur[g][0];
              *reinterpret_cast<uint4*>(dst + 512) = cur[g][1];
              fence_async_shared();
              __syncwarp();
              if (lane == 0) mbar_arrive(full(s));
              if (++s == kStages) { s = 0; ph ^= 1; }
            }
          }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
          cur[g][0] = nxt[g][0];
          cur[g][1] = nxt[g][1];
        }
      }
    }
  } else if (warp == 1) {
    // ---- products -----------------------------------------------------------
    int s = 0, ph = 0, n = 0, tile = 0;
    bool ok = true;
    const uint64_t da0 = desc_sw128(smem_u32(smem)), db0 = desc_sw128(smem_u32(smem + kOffB));
    const uint64_t dsa0 = desc_plain(smem_u32(smem + kOffSA)), dsb0 = desc_plain(smem_u32(smem + kOffSB));
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++tile) {
      const Tile T = decode_tile(t, cut, tile_start, off_s, E, P.N);
      const uint32_t id0 = idesc_mxf4(T.nn, 0), id1 = idesc_mxf4(T.nn, 1);
      if (tile >= 1) {  // the columns shared with the tile before
        ok = warp_wait(acc_free(tile - 1), ((tile - 1) >> 1) & 1, abort_flag, P.status, P.wait_ns);
        if (!ok) break;
      }
      tc_fence_after();
      const uint32_t d = tmem + (tile & 1) * kAcc1;
      // A stage's copies and products in one straight line: between branches the
      // compiler moved every operand through ordinary registers (60 cycles an
      // instruction instead of 10).
      auto stage = [&](auto two, uint32_t later) {
        if (!warp_wait(full(s), ph, abort_flag, P.status, P.wait_ns)) return false;
        // the products of kSets stages ago, which read this set of scale columns
        if (n >= kSets &&
            !warp_wait(empty((n - kSets) % kStages), ((n - kSets) / kStages) & 1, abort_flag, P.status, P.wait_ns))
          return false;
        tc_fence_after();
        const uint32_t sfa = tmem + kSF0 + (n % kSets) * kSFCols, sfb = sfa + 8;
        const uint64_t da = da0 + s * (kA >> 4), db = db0 + s * (kB >> 4);
        const uint64_t dsa = dsa0 + s * (kSA >> 4), dsb = dsb0 + s * (kSB >> 4);
        // (a tile of 128 outputs: the second tile of scales is stale and unused)
        tc_copy_scales(sfa, dsa);
        tc_copy_scales(sfb, dsb);
        tc_copy_scales(sfb + 4, dsb + 64);
        if constexpr (two.value) {
          tc_copy_scales(sfa + 4, dsa + 32);
          tc_copy_scales(sfb + 8, dsb + 32);
          tc_copy_scales(sfb + 12, dsb + 96);
        }
        mma_mxf4(d, da, db, id0, sfa, sfb, later);
        mma_mxf4(d, da + 2, db + 2, id1, sfa, sfb, 1u);
        if constexpr (two.value) {
          mma_mxf4(d, da + 4, db + 4, id0, sfa + 4, sfb + 8, 1u);
          mma_mxf4(d, da + 6, db + 6, id1, sfa + 4, sfb + 8, 1u);
        }
        tc_commit(empty(s));
        if (++s == kStages) { s = 0; ph ^= 1; }
        ++n;
        return true;
      };
      for (int kb = 0; kb < P.K / kKS && ok; ++kb) ok = stage(std::true_type{}, kb != 0);
      if (ok && P.K % kKS) ok = stage(std::false_type{}, P.K > kKS);
      if (!ok) break;
      if (!(P.stall && blockIdx.x == 0 && tile == 0)) tc_commit(acc_full(tile));
    }
    // every product issued here completes before tensor memory is released
    tc_commit(drain_bar);
    const uint64_t t0 = global_ns();
    while (!mbar_try(drain_bar, 0) && global_ns() - t0 < P.wait_ns) {}
    __syncwarp();
  } else if (warp >= 4) {
    // ---- epilogue: lane = row of the tile, quadrant = warp % 4; the quadrant's
    // two warps take the even and the odd groups of 64 columns ------------------
    const int q = warp & 3, half = (warp - 4) >> 2;
    const int r = 32 * q + lane;
    int tile = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x, ++tile) {
      const Tile T = decode_tile(t, cut, tile_start, off_s, E, P.N);
      ok = warp_wait(acc_full(tile), (tile >> 1) & 1, abort_flag, P.status, P.wait_ns);
      if (!ok) break;
      tc_fence_after();
      const uint32_t tb = tmem + (static_cast<uint32_t>(32 * q) << 16) + (tile & 1) * kAcc1;
      const bool live = r < T.nrows;
      const bool any = 32 * q < T.nrows;
      const int groups = T.nn / 64;
      bool bad = false;
      // 256 columns: the group in the shared columns is the last of the first
      // accumulator, the first of the second; the warp that has it takes it
      // first and then frees the columns, the other frees them at once
      const bool last_first = (tile & 1) == 0;
      auto freed = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_free(tile));
      };
      if (half != (last_first ? 1 : 0)) freed();
#pragma unroll 1
      for (int i = half; i < 4; i += 2) {
        const int grp = last_first && half == 1 ? 4 - i : i;
        const int c = grp * 64;
        if (grp < groups && any) {
          bad |= store_group<OUT>(P.out, P.out_scales, tb + c, smem + kOffOut + (warp - 4) * kStageOut, lane,
                                  T.row0 + 32 * q, T.nrows - 32 * q, T.n0 + c, P.N);
        }
        if (i == half && half == (last_first ? 1 : 0)) freed();
      }
      if (bad && live) flag_status(P.status, MOE_DEV_RANGE);
    }
  }

  __syncwarp();
  tc_fence_before();
  if (lane == 0) mbar_arrive(exit_bar);
  if (warp == 3) {  // frees tensor memory once every warp has left its loop
    const uint64_t t0 = global_ns();
    while (!mbar_try(exit_bar, 0) && global_ns() - t0 < 2 * P.wait_ns) {}
    __syncwarp();
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

// ---- host side ----------------------------------------------------------------

PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Codes: rows of bytes, 128B swizzle.
bool encode_bytes(CUtensorMap* m, int rank, const void* base, const cuuint64_t* dims, const cuuint64_t* strides,
                         const cuuint32_t* box) {
  auto fn = get_encode();
  if (!fn) return false;
  const cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int OUT>
moe_status_t launch(const MxGemmArgs& a, cudaStream_t s) {
  Params P{};
  {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.K / 2), static_cast<cuuint64_t>(a.rows)};
    const cuuint64_t str[1] = {static_cast<cuuint64_t>(a.K / 2)};
    const cuuint32_t box[2] = {128, kABox};
    const cuuint64_t dimb[3] = {static_cast<cuuint64_t>(a.K / 2), static_cast<cuuint64_t>(a.N),
                                static_cast<cuuint64_t>(a.E)};
    const cuuint64_t strb[2] = {static_cast<cuuint64_t>(a.K / 2), static_cast<cuuint64_t>(a.mat_stride)};
    const cuuint32_t boxb[3] = {128, kNT, 1}, boxh[3] = {128, kNT / 2, 1};
    const cuuint32_t box_all[2] = {128, kM};
    if (!encode_bytes(&P.a, 2, a.a_codes, dims, str, box) || !encode_bytes(&P.a_all, 2, a.a_codes, dims, str, box_all) ||
        !encode_bytes(&P.b, 3, a.mats, dimb, strb, boxb) || !encode_bytes(&P.b_half, 3, a.mats, dimb, strb, boxh)) {
      set_error("tensor map (MXFP4 codes) could not be encoded");
      return MOE_ERR_CUDA;
    }
  }
  P.a_scales = a.a_scales;
  P.b_scales = a.mats + static_cast<size_t>(a.N) * (a.K / 2);
  P.mat_stride = a.mat_stride;
  P.offsets = a.offsets;
  P.rows = a.rows;
  P.E = a.E;
  P.N = a.N;
  P.K = a.K;
  P.out = a.out;
  P.out_scales = a.out_scales;
  P.status = a.status;
  P.wait_ns = g_mx_stall ? kStallLimitNs : kWaitLimitNs;
  P.stall = g_mx_stall;
  // shared-memory opt-in: a per-device attribute, set once per device (the
  // first call on a device precedes any stream capture)
  static std::atomic<uint64_t> attr_set{0};
  static std::atomic<int> sms[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_check(e, "MXFP4 product: cudaGetDevice");
  if (dev < 0 || dev >= 64) {
    set_error("MXFP4 product: device %d beyond the supported 64", dev);
    return MOE_ERR_UNSUPPORTED_SHAPE;
  }
  auto kern = k_mx_gemm<OUT>;
  if (!(attr_set.load() & (1ull << dev))) {
    int n = 0;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_check(e, "MXFP4 product: shared-memory attribute");
    sms[dev].store(n);
    attr_set.fetch_or(1ull << dev);
  }
  const long most = (static_cast<long>(a.rows) / kM + std::min(a.E, a.rows)) * ceil_div(a.N, kNT) * 2;
  const int grid = static_cast<int>(std::min<long>(most, sms[dev].load()));
  return cuda_check(launch_pdl(pdl_for(a.rows), kern, dim3(grid), dim3(kThreads), kSmem, s, P),
                    "MXFP4 product launch");
}

}  // namespace

int g_mx_stall = 0;

moe_status_t launch_mx_gemm(const MxGemmArgs& a, cudaStream_t s) {
  if (a.rows == 0) return MOE_OK;
  switch (a.out_kind) {
    case kMxOutF16: return launch<kMxOutF16>(a, s);
    case kMxOutBf16: return launch<kMxOutBf16>(a, s);
    case kMxOutF32: return launch<kMxOutF32>(a, s);
    default: return launch<kMxOutSwiglu>(a, s);
  }
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Checks shared by the two entry points.
moe_status_t check(const char* fn, const void* codes, const void* scales, const int32_t* offsets, const void* mats,
                   const void* out, int rows, int E, int N, int K) {
  if (rows < 0 || E <= 0 || N <= 0 || K <= 0) {
    set_error("%s: bad sizes rows=%d E=%d N=%d K=%d", fn, rows, E, N, K);
    return MOE_ERR_INVALID_ARG;
  }
  if (N % 128 || K % 128 || N > (1 << 24) || K > (1 << 24) || E > kMxMaxExperts) {
    set_error("%s: N=%d and K=%d must be multiples of 128 (up to 2^24), E=%d at most %d", fn, N, K, E, kMxMaxExperts);
    return MOE_ERR_UNSUPPORTED_SHAPE;
  }
  // tile numbers are 32-bit, whatever the offsets hold (out of order, every
  // expert could claim all the rows)
  if ((static_cast<long>(rows) / kM + 1) * E * ceil_div(N, kNT) * 2 > 0x7FFFFFFFL) {
    set_error("%s: rows=%d, E=%d, N=%d could make more than 2^31 - 1 tiles", fn, rows, E, N);
    return MOE_ERR_UNSUPPORTED_SHAPE;
  }
  if (rows == 0) return MOE_OK;
  if (!codes || !scales || !offsets || !mats || !out) {
    set_error("%s: null pointer", fn);
    return MOE_ERR_INVALID_ARG;
  }
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(mats) || !aligned16(out)) {
    set_error("%s: codes, scales, weights and output must be 16-byte aligned", fn);
    return MOE_ERR_INVALID_ARG;
  }
  return MOE_OK;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace
}  // namespace moeq

using namespace moeq;

extern "C" {

moe_status_t moe_mx_grouped_gemm(const void* codes, const void* scales, const int32_t* offsets, const void* mats,
                                 int rows, int E, int N, int K, int out_dtype, void* out, int32_t* status,
                                 moe_stream_t stream) {
  const char* fn = "moe_mx_grouped_gemm";
  const moe_status_t st = check(fn, codes, scales, offsets, mats, out, rows, E, N, K);
  if (st != MOE_OK) return st;
  if (out_dtype != MOE_F32 && out_dtype != MOE_BF16 && out_dtype != MOE_F16) {
    set_error("%s: unknown output dtype %d", fn, out_dtype);
    return MOE_ERR_INVALID_ARG;
  }
  MxGemmArgs a{};
  a.a_codes = static_cast<const uint8_t*>(codes);
  a.a_scales = static_cast<const uint8_t*>(scales);
  a.offsets = offsets;
  a.mats = static_cast<const uint8_t*>(mats);
  a.mat_stride = mx_matrix_bytes(N, K);
  a.rows = rows;
  a.E = E;
  a.N = N;
  a.K = K;
  a.out_kind = out_dtype == MOE_F32 ? kMxOutF32 : out_dtype == MOE_BF16 ? kMxOutBf16 : kMxOutF16;
  a.out = out;
  a.status = status;
  return launch_mx_gemm(a, static_cast<cudaStream_t>(stream));
}

// Codes of h, then its scales.
size_t moe_ffn_mx_workspace_bytes(int rows, int F) {
  if (rows <= 0 || F <= 0) return 256;
  return up256(static_cast<size_t>(rows) * (F / 2)) + up256(static_cast<size_t>(rows) * (F / 32));
}

moe_status_t moe_grouped_ffn_mx(const void* codes, const void* scales, const int32_t* offsets, const void* blobs,
                                int rows, int E, int d, int F, void* workspace, size_t workspace_bytes, void* y_perm,
                                int32_t* status, moe_stream_t stream) {
  const char* fn = "moe_grouped_ffn_mx";
  moe_status_t st = check(fn, codes, scales, offsets, blobs, y_perm, rows, E, d, F);
  if (st == MOE_OK) st = check(fn, codes, scales, offsets, blobs, y_perm, rows, E, 2 * F, d);
  if (st != MOE_OK) return st;
  if (rows == 0) return MOE_OK;
  const size_t need = moe_ffn_mx_workspace_bytes(rows, F);
  if (!workspace || workspace_bytes < need) {
    set_error("%s: workspace %zu < %zu bytes", fn, workspace_bytes, need);
    return MOE_ERR_WORKSPACE;
  }
  if (!aligned16(workspace)) {
    set_error("%s: workspace must be 16-byte aligned", fn);
    return MOE_ERR_INVALID_ARG;
  }
  uint8_t* hc = static_cast<uint8_t*>(workspace);
  uint8_t* hs = hc + up256(static_cast<size_t>(rows) * (F / 2));
  MxGemmArgs a{};
  a.a_codes = static_cast<const uint8_t*>(codes);
  a.a_scales = static_cast<const uint8_t*>(scales);
  a.offsets = offsets;
  a.mats = static_cast<const uint8_t*>(blobs);
  a.mat_stride = mx_matrix_bytes(2 * F, d) + mx_matrix_bytes(d, F);
  a.rows = rows;
  a.E = E;
  a.N = 2 * F;
  a.K = d;
  a.out_kind = kMxOutSwiglu;
  a.out = hc;
  a.out_scales = hs;
  a.status = status;
  st = launch_mx_gemm(a, static_cast<cudaStream_t>(stream));
  if (st != MOE_OK) return st;
  a.a_codes = hc;
  a.a_scales = hs;
  a.mats = static_cast<const uint8_t*>(blobs) + mx_matrix_bytes(2 * F, d);
  a.N = d;
  a.K = F;
  a.out_kind = kMxOutF16;
  a.out = y_perm;
  a.out_scales = nullptr;
  return launch_mx_gemm(a, static_cast<cudaStream_t>(stream));
}

void moe_debug_mx_timeout(int enable) { g_mx_stall = enable ? 1 : 0; }

}  // extern "C"
