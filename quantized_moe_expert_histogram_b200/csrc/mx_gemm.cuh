// What the two MXFP4 product kernels (one SM to a tile, two SMs to a tile)
// share: the tile list, the epilogue, the tensor maps.
#pragma once

#include <cudaTypedefs.h>

#include <mutex>

#include "mx.cuh"
#include "ptx.cuh"

namespace moeq {

namespace {

constexpr int kABox = 32;     // rows of one activation box
constexpr int kEpiWarps = 8;
constexpr int kStageOut = 1024;  // staging bytes of an epilogue warp: 32 rows x 32 bytes

struct Tile {
  int e, row0, at, nrows, n0, nn;  // `at`: row0 within the expert
};

template <int M, int NT>
__device__ __forceinline__ Tile decode_tile(int t, const int* tile_start, const int* off, int E, int N) {
  int lo = 0, hi = E;  // largest e with tile_start[e] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tile_start[mid] <= t) lo = mid; else hi = mid;
  }
  // the same in every lane; the shuffles tell the compiler so, which keeps what
  // follows from them in uniform registers
  lo = __shfl_sync(0xffffffffu, lo, 0);
  const int o0 = __shfl_sync(0xffffffffu, off[lo], 0), o1 = __shfl_sync(0xffffffffu, off[lo + 1], 0);
  const int start = __shfl_sync(0xffffffffu, tile_start[lo], 0);
  Tile T;
  T.e = lo;
  const int n = o1 - o0;
  const int mt = (n + M - 1) / M;
  const int local = t - start;
  // row tiles inside a weight tile: CTAs that run together share its codes
  const int nb = local / mt, mb = local - nb * mt;
  T.at = mb * M;
  T.row0 = o0 + T.at;
  T.nrows = min(M, n - mb * M);
  T.n0 = nb * NT;
  T.nn = min(NT, N - T.n0);
  return T;
}


// Tiles of M rows per expert -> exclusive scan over the experts, by all
// threads; ends with warp 0 having written tile_start (the caller
// synchronises).  Offsets are clamped into [0, rows]: no table can send a tile
// outside.
template <int M>
__device__ __forceinline__ void build_tiles(const int32_t* offsets, int E, int rows, int NB, int32_t* status,
                                            int* tile_start, int* off_s) {
  const int tid = threadIdx.x, lane = tid & 31;
  for (int b = tid; b <= E; b += blockDim.x) {
    const int v = offsets[b];
    const int c = min(max(v, 0), rows);
    if (c != v || (b == E ? v != rows : offsets[b + 1] < v)) flag_status(status, MOE_DEV_BAD_INDEX);
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
        run += (n + M - 1) / M * NB;
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
// value left the range.  SwiGLU: scale(lane's row, 32-block) is the scale
// byte's place.
template <int OUT, typename Scale>
__device__ __forceinline__ bool store_group(void* out_v, Scale scale, uint32_t taddr, uint8_t* st, int lane, int row0,
                                            int live, int n0, int N) {
  using namespace ptx;
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
      // past the tile's hold, took 4 times as long as all the rest of the kernel)
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
      *scale(n0 / 64) = static_cast<uint8_t>(byte);
    }
    return bad;
  }
  // 32 bytes of every row at a time through the warp's staging rows (16-byte
  // pieces swapped by row), so that a store instruction covers whole sectors
  constexpr int ES = OUT == kMxOutF32 ? 4 : 2, CW = 32 / ES;
  uint8_t* out = static_cast<uint8_t*>(out_v) + (static_cast<size_t>(row0) * N + n0) * ES + (lane & 1) * 16;
  uint32_t v[32];
#pragma unroll
  for (int c = 0; c < 64; c += CW) {
    if (c % 32 == 0) {
      tmem_ld32(taddr + c, v);
      tmem_ld_wait();
    }
    __syncwarp();  // the rows staged before have been read
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (OUT == kMxOutF32) {
          w[k] = v[c % 32 + 4 * j + k];
        } else {
          const float y0 = __uint_as_float(v[c % 32 + 8 * j + 2 * k]);
          const float y1 = __uint_as_float(v[c % 32 + 8 * j + 2 * k + 1]);
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
      *reinterpret_cast<uint4*>(st + lane * 32 + ((j ^ ((lane >> 2) & 1)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int row = 16 * k + (lane >> 1);
      if (row < live)
        *reinterpret_cast<uint4*>(out + (static_cast<size_t>(row) * N + c) * ES) =
            *reinterpret_cast<const uint4*>(st + row * 32 + (((lane & 1) ^ ((row >> 2) & 1)) << 4));
    }
  }
  return bad && lane < live;
}

inline PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
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
inline bool encode_bytes(CUtensorMap* m, int rank, const void* base, const cuuint64_t* dims, const cuuint64_t* strides,
                         const cuuint32_t* box) {
  auto fn = get_encode();
  if (!fn) return false;
  const cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace moeq
