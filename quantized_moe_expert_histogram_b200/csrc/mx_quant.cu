// MXFP4 quantisation of rows and of weight matrices, and the way back.
//
// A block of 32 elements is four lanes of 8: each lane loads 16 bytes (two
// loads of 16 for fp32), the block's largest magnitude is two shuffles away,
// and a lane's eight codes are one 32-bit word, so loads and stores of a
// warp are contiguous.  A warp takes up to 1024 elements of one row (four
// pieces of 256, their loads in flight together); the 32 scale bytes of the
// chunk are exchanged so that they leave as one 32-byte run.
//
// Rows in expert order: a token's row is quantised once and its codes are
// written to the k places inv_perm names, so x is read once and the
// arithmetic is done once per token, not per assignment.  Bound: HBM (reads of
// x, writes of 17/32 byte per element and assignment).
//
// A block's work is one pass (a persistent grid of 8 blocks an SM took 6 to 8 %
// longer), and what is used once goes through the caches as streaming: fp32
// rows in (134.0 -> 125.5 us for 28673 x 4096 to MXFP4 and back), bf16 values
// out (41.5 -> 35.2 us for 4096 x 2048 to 8 places and back).  In a captured
// graph the two take 122 and 31.6 us: 96 % and 90 % of the copy bandwidth.
// Packing weights (offline): 64 experts of 3 x 2048 x 1024 in 227 us from bf16
// (4.5 TB/s) and 286 us from fp32 (6.4 TB/s); scale bytes leave one by one.
#include "mx.cuh"

namespace moeq {
namespace {

constexpr int kPiece = 256;  // elements of one warp-wide load
constexpr int kPieces = 4;
constexpr int kChunk = kPiece * kPieces;
constexpr int kThreads = 256;
constexpr int kValuesPerBlock = 4 * kThreads;  // words of 8 codes a block of k_mx_values takes

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 r = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const __half* p, float (&v)[8]) {
  const uint4 r = *reinterpret_cast<const uint4*>(p);
  const __half2* h = reinterpret_cast<const __half2*>(&r);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(h[j]);
    v[2 * j] = f.x;
    v[2 * j + 1] = f.y;
  }
}

// Codes and scale byte (the same in a block's four lanes) of the lane's 8
// elements; every lane of the warp takes part.
__device__ __forceinline__ uint32_t quantize8(float (&v)[8], uint32_t& byte) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);  // NaN bits compare above Inf
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  byte = mx_scale_byte(m);
  if (byte == 255u) return 0u;
  const float inv = mx_inv_scale(byte);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= inv;
  return mx_encode8(v);
}

// Codes of a warp's chunk (piece p: elements k0 + 256 p + 8 lane .. + 7) and
// the scale bytes, lane i's being block i of the chunk.  `base` is the
// chunk's first element, `n` its length (a multiple of 32, at most 1024).
template <typename T>
__device__ __forceinline__ bool quantize_chunk(const T* base, int n, int lane, uint32_t (&codes)[kPieces],
                                               uint32_t& scale) {
  float v[kPieces][8];
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const int i = p * kPiece + lane * 8;
    if (i < n) {
      load8(base + i, v[p]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[p][j] = 0.0f;
    }
  }
  uint32_t byte[kPieces];
  bool bad = false;
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    codes[p] = quantize8(v[p], byte[p]);
    bad |= byte[p] == 255u;
  }
  scale = 0;
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {  // block 8 p + (lane & 7) is lanes 4 (lane & 7) .. + 3 of piece p
    const uint32_t b = __shfl_sync(0xffffffffu, byte[p], (lane & 7) * 4);
    if ((lane >> 3) == p) scale = b;
  }
  return bad;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_mx_rows(const T* __restrict__ x, int rows, int K, long ld,
                                                      const int32_t* __restrict__ inv_perm, int k,
                                                      uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                      int32_t* status) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int chunks = (K + kChunk - 1) / kChunk;
  const long items = static_cast<long>(rows) * chunks;
  const long out_rows = static_cast<long>(rows) * k;
  const long warps = static_cast<long>(gridDim.x) * (kThreads / 32);
  unsigned flags = 0;
  for (long it = static_cast<long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); it < items; it += warps) {
    const int t = static_cast<int>(it / chunks);
    const int k0 = static_cast<int>(it - static_cast<long>(t) * chunks) * kChunk;
    const int n = min(kChunk, K - k0);
    uint32_t c[kPieces], sc;
    if (quantize_chunk(x + static_cast<size_t>(t) * ld + k0, n, lane, c, sc)) flags |= MOE_DEV_RANGE;
    for (int j = 0; j < k; ++j) {
      long p = t;
      if (inv_perm) {
        p = inv_perm[static_cast<size_t>(t) * k + j];
        if (p < 0 || p >= out_rows) {  // no such row: nothing is written for it
          flags |= MOE_DEV_BAD_INDEX;
          continue;
        }
      }
      uint8_t* cr = codes + static_cast<size_t>(p) * (K / 2) + k0 / 2;
#pragma unroll
      for (int q = 0; q < kPieces; ++q)
        if (q * kPiece + lane * 8 < n) reinterpret_cast<uint32_t*>(cr)[q * 32 + lane] = c[q];
      if (lane * 32 < n) scales[static_cast<size_t>(p) * (K / 32) + k0 / 32 + lane] = static_cast<uint8_t>(sc);
    }
  }
  if (flags) flag_status(status, flags);
}

// Weight matrices: source row r of expert e becomes row map(r) of the
// expert's matrix at out + e * stride.  mode 0: rows as they are; 1 / 2: the
// gate / up rows of an interleaved gate-and-up matrix (32 gate rows, 32 up
// rows, 32 gate rows, ...).
template <typename T>
__global__ void __launch_bounds__(kThreads) k_mx_pack(const T* __restrict__ w, int E, int n_rows, int K, int mode,
                                                      int N, uint8_t* __restrict__ out, size_t stride,
                                                      int32_t* status) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int chunks = (K + kChunk - 1) / kChunk;
  const long items = static_cast<long>(E) * n_rows * chunks;
  const long warps = static_cast<long>(gridDim.x) * (kThreads / 32);
  bool bad = false;
  for (long it = static_cast<long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); it < items; it += warps) {
    const long row = it / chunks;
    const int k0 = static_cast<int>(it - row * chunks) * kChunk;
    const int e = static_cast<int>(row / n_rows);
    const int r = static_cast<int>(row - static_cast<long>(e) * n_rows);
    const int to = mode == 0 ? r : ((r >> 5) << 6) + (mode == 2 ? 32 : 0) + (r & 31);
    const int n = min(kChunk, K - k0);
    uint32_t c[kPieces], sc;
    bad |= quantize_chunk(w + static_cast<size_t>(row) * K + k0, n, lane, c, sc);
    uint8_t* mat = out + static_cast<size_t>(e) * stride;
    uint8_t* cr = mat + static_cast<size_t>(to) * (K / 2) + k0 / 2;
#pragma unroll
    for (int q = 0; q < kPieces; ++q)
      if (q * kPiece + lane * 8 < n) reinterpret_cast<uint32_t*>(cr)[q * 32 + lane] = c[q];
    if (lane * 32 < n)
      mat[static_cast<size_t>(N) * (K / 2) + mx_scale_at(to, k0 / 32 + lane, K)] = static_cast<uint8_t>(sc);
  }
  if (bad) flag_status(status, MOE_DEV_RANGE);
}

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint4 r;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&r);
#pragma unroll
  for (int j = 0; j < 4; ++j) h[j] = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
  __stcs(reinterpret_cast<uint4*>(p), r);
}

// A thread turns 8 codes into 8 values; four words in flight per thread.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_mx_values(const uint8_t* __restrict__ codes,
                                                        const uint8_t* __restrict__ scales, long words,
                                                        T* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  constexpr int U = kValuesPerBlock / kThreads;
  const long step = static_cast<long>(gridDim.x) * kThreads * U;
  for (long i0 = static_cast<long>(blockIdx.x) * kThreads * U + threadIdx.x; i0 < words; i0 += step) {
    uint32_t w[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long i = i0 + u * kThreads;
      w[u] = i < words ? reinterpret_cast<const uint32_t*>(codes)[i] : 0u;
      b[u] = i < words ? scales[i >> 2] : 0u;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long i = i0 + u * kThreads;
      if (i >= words) break;
      float v[8];
      mx_decode8(w[u], v);
      const float s = mx_scale(b[u]);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= s;
      store8(out + i * 8, v);
    }
  }
}

int blocks_for(long work, long per_block) {
  return static_cast<int>(std::min<long>((work + per_block - 1) / per_block, 1L << 30));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool known_dtype(int dtype) { return dtype == MOE_F32 || dtype == MOE_BF16 || dtype == MOE_F16; }

template <typename T>
cudaError_t pack_one(const void* w, int E, int n_rows, int K, int mode, int N, uint8_t* out, size_t stride,
                     int32_t* status, cudaStream_t s) {
  const long items = static_cast<long>(E) * n_rows * ((K + kChunk - 1) / kChunk);
  return launch_pdl(false, k_mx_pack<T>, dim3(blocks_for(items, kThreads / 32)), dim3(kThreads), 0, s, static_cast<const T*>(w), E,
                    n_rows, K, mode, N, out, stride, status);
}

moe_status_t pack(const void* w, int dtype, int E, int n_rows, int K, int mode, int N, uint8_t* out, size_t stride,
                  int32_t* status, cudaStream_t s, const char* fn) {
  return cuda_check(dtype == MOE_F32    ? pack_one<float>(w, E, n_rows, K, mode, N, out, stride, status, s)
                    : dtype == MOE_BF16 ? pack_one<__nv_bfloat16>(w, E, n_rows, K, mode, N, out, stride, status, s)
                                        : pack_one<__half>(w, E, n_rows, K, mode, N, out, stride, status, s),
                    fn);
}

}  // namespace
}  // namespace moeq

using namespace moeq;

extern "C" {

size_t moe_mx_matrix_bytes(int N, int K) {
  if (N <= 0 || K <= 0 || N % 128 || K % 128) return 0;
  return mx_matrix_bytes(N, K);
}

size_t moe_mx_blob_bytes(int d, int F) {
  if (d <= 0 || F <= 0 || d % 128 || F % 128 || F > (1 << 29)) return 0;
  return mx_matrix_bytes(2 * F, d) + mx_matrix_bytes(d, F);
}

moe_status_t moe_mx_quantize(const void* x, int dtype, int rows, int K, size_t ld, const int32_t* inv_perm, int k,
                             void* codes, void* scales, int32_t* status, moe_stream_t stream) {
  const char* fn = "moe_mx_quantize";
  if (rows < 0 || K <= 0 || k <= 0 || ld < static_cast<size_t>(K) || ld > (static_cast<size_t>(1) << 40) || !known_dtype(dtype)) {
    set_error("%s: bad arguments rows=%d K=%d ld=%zu k=%d dtype=%d", fn, rows, K, ld, k,
              dtype);
    return MOE_ERR_INVALID_ARG;
  }
  if (!inv_perm && k != 1 && rows > 0) {
    set_error("%s: k=%d places a row need inv_perm", fn, k);
    return MOE_ERR_INVALID_ARG;
  }
  const int size = dtype == MOE_F32 ? 4 : 2;
  if (K % kMxBlock || (ld * size) % 16) {
    set_error("%s: K=%d must be a multiple of 32 and rows (ld=%zu) multiples of 16 bytes apart", fn, K, ld);
    return MOE_ERR_UNSUPPORTED_SHAPE;
  }
  if (static_cast<long>(rows) * k > 0x7FFFFFFFL) {
    set_error("%s: rows*k = %ld exceeds 2^31 - 1", fn, static_cast<long>(rows) * k);
    return MOE_ERR_UNSUPPORTED_SHAPE;
  }
  if (rows == 0) return MOE_OK;
  if (!x || !codes || !scales) {
    set_error("%s: null pointer", fn);
    return MOE_ERR_INVALID_ARG;
  }
  if (!aligned16(x) || !aligned16(codes)) {
    set_error("%s: x and codes must be 16-byte aligned", fn);
    return MOE_ERR_INVALID_ARG;
  }
  const long items = static_cast<long>(rows) * ((K + kChunk - 1) / kChunk);
  const dim3 grid(blocks_for(items, kThreads / 32)), block(kThreads);
  const bool pdl = pdl_for(static_cast<long>(rows) * k);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* c = static_cast<uint8_t*>(codes);
  uint8_t* sc = static_cast<uint8_t*>(scales);
  const long l = static_cast<long>(ld);
  cudaError_t e;
  if (dtype == MOE_F32)
    e = launch_pdl(pdl, k_mx_rows<float>, grid, block, 0, s, static_cast<const float*>(x), rows, K, l, inv_perm, k, c,
                   sc, status);
  else if (dtype == MOE_BF16)
    e = launch_pdl(pdl, k_mx_rows<__nv_bfloat16>, grid, block, 0, s, static_cast<const __nv_bfloat16*>(x), rows, K, l,
                   inv_perm, k, c, sc, status);
  else
    e = launch_pdl(pdl, k_mx_rows<__half>, grid, block, 0, s, static_cast<const __half*>(x), rows, K, l, inv_perm, k,
                   c, sc, status);
  return cuda_check(e, "moe_mx_quantize launch");
}

moe_status_t moe_mx_dequantize(const void* codes, const void* scales, int rows, int K, int dtype, void* out,
                               moe_stream_t stream) {
  const char* fn = "moe_mx_dequantize";
  if (rows < 0 || K <= 0 || (dtype != MOE_F32 && dtype != MOE_BF16)) {
    set_error("%s: bad arguments rows=%d K=%d dtype=%d (fp32 or bf16, where every value is exact)", fn, rows, K, dtype);
    return MOE_ERR_INVALID_ARG;
  }
  if (K % kMxBlock) {
    set_error("%s: K=%d must be a multiple of 32", fn, K);
    return MOE_ERR_UNSUPPORTED_SHAPE;
  }
  if (rows == 0) return MOE_OK;
  if (!codes || !scales || !out) {
    set_error("%s: null pointer", fn);
    return MOE_ERR_INVALID_ARG;
  }
  if (!aligned16(codes) || !aligned16(out)) {
    set_error("%s: codes and out must be 16-byte aligned", fn);
    return MOE_ERR_INVALID_ARG;
  }
  const long words = static_cast<long>(rows) * (K / 8);
  const dim3 grid(blocks_for(words, kValuesPerBlock)), block(kThreads);
  const bool pdl = pdl_for(rows);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const uint8_t* c = static_cast<const uint8_t*>(codes);
  const uint8_t* sc = static_cast<const uint8_t*>(scales);
  const cudaError_t e =
      dtype == MOE_F32
          ? launch_pdl(pdl, k_mx_values<float>, grid, block, 0, s, c, sc, words, static_cast<float*>(out))
          : launch_pdl(pdl, k_mx_values<__nv_bfloat16>, grid, block, 0, s, c, sc, words,
                       static_cast<__nv_bfloat16*>(out));
  return cuda_check(e, "moe_mx_dequantize launch");
}

moe_status_t moe_mx_pack(const void* w, int dtype, int E, int N, int K, void* mats, int32_t* status,
                         moe_stream_t stream) {
  const char* fn = "moe_mx_pack";
  if (!w || !mats || E <= 0 || !known_dtype(dtype)) {
    set_error("%s: null pointer, E=%d or dtype=%d", fn, E, dtype);
    return MOE_ERR_INVALID_ARG;
  }
  if (!moe_mx_matrix_bytes(N, K)) {
    set_error("%s: N=%d and K=%d must be multiples of 128", fn, N, K);
    return MOE_ERR_UNSUPPORTED_SHAPE;
  }
  if (!aligned16(w) || !aligned16(mats)) {
    set_error("%s: w and mats must be 16-byte aligned", fn);
    return MOE_ERR_INVALID_ARG;
  }
  return pack(w, dtype, E, N, K, 0, N, static_cast<uint8_t*>(mats), mx_matrix_bytes(N, K), status,
              static_cast<cudaStream_t>(stream), "moe_mx_pack launch");
}

moe_status_t moe_mx_pack_ffn(const void* w_gate, const void* w_up, const void* w_down, int dtype, int E, int d, int F,
                             void* blobs, int32_t* status, moe_stream_t stream) {
  const char* fn = "moe_mx_pack_ffn";
  if (!w_gate || !w_up || !w_down || !blobs || E <= 0 || !known_dtype(dtype)) {
    set_error("%s: null pointer, E=%d or dtype=%d", fn, E, dtype);
    return MOE_ERR_INVALID_ARG;
  }
  const size_t stride = moe_mx_blob_bytes(d, F);
  if (!stride) {
    set_error("%s: d=%d and F=%d must be multiples of 128", fn, d, F);
    return MOE_ERR_UNSUPPORTED_SHAPE;
  }
  if (!aligned16(w_gate) || !aligned16(w_up) || !aligned16(w_down) || !aligned16(blobs)) {
    set_error("%s: the weights and blobs must be 16-byte aligned", fn);
    return MOE_ERR_INVALID_ARG;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* b = static_cast<uint8_t*>(blobs);
  moe_status_t st = pack(w_gate, dtype, E, F, d, 1, 2 * F, b, stride, status, s, "moe_mx_pack_ffn launch (gate)");
  if (st == MOE_OK) st = pack(w_up, dtype, E, F, d, 2, 2 * F, b, stride, status, s, "moe_mx_pack_ffn launch (up)");
  if (st == MOE_OK)
    st = pack(w_down, dtype, E, d, F, 0, d, b + mx_matrix_bytes(2 * F, d), stride, status, s,
              "moe_mx_pack_ffn launch (down)");
  return st;
}

}  // extern "C"
