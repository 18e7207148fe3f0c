// Router logits on the tensor cores, with a proven bound.
//
// x is bf16 and W_r fp32.  Each weight is split into three bf16 parts,
// w = hi + mid + lo + r with |mid| <= 2^-9 |w| (1 + 2^-9), |lo| <= 2^-18 |w|
// (1 + 2^-9) and |r| <= 2^-27 |w| (k_route_split), so x . w is three bf16
// products whose element products are exact in fp32.
//
// Bound.  The accumulation is "at least single precision": a sum of m exact
// products, in any order and rounded in any direction, errs by at most
// m 2^-23 (1 + m 2^-23) times the sum of their magnitudes, which is at most
// |x| |W_e|.  A chain over all of d would make that useless, so the hi
// products are taken 64 at a time: after each 64-wide chunk the accumulator
// is read and added in fp32 (round to nearest) to running totals.  The mid
// and lo products are 2^-9 as large and stay in one accumulator.  With
// chunks = d / 64 and S slices of d:
//   |L - l| <= |x| |W_e| (64 2^-23 + (chunks + S + 2) 2^-24
//                         + 2 d 2^-23 2^-9 1.01 + 2^-26)
// and the select kernel takes 1.1 times that (second-order terms).  Parts and
// activations that are subnormal in bf16 may count as zero, 2^-126 each: at
// most 2^-126 sqrt(d) (3 |x| + |W_e|), which the select kernel adds.  Products
// and sums below fp32's range lose at most 2^-126 each, 12 d of them less than
// 1e-32: under the 1e-30 that it adds too.  |x| and |W_e| come from fp32 sums of
// squares, and a square below 2^-150 counts there as zero: the select kernel
// adds d 2^-149 to each sum (a row of 2^-76 had norm 0 without it, and its
// near ties were settled on the fp32 sums).
//
// A CTA computes 128 experts x 256 tokens of one slice of d: the experts are
// the M side (a lane of tensor memory is an expert, so a warp's stores of
// one token are 128 contiguous bytes), the tokens N.  Per 64 K: four
// instructions for hi, whose result the epilogue drains (8 warps, half of
// the tokens each) while the eight of mid and lo run into the second
// accumulator; both take all 512 columns.  80 KB a stage for 12 x 128 cycles
// of instructions: 53 bytes a cycle and SM, about what L2 delivers.  8191
// tokens, 256 experts, d = 4096: 51 us (1.0 PFLOP/s of bf16 products, 61 % of
// the measured rate, on 128 of the 148 SMs; the tensor pipe is busy 61 % of the
// time; fp32 sums took 683 us with their selection).
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>

#include "mx.cuh"
#include "ptx.cuh"

namespace moeq {
namespace {

using namespace ptx;

constexpr int kE = 128, kT = 256;     // experts, tokens of a tile
constexpr int kThreads = 384;
constexpr int kStages = 2;
constexpr int kX = kT * 128, kW = kE * 128;  // bytes of a stage's tokens, of one part of its weights
constexpr int kStage = kX + 3 * kW;
constexpr int kOffBar = kStages * kStage;
constexpr int kSmem = kOffBar + 8 * (2 * kStages + 5) + 16;
static_assert(kSmem <= 232448, "shared memory");

struct Params {
  CUtensorMap x;  // bf16 [T][d]
  CUtensorMap w;  // bf16 [3][E][d]
  float* partial;  // [S][T][E]
  float* xsq;      // [S][T]
  int T, E, chunks, per_split;
  int32_t* status;
  uint64_t wait_ns;  // limit of a wait
  int stall;         // test hook: the first CTA does not say that its first sums are complete
};

__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// fp32 sums of bf16 products (both K-major), M = 128, N = 256
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(kT >> 3) << 17) |
                            (static_cast<uint32_t>(kE >> 4) << 24);

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// W_r row -> its three parts, and its sum of squares.  A CTA per expert.
__global__ void __launch_bounds__(256) k_route_split(const float* __restrict__ w, int E, int d,
                                                     __nv_bfloat16* __restrict__ parts, float* __restrict__ wsq,
                                                     int32_t* __restrict__ list) {
  pdl_wait();
  pdl_trigger();
  const int e = blockIdx.x;
  if (e == 0 && threadIdx.x == 0) list[0] = 0;
  const size_t plane = static_cast<size_t>(E) * d;
  float sq = 0.f;
  for (int i = threadIdx.x * 4; i < d; i += 1024) {
    const float4 v = *reinterpret_cast<const float4*>(w + static_cast<size_t>(e) * d + i);
    const float a[4] = {v.x, v.y, v.z, v.w};
    __nv_bfloat16 h[3][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float r = a[j];
      sq = fmaf(r, r, sq);
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        h[p][j] = __float2bfloat16_rn(r);
        r -= __bfloat162float(h[p][j]);  // exact
      }
    }
#pragma unroll
    for (int p = 0; p < 3; ++p)
      *reinterpret_cast<uint2*>(parts + p * plane + static_cast<size_t>(e) * d + i) =
          *reinterpret_cast<const uint2*>(h[p]);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
  __shared__ float part[8];
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sq;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 8; ++i) sq += part[i];
    wsq[e] = sq;
  }
}

__global__ void __launch_bounds__(kThreads, 1) k_route_tc(const __grid_constant__ Params P) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kSmem - 16);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kSmem - 12);
  const uint32_t bar0 = smem_u32(smem + kOffBar);
  auto full = [&](int i) { return bar0 + 8u * i; };
  auto empty = [&](int i) { return bar0 + 8u * (kStages + i); };
  const uint32_t hi_full = bar0 + 8u * (2 * kStages), hi_free = hi_full + 8u, ml_full = hi_free + 8u;
  const uint32_t exit_bar = ml_full + 8u, drain_bar = exit_bar + 8u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t0 = blockIdx.x * kT, e0 = blockIdx.y * kE, split = blockIdx.z;
  const int c0 = split * P.per_split, n = max(0, min(P.per_split, P.chunks - c0));
  const bool norms = blockIdx.y == 0;  // this CTA also sums the squares of its tokens' slices

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), norms ? 9 : 1);  // the products; the 8 warps that read the tokens
    }
    mbar_init(hi_full, 1);
    mbar_init(hi_free, 8);
    mbar_init(ml_full, 1);
    mbar_init(exit_bar, kThreads / 32);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 2) tmem_alloc(smem_u32(tmem_slot), 512);
  pdl_wait();
  pdl_trigger();
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    bool ok = true;
    int armed = 0;
    for (int c = 0; c < n; ++c) {
      const int s = c % kStages;
      ok = warp_wait(empty(s), ((c / kStages) & 1) ^ 1, abort_flag, P.status, P.wait_ns);
      if (!ok) break;
      const uint32_t dst = smem_u32(smem + s * kStage);
      elect_expect_tx(full(s), kStage);
      tma_load_2d(dst, &P.x, (c0 + c) * 64, t0, full(s));
      for (int p = 0; p < 3; ++p) tma_load_3d(dst + kX + p * kW, &P.w, (c0 + c) * 64, e0, p, full(s));
      armed = c + 1;
    }
    // the copies issued here land before the CTA goes, also where another warp
    // gives up after the last of them was issued
    uint64_t g0 = 0;
    for (int c = max(0, armed - kStages); c < armed; ++c)
      mbar_drain(full(c % kStages), (c / kStages) & 1, P.wait_ns, g0);
    __syncwarp();
  } else if (warp == 1) {
    bool ok = true;
    const uint64_t d0 = desc_sw128(smem_u32(smem));
    for (int c = 0; c < n; ++c) {
      const int s = c % kStages;
      ok = warp_wait(full(s), (c / kStages) & 1, abort_flag, P.status, P.wait_ns);
      if (ok && c > 0) ok = warp_wait(hi_free, (c - 1) & 1, abort_flag, P.status, P.wait_ns);
      if (!ok) break;
      tc_fence_after();
      const uint64_t bx = d0 + s * (kStage >> 4), aw = bx + (kX >> 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) mma_bf16(tmem, aw + 2 * k, bx + 2 * k, kIdesc, k != 0);
      if (!(P.stall && (blockIdx.x | blockIdx.y | blockIdx.z) == 0 && c == 0)) tc_commit(hi_full);
#pragma unroll
      for (int p = 1; p < 3; ++p)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_bf16(tmem + 256, aw + p * (kW >> 4) + 2 * k, bx + 2 * k, kIdesc, c != 0 || p != 1 || k != 0);
      tc_commit(empty(s));
    }
    if (ok) tc_commit(ml_full);
    tc_commit(drain_bar);  // every product completes before tensor memory is released
    const uint64_t g0 = global_ns();
    while (!mbar_try(drain_bar, 0) && global_ns() - g0 < P.wait_ns) {}
    __syncwarp();
  } else if (warp >= 4) {
    // lane = expert 32 q + lane of the tile, 128 tokens; as a norm thread, token `row`
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t tb = tmem + (static_cast<uint32_t>(32 * q) << 16) + half * 128;
    const int row = tid - 128;
    float tot[128];
#pragma unroll
    for (int i = 0; i < 128; ++i) tot[i] = 0.f;
    float sq = 0.f;
    bool ok = true;
    for (int c = 0; c < n; ++c) {
      const int s = c % kStages;
      if (norms) {
        ok = warp_wait(full(s), (c / kStages) & 1, abort_flag, P.status, P.wait_ns);
        if (!ok) break;
        const uint8_t* xr = smem + s * kStage + row * 128;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint4 v = *reinterpret_cast<const uint4*>(xr + ((j ^ (row & 7)) << 4));
          const uint32_t b[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float lo = __uint_as_float(b[i] << 16), hi = __uint_as_float(b[i] & 0xFFFF0000u);
            sq = fmaf(lo, lo, fmaf(hi, hi, sq));
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty(s));
      }
      ok = warp_wait(hi_full, c & 1, abort_flag, P.status, P.wait_ns);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < 128; i += 16) {
        uint32_t v[16];
        tmem_ld16(tb + i, v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) tot[i + j] += __uint_as_float(v[j]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(hi_free);
    }
    if (ok && n > 0) ok = warp_wait(ml_full, 0, abort_flag, P.status, P.wait_ns);
    if (ok) {
      tc_fence_after();
      const int e = e0 + 32 * q + lane;
      float* out = P.partial + static_cast<size_t>(split) * P.T * P.E + e;
#pragma unroll
      for (int i = 0; i < 128; i += 16) {
        uint32_t v[16];
        if (n > 0) {
          tmem_ld16(tb + 256 + i, v);
          tmem_ld_wait();
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int t = t0 + half * 128 + i + j;
          if (t < P.T && e < P.E)
            out[static_cast<size_t>(t) * P.E] = n > 0 ? tot[i + j] + __uint_as_float(v[j]) : 0.f;
        }
      }
      if (norms && t0 + row < P.T) P.xsq[static_cast<size_t>(split) * P.T + t0 + row] = sq;
    }
  }
  __syncwarp();
  tc_fence_before();
  if (lane == 0) mbar_arrive(exit_bar);
  if (warp == 2) {  // frees tensor memory once every warp has left its loop
    const uint64_t g0 = global_ns();
    while (!mbar_try(exit_bar, 0) && global_ns() - g0 < 2 * P.wait_ns) {}
    __syncwarp();
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

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

bool encode(CUtensorMap* m, int rank, const void* base, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
  auto fn = get_encode();
  const cuuint32_t es[3] = {1, 1, 1};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Plan {
  int splits, per_split, chunks;
  size_t xsq, wsq, list, parts, bytes;  // offsets in the workspace
};

Plan plan_for(int T, int d, int E) {
  Plan p;
  p.chunks = ceil_div(d, 64);
  const int tiles = ceil_div(T, kT) * ceil_div(E, kE);
  const int want = std::max(1, std::min(std::min(16, p.chunks), 148 / tiles));  // about one CTA per SM
  p.per_split = ceil_div(p.chunks, want);
  p.splits = ceil_div(p.chunks, p.per_split);
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  p.xsq = up(static_cast<size_t>(std::max(p.splits, 2)) * T * E * 4);  // (two: one fp64 logit each)
  p.wsq = p.xsq + up(static_cast<size_t>(p.splits) * T * 4);
  p.list = p.wsq + up(static_cast<size_t>(E) * 4);
  p.parts = p.list + up((static_cast<size_t>(T) + 1) * 4);
  p.bytes = p.parts + static_cast<size_t>(3) * E * d * 2;
  return p;
}

}  // namespace

// Enough for every smaller T too (fewer tokens are cut into more slices).
size_t route_tc_workspace_bytes(int T, int d, int E) {
  size_t most = plan_for(T, d, E).bytes;
  for (int a = 1; a <= 148 && a * kT < T; ++a) most = std::max(most, plan_for(a * kT, d, E).bytes);
  return most;
}

moe_status_t launch_route_partials_tc(const void* x, const float* w_router, int T, int d, int E, void* workspace,
                                      int32_t* status, RoutePartials* out, cudaStream_t s) {
  const Plan p = plan_for(T, d, E);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  __nv_bfloat16* parts = reinterpret_cast<__nv_bfloat16*>(ws + p.parts);
  float* wsq = reinterpret_cast<float*>(ws + p.wsq);
  Params P{};
  const cuuint64_t dd = static_cast<cuuint64_t>(d);
  const cuuint64_t dx[2] = {dd, static_cast<cuuint64_t>(T)}, sx[1] = {2 * dd};
  const cuuint32_t bx[2] = {64, kT};
  const cuuint64_t dw[3] = {dd, static_cast<cuuint64_t>(E), 3}, sw[2] = {2 * dd, 2 * dd * E};
  const cuuint32_t bw[3] = {64, kE, 1};
  if (!encode(&P.x, 2, x, dx, sx, bx) || !encode(&P.w, 3, parts, dw, sw, bw)) {
    set_error("moe_route_scored: tensor map could not be encoded");
    return MOE_ERR_CUDA;
  }
  P.partial = reinterpret_cast<float*>(ws);
  P.xsq = reinterpret_cast<float*>(ws + p.xsq);
  P.T = T;
  P.E = E;
  P.chunks = p.chunks;
  P.per_split = p.per_split;
  P.status = status;
  P.wait_ns = g_mx_stall ? kStallLimitNs : kWaitLimitNs;
  P.stall = g_mx_stall;
  // shared-memory opt-in: a per-device attribute, set once per device (the
  // first call on a device precedes any stream capture)
  static std::atomic<uint64_t> attr_set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_check(e, "moe_route_scored cudaGetDevice");
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!bit || !(attr_set.load() & bit)) {
    e = cudaFuncSetAttribute(k_route_tc, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return cuda_check(e, "moe_route_scored shared-memory attribute");
    attr_set.fetch_or(bit);
  }
  moe_status_t st = cuda_check(launch_pdl(false, k_route_split, dim3(E), dim3(256), 0, s, w_router, E, d, parts, wsq,
                                          reinterpret_cast<int32_t*>(ws + p.list)),
                               "moe_route_scored split launch");
  if (st != MOE_OK) return st;
  st = cuda_check(launch_pdl(true, k_route_tc, dim3(ceil_div(T, kT), ceil_div(E, kE), p.splits), dim3(kThreads), kSmem,
                             s, P),
                  "moe_route_scored logits launch");
  const double u = 1.0 / 16777216.0;
  const double g = 64 * 2 * u + (p.chunks + p.splits + 2) * u + 2.0 * d * 2 * u / 512 * 1.01 + u / 4;
  *out = {P.partial, P.xsq, wsq, p.splits, static_cast<float>(1.1 * g), reinterpret_cast<int32_t*>(ws + p.list),
          reinterpret_cast<double*>(ws), p.xsq};
  return st;
}

}  // namespace moeq
