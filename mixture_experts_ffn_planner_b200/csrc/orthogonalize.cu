// An expert's update made orthogonal by Newton-Schulz steps, for a batch of
// matrices G (M x N): X = G / (|G|_F + eps), then `steps` times
//   A = X X^T,  B = b A + c A A,  X <- a X + B X        (M <= N)
//   A = X^T X,  B = b A + c A A,  X <- a X + X B        (M > N)
// which is the same iteration on the shorter side; A and B are symmetric, so
// the tall form needs no transpose either (tile_gemm.cuh reads MN-major
// operands as they lie).
//
// Precision.  The matrix operands X, A and B are fp16 (11 bits; X is held
// times kScale = 64, which keeps the entries of a unit-norm matrix of 2^22
// elements normal), the sums fp32.  That alone is not enough on a gradient,
// whose spectrum falls off: the step multiplies weak directions by a = 3.44,
// and with them the rounding noise of the strong ones (error 2e-2 of the
// result at rank S/4 + noise).  The term that carries the noise is a X, which
// needs no matrix product, so X is kept as a pair hi + lo / 2048 (22 bits) and
// a X is taken from the pair: 2.0e-3, of which 1.7e-3 is the rounding of the
// bf16 result.  From the fourth step on, when X is nearly orthogonal and B
// nearly a multiple of I, the rounding of B's diagonal is what is left; it is
// taken out of B into fp32 and joins a: 1.7e-3 to 2.3e-3 for matrices of
// sides 65 to 2048, Gaussian, of rank 1 to S/4 with noise or without, or with
// singular values over two to eight decades.  (Earlier it must not be: B's
// product with the strong directions has to stay in one matrix product.)
// Where the values of a result are all alike (of the identity, or of a matrix
// of ones) they are all rounded alike, by up to 2^-8, and 5.3e-3 was met.
//
// Three ways, by the sides:
//   up to 64        fp32, without tensor cores (whose fp16 noise the steps may
//                   amplify to 1e-2 on matrices of a few rows), as one launch:
//                   a cluster of up to 8 CTAs a matrix, each with its share of
//                   the longer side in shared memory from the first step to
//                   the last.  A step sums G G^T over the cluster through
//                   distributed shared memory; everything else is local.
//   65 to 256, the longer side at most 512 (1024 up to 128), few matrices:
//                   one launch on the tensor cores (ns_resident.cuh).
//   else            three chained launches a step (tile_gemm.cuh), of which the
//                   first two compute half of their symmetric results.
// Where the longer side of a matrix of up to 64 rows does not fit (above 5120)
// the iteration runs on S x S matrices alone, in 64 bits, with X = Q G,
//   P = a I + b A + c A A,  Q <- P Q,  A <- P A P     from A = G G^T / (|G| + eps)^2, Q = I / (|G| + eps)
// (|G|_F^2 is the trace of G G^T), in one block a matrix, between one pass over
// G for G G^T and one for Q G.  That takes 64 bits because G G^T squares G's
// range, and because P, Q and A commute only up to rounding, which the steps
// amplify as well: in fp32 a 3 x 5 matrix of rank one plus noise came out 6e-4
// off, and 0.3 where Q stood for its transpose.
//
// |G|_F is summed in 64 bits.  Every sum has a fixed order.  The launches of a
// call are chained by programmatic dependent launch.  16 matrices of 2048 x
// 2048 take 2.5 ms by themselves on a GPU that was idle, and 2.9 to 3.0 ms among
// others of their kind under the power limit: a step 110 us for A, 109 for B
// (tensor pipe 74 % busy at 1.58 GHz), 209 for the update, which moves 652 MB
// beside its product.
#include <algorithm>
#include <cmath>

#include "tile_gemm.cuh"

namespace moe {

constexpr float kNsScale = 64.0f;
constexpr int kNsDiagFrom = 3;      // steps 0, 1, 2 keep B whole
constexpr int kNsChunks = 128;      // blocks that share a matrix's norm, at most
constexpr int kNsThreads = 256;

__device__ __forceinline__ float ns_load(const void* g, int f32, int64_t i) {
  return f32 ? __ldg(static_cast<const float*>(g) + i)
             : __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(g) + i));
}

// 8 elements from i on; vec: a 16-byte (bf16) or two (fp32) aligned loads.
__device__ __forceinline__ void ns_load8(const void* g, int f32, int64_t i, int n, bool vec, float (&v)[8]) {
  if (vec) {
    if (f32) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(g) + i));
      const float4 b = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(g) + i) + 1);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(g) + i));
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = unpack_b16(w[j]);
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? ns_load(g, f32, i + j) : 0.f;
  }
}

// kNsScale / norm (norm: |G| + eps) as two factors, x = (g * pre) * post.  Below 1.9e-37 it is beyond fp32; pre is then
// 2^100, which takes subnormals into range without rounding, and 1 otherwise.
struct NsFactors {
  float pre, post;
};
__device__ __forceinline__ NsFactors ns_factors(double norm) {
  constexpr double kPre = 1267650600228229401496703205376.0;  // 2^100
  const double f = static_cast<double>(kNsScale) / norm;
  const bool tiny = f > 1e18;
  return {tiny ? static_cast<float>(kPre) : 1.0f, static_cast<float>(tiny ? f / kPre : f)};
}

// part[z][chunk] = sum of squares over the chunk's share of matrix z.
__global__ void __launch_bounds__(kNsThreads)
    ns_norm_kernel(const void* __restrict__ g, int f32, int64_t mn, int vec, double* __restrict__ part) {
  pdl_launch_dependents();
  const int64_t groups = (mn + 7) / 8;
  const int64_t base = static_cast<int64_t>(blockIdx.y) * mn;
  double sum = 0.0;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kNsThreads + threadIdx.x; i < groups;
       i += static_cast<int64_t>(gridDim.x) * kNsThreads) {
    float v[8];
    ns_load8(g, f32, base + 8 * i, static_cast<int>(min(static_cast<int64_t>(8), mn - 8 * i)), vec && 8 * i + 8 <= mn, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += static_cast<double>(v[j]) * static_cast<double>(v[j]);
  }
  __shared__ double warps[kNsThreads / 32];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int w = 0; w < kNsThreads / 32; ++w) s += warps[w];
    part[static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x] = s;
  }
}

// hi + lo / 2048 = kNsScale * G / (|G| + eps), rows padded to ld with zeros.
__global__ void __launch_bounds__(kNsThreads)
    ns_init_kernel(const void* __restrict__ g, int f32, int M, int N, int ld, int vec, const double* part, int chunks,
                   double eps, __half* __restrict__ hi, __half* __restrict__ lo) {
  pdl_launch_dependents();
  pdl_wait();  // the partial sums
  __shared__ NsFactors shared_scale;
  if (threadIdx.x < 32) {  // one warp a block: by every thread, one after another, the sums took 1.7 of 1.8 ms at 16 x 2048^2
    double s = 0.0;
    for (int c = static_cast<int>(threadIdx.x); c < chunks; c += 32)
      s += __ldcg(part + static_cast<int64_t>(blockIdx.y) * chunks + c);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (threadIdx.x == 0) shared_scale = ns_factors(sqrt(s) + eps);
  }
  __syncthreads();
  const NsFactors scale = shared_scale;
  const int per_row = ld / 8;
  const int64_t groups = static_cast<int64_t>(M) * per_row;
  const int64_t z = blockIdx.y;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kNsThreads + threadIdx.x; i < groups;
       i += static_cast<int64_t>(gridDim.x) * kNsThreads) {
    const int64_t row = i / per_row;
    const int col = static_cast<int>(i - row * per_row) * 8;
    float v[8];
    ns_load8(g, f32, (z * M + row) * N + col, N - col, vec && col + 8 <= N, v);
    uint32_t wh[4], wl[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x0 = v[2 * j] * scale.pre * scale.post, x1 = v[2 * j + 1] * scale.pre * scale.post;
      wh[j] = pack_f16(x0, x1);
      const float2 h = unpack_f16(wh[j]);
      wl[j] = pack_f16((x0 - h.x) * kLoScale, (x1 - h.y) * kLoScale);
    }
    const int64_t o = (z * M + row) * ld + col;
    *reinterpret_cast<uint4*>(hi + o) = make_uint4(wh[0], wh[1], wh[2], wh[3]);
    *reinterpret_cast<uint4*>(lo + o) = make_uint4(wl[0], wl[1], wl[2], wl[3]);
  }
}

}  // namespace moe

#include "ns_resident.cuh"

namespace moe {

// ------------------------------------------------------- a side of at most 64
constexpr int kNsSmall = 64;
constexpr int kNsSmallChunks = 32;  // blocks that share a matrix's G G^T, at most
using NsRow64 = double[kNsSmall + 2];
using NsRow32 = float[kNsSmall + 4];

// Element (i, l) of a matrix seen from its shorter side: i < side, l < len.
struct NsSide {
  const void* g;
  int f32, tall, side, len;
  __device__ __forceinline__ int64_t at(int64_t z, int i, int l) const {
    return z * side * len + (tall ? static_cast<int64_t>(l) * side + i : static_cast<int64_t>(i) * len + l);
  }
  // (i, l) of the e-th of 64 x 64 elements, consecutive in memory for consecutive e
  __device__ __forceinline__ int i_of(int e) const { return tall ? e % kNsSmall : e / kNsSmall; }
  __device__ __forceinline__ int l_of(int e) const { return tall ? e / kNsSmall : e % kNsSmall; }
};

__device__ __forceinline__ void ns_load4(const double* p, double (&v)[4]) {
  const double2 a = reinterpret_cast<const double2*>(p)[0], b = reinterpret_cast<const double2*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}
__device__ __forceinline__ void ns_load4(const float* p, double (&v)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}

// acc[r][s] += sum over k < n of x[k][i0 + r] * y[k][j0 + s]
template <typename RowX, typename RowY>
__device__ __forceinline__ void ns_outer(const RowX* x, const RowY* y, int n, int i0, int j0, double (&acc)[4][4]) {
#pragma unroll 2
  for (int k = 0; k < n; ++k) {
    double u[4], v[4];
    ns_load4(&x[k][i0], u);
    ns_load4(&y[k][j0], v);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int s = 0; s < 4; ++s) acc[r][s] = fma(u[r], v[s], acc[r][s]);
  }
}

// part[z][chunk] (64 x 64) = the chunk's share of G G^T.
__global__ void __launch_bounds__(kNsThreads) ns_small_gram_kernel(const NsSide n, double* __restrict__ part) {
  __shared__ __align__(16) NsRow32 tile[kNsSmall];  // [l][i]
  pdl_launch_dependents();
  const int i0 = (threadIdx.x / 16) * 4, j0 = (threadIdx.x % 16) * 4;
  double acc[4][4] = {};
  for (int l0 = static_cast<int>(blockIdx.x) * kNsSmall; l0 < n.len; l0 += static_cast<int>(gridDim.x) * kNsSmall) {
    __syncthreads();
    for (int e = threadIdx.x; e < kNsSmall * kNsSmall; e += kNsThreads) {
      const int i = n.i_of(e), l = n.l_of(e);
      tile[l][i] = i < n.side && l0 + l < n.len ? ns_load(n.g, n.f32, n.at(blockIdx.y, i, l0 + l)) : 0.f;
    }
    __syncthreads();
    if (i0 < n.side && j0 < n.side) ns_outer(tile, tile, min(kNsSmall, n.len - l0), i0, j0, acc);
  }
  double* dst = part + (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * kNsSmall * kNsSmall;
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int s = 0; s < 4; ++s) dst[(i0 + r) * kNsSmall + j0 + s] = acc[r][s];
}

constexpr int kNsStepsSmem = 4 * kNsSmall * static_cast<int>(sizeof(NsRow64));
constexpr int kNsApplySmem = kNsSmall * static_cast<int>(sizeof(NsRow64) + sizeof(NsRow32));

// The iteration on S x S matrices, a block a matrix; qt[z] (64 x 64) = Q^T.
// Bound by fp64 issue: 19 products of 64^3 at 64 fmas a clock.
__global__ void __launch_bounds__(kNsThreads)
    ns_small_steps_kernel(const double* part, int chunks, int side, int steps, double a, double b, double c, double eps,
                          double* __restrict__ qt) {
  extern __shared__ __align__(16) uint8_t ns_smem[];
  NsRow64* A = reinterpret_cast<NsRow64*>(ns_smem);
  NsRow64 *P = A + kNsSmall, *Q = P + kNsSmall, *T = Q + kNsSmall;
  pdl_launch_dependents();
  pdl_wait();
  const double* src = part + static_cast<int64_t>(blockIdx.x) * chunks * kNsSmall * kNsSmall;
  for (int e = threadIdx.x; e < kNsSmall * kNsSmall; e += kNsThreads) {
    double s = 0.0;
    for (int k = 0; k < chunks; ++k) s += __ldcg(src + k * kNsSmall * kNsSmall + e);
    A[e / kNsSmall][e % kNsSmall] = s;
  }
  __syncthreads();
  double trace = 0.0;
  for (int i = 0; i < side; ++i) trace += A[i][i];
  const double inv = 1.0 / (sqrt(trace) + eps);
  __syncthreads();
  for (int e = threadIdx.x; e < kNsSmall * kNsSmall; e += kNsThreads) {
    const int i = e / kNsSmall, j = e % kNsSmall;
    A[i][j] = A[i][j] * inv * inv;
    Q[i][j] = i == j && i < side ? inv : 0.0;
  }
  __syncthreads();
  const int nt = (side + 3) / 4;  // 4 x 4 tiles a row
  const bool works = static_cast<int>(threadIdx.x) < nt * nt;
  const int i0 = works ? static_cast<int>(threadIdx.x) / nt * 4 : 0, j0 = works ? static_cast<int>(threadIdx.x) % nt * 4 : 0;
  // dst = f(x^T y); x is A or P, which are symmetric; dst is written after all have read
  auto product = [&](const NsRow64* x, const NsRow64* y, NsRow64* dst, auto f) {
    double acc[4][4] = {};
    if (works) ns_outer(x, y, side, i0, j0, acc);
    __syncthreads();
    if (works) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int s = 0; s < 4; ++s) dst[i0 + r][j0 + s] = f(i0 + r, j0 + s, acc[r][s]);
    }
    __syncthreads();
  };
  auto same = [](int, int, double v) { return v; };
  for (int k = 0; k < steps; ++k) {
    product(A, A, P, [&](int i, int j, double v) { return fma(c, v, fma(b, A[i][j], i == j && i < side ? a : 0.0)); });
    product(P, Q, Q, same);
    if (k + 1 < steps) {
      product(P, A, T, same);
      product(P, T, A, same);
      // the product is symmetric only up to rounding: keep the mean
      double m[4][4];
      if (works) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int s = 0; s < 4; ++s) m[r][s] = 0.5 * (A[i0 + r][j0 + s] + A[j0 + s][i0 + r]);
      }
      __syncthreads();
      if (works) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int s = 0; s < 4; ++s) A[i0 + r][j0 + s] = m[r][s];
      }
      __syncthreads();
    }
  }
  double* dst = qt + static_cast<int64_t>(blockIdx.x) * kNsSmall * kNsSmall;
  for (int e = threadIdx.x; e < kNsSmall * kNsSmall; e += kNsThreads) dst[e] = Q[e % kNsSmall][e / kNsSmall];
}

// out = Q G, 64 places of the longer side a block.
__global__ void __launch_bounds__(kNsThreads)
    ns_small_apply_kernel(const NsSide n, const double* qt, __nv_bfloat16* out) {
  extern __shared__ __align__(16) uint8_t ns_smem[];
  NsRow64* q = reinterpret_cast<NsRow64*>(ns_smem);              // [k][i]
  NsRow32* tile = reinterpret_cast<NsRow32*>(q + kNsSmall);      // [k][l]
  pdl_wait();
  const int64_t z = blockIdx.y;
  const int l0 = static_cast<int>(blockIdx.x) * kNsSmall;
  const double* src = qt + z * kNsSmall * kNsSmall;
  for (int e = threadIdx.x; e < kNsSmall * kNsSmall; e += kNsThreads) {
    q[e / kNsSmall][e % kNsSmall] = __ldcg(src + e);
    const int i = n.i_of(e), l = n.l_of(e);
    tile[i][l] = i < n.side && l0 + l < n.len ? ns_load(n.g, n.f32, n.at(z, i, l0 + l)) : 0.f;
  }
  __syncthreads();
  const int i0 = (threadIdx.x / 16) * 4, j0 = (threadIdx.x % 16) * 4;
  double acc[4][4] = {};
  if (i0 < n.side) ns_outer(q, tile, n.side, i0, j0, acc);
  __syncthreads();  // this block's part of g has been read: out may be g
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int s = 0; s < 4; ++s) tile[i0 + r][j0 + s] = static_cast<float>(acc[r][s]);
  __syncthreads();
  for (int e = threadIdx.x; e < kNsSmall * kNsSmall; e += kNsThreads) {
    const int i = n.i_of(e), l = n.l_of(e);
    if (i < n.side && l0 + l < n.len) out[n.at(z, i, l0 + l)] = __float2bfloat16_rn(tile[i][l]);
  }
}

// ------------------------------------- a side of at most 64, the longer one in shared memory
constexpr int kNsClusterLen = 640;                     // places of the longer side a CTA
constexpr int kNsClusterMax = 8 * kNsClusterLen;
constexpr int kNsMatSmem = kNsSmall * static_cast<int>(sizeof(NsRow32));

__device__ __forceinline__ float4 ld_dsmem4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_dsmem4(uint32_t addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

// acc[r][s] += sum over k < n of x[k][i0 + r] * x[k][j0 + s]
__device__ __forceinline__ void ns_outer32(const NsRow32* x, int n, int i0, int j0, float (&acc)[4][4]) {
#pragma unroll 8
  for (int k = 0; k < n; ++k) {
    const float4 u4 = *reinterpret_cast<const float4*>(&x[k][i0]), v4 = *reinterpret_cast<const float4*>(&x[k][j0]);
    const float u[4] = {u4.x, u4.y, u4.z, u4.w}, v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int s = 0; s < 4; ++s) acc[r][s] = fmaf(u[r], v[s], acc[r][s]);
  }
}

// A cluster a matrix; `per` places of the longer side a CTA, lc >= per a
// multiple of 64.  Bound by shared memory's reads for 4 x 4 sums a thread: 64 x
// 64, 5 steps of three products of 64^3, takes 35 us (17 at 128 fmas a clock);
// in 64 bits on one CTA it took 139.
__global__ void __launch_bounds__(kNsThreads, 2)  // two an SM: 16 matrices of 64 x 2000 need 128 CTAs in clusters of 8
    ns_cluster_kernel(const NsSide n, int per, int lc, int steps, float a, float b, float c, double eps,
                      __nv_bfloat16* out) {
  extern __shared__ __align__(16) uint8_t ns_smem[];
  NsRow32* A = reinterpret_cast<NsRow32*>(ns_smem);
  NsRow32* P = A + kNsSmall;
  NsRow32* X = P + kNsSmall;  // [l][i]
  __shared__ double warps[kNsThreads / 32];
  __shared__ double norm2;
  const int tid = threadIdx.x;
  const uint32_t rank = cluster_ctarank(), ranks = cluster_nctarank();
  const int64_t z = blockIdx.y;
  const int base = static_cast<int>(rank) * per;
  const int nl = max(0, min(per, n.len - base));  // this CTA's places
  double sum = 0.0;
  // A thread's 16 values of a panel are loaded at once, from a clamped place and without a condition: behind one each,
  // they were waited for one by one (64 x 2000: 29 thousand cycles).
  for (int l0 = 0; l0 < lc; l0 += kNsSmall) {
    constexpr int kTurns = kNsSmall * kNsSmall / kNsThreads;
    float v[kTurns];
    auto take = [&](auto load) {
#pragma unroll
      for (int k = 0; k < kTurns; ++k) {
        const int i = n.i_of(tid + k * kNsThreads), l = base + l0 + n.l_of(tid + k * kNsThreads);
        v[k] = load(n.at(z, min(i, n.side - 1), min(l, n.len - 1)));
      }
    };
    if (n.f32)
      take([&](int64_t at) { return __ldg(static_cast<const float*>(n.g) + at); });
    else
      take([&](int64_t at) { return __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(n.g) + at)); });
#pragma unroll
    for (int k = 0; k < kTurns; ++k) {
      const int i = n.i_of(tid + k * kNsThreads), l = l0 + n.l_of(tid + k * kNsThreads);
      if (i >= n.side || l >= nl) v[k] = 0.f;
      X[l][i] = v[k];
      sum += static_cast<double>(v[k]) * static_cast<double>(v[k]);
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if ((tid & 31) == 0) warps[tid >> 5] = sum;
  __syncthreads();
  if (tid == 0) {
    double s = 0.0;
    for (int w = 0; w < kNsThreads / 32; ++w) s += warps[w];
    norm2 = s;
  }
  __syncthreads();
  double total = 0.0;
  if (ranks > 1) {
    cluster_sync();
    for (uint32_t q = 0; q < ranks; ++q) {
      double v;
      asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(cluster_addr(&norm2, q)) : "memory");
      total += v;
    }
  } else {
    total = norm2;
  }
  const double inv = 1.0 / (sqrt(total) + eps);
  for (int e = tid; e < nl * kNsSmall; e += kNsThreads) {
    float* x = &X[e / kNsSmall][e % kNsSmall];
    *x = static_cast<float>(static_cast<double>(*x) * inv);
  }
  __syncthreads();
  const int ty = tid / 16, tx = tid % 16, i0 = ty * 4, j0 = tx * 4;
  const bool works = i0 < n.side && j0 < n.side;
  for (int step = 0; step < steps; ++step) {
    // A = X X^T, summed over the cluster by slices of rows
    {
      NsRow32* dst = ranks > 1 ? P : A;
      float acc[4][4] = {};
      if (works) ns_outer32(X, nl, i0, j0, acc);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *reinterpret_cast<float4*>(&dst[i0 + r][j0]) = make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
    }
    if (ranks > 1) {
      cluster_sync();
      const int rows = kNsSmall / static_cast<int>(ranks);
      for (int e = tid; e < rows * (kNsSmall / 4); e += kNsThreads) {
        const int i = static_cast<int>(rank) * rows + e / (kNsSmall / 4), j = e % (kNsSmall / 4) * 4;
        float4 v[8];
#pragma unroll
        for (uint32_t q = 0; q < 8; ++q)
          if (q < ranks) v[q] = ld_dsmem4(cluster_addr(&P[i][j], q));
        float4 s = v[0];
#pragma unroll
        for (uint32_t q = 1; q < 8; ++q)
          if (q < ranks) {
            s.x += v[q].x; s.y += v[q].y; s.z += v[q].z; s.w += v[q].w;
          }
#pragma unroll
        for (uint32_t q = 0; q < 8; ++q)
          if (q < ranks) st_dsmem4(cluster_addr(&A[i][j], q), s);
      }
      cluster_sync();
    } else {
      __syncthreads();
    }
    // P = a I + b A + c A A
    if (works) {
      float acc[4][4] = {};
      ns_outer32(A, n.side, i0, j0, acc);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int s = 0; s < 4; ++s)
          P[i0 + r][j0 + s] = fmaf(c, acc[r][s], fmaf(b, A[i0 + r][j0 + s], i0 + r == j0 + s ? a : 0.f));
    }
    __syncthreads();
    // X <- P X, 64 places at a time: 4 places by 4 rows a thread
    for (int l0 = 0; l0 < nl; l0 += kNsSmall) {
      float acc[4][4] = {};
      const bool live = l0 + i0 < nl && j0 < n.side;
      if (live) {
#pragma unroll 2
        for (int k = 0; k < n.side; k += 4) {  // X is zero from the side on
          float xv[4][4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float4 v = *reinterpret_cast<const float4*>(&X[l0 + i0 + r][k]);
            xv[r][0] = v.x; xv[r][1] = v.y; xv[r][2] = v.z; xv[r][3] = v.w;
          }
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const float4 p4 = *reinterpret_cast<const float4*>(&P[k + kk][j0]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              acc[r][0] = fmaf(xv[r][kk], p4.x, acc[r][0]);
              acc[r][1] = fmaf(xv[r][kk], p4.y, acc[r][1]);
              acc[r][2] = fmaf(xv[r][kk], p4.z, acc[r][2]);
              acc[r][3] = fmaf(xv[r][kk], p4.w, acc[r][3]);
            }
          }
        }
      }
      __syncthreads();
      if (live) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          *reinterpret_cast<float4*>(&X[l0 + i0 + r][j0]) = make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
      }
    }
    __syncthreads();
  }
  for (int l0 = 0; l0 < nl; l0 += kNsSmall)
    for (int e = tid; e < kNsSmall * kNsSmall; e += kNsThreads) {
      const int i = n.i_of(e), l = l0 + n.l_of(e);
      if (i < n.side && l < nl) out[n.at(z, i, base + l)] = __float2bfloat16_rn(X[l][i]);
    }
  if (ranks > 1) cluster_sync();  // no CTA leaves while another may still read its sums
}

static int run_ns_cluster(const char* nm, const void* g, int f32, int E, int M, int N, int steps, float a, float b,
                          float c, float eps, void* out, cudaStream_t stream) {
  const NsSide n{g, f32, M > N ? 1 : 0, std::min(M, N), std::max(M, N)};
  const int ranks = n.len > 4 * kNsSmall ? 8 : n.len > 2 * kNsSmall ? 4 : n.len > kNsSmall ? 2 : 1;
  const int per = (n.len + ranks - 1) / ranks;
  const int lc = (per + kNsSmall - 1) / kNsSmall * kNsSmall;
  cudaError_t err = cudaFuncSetAttribute(ns_cluster_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         2 * kNsMatSmem + kNsClusterLen * static_cast<int>(sizeof(NsRow32)));
  if (err != cudaSuccess) return cuda_fail(nm, err);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ranks, E, 1);
  cfg.blockDim = dim3(kNsThreads, 1, 1);
  cfg.dynamicSmemBytes = 2 * kNsMatSmem + lc * sizeof(NsRow32);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  err = cudaLaunchKernelEx(&cfg, ns_cluster_kernel, n, per, lc, steps, a, b, c, static_cast<double>(eps),
                           static_cast<__nv_bfloat16*>(out));
  return err == cudaSuccess ? MOE_OK : cuda_fail(nm, err);
}

// ------------------------------------- a side of at most 64, any length: S x S matrices alone
static int ns_small_chunks(int M, int N) { return std::min((std::max(M, N) + kNsSmall - 1) / kNsSmall, kNsSmallChunks); }

static int run_ns_small(const char* nm, const void* g, int f32, int E, int M, int N, int steps, float a, float b,
                        float c, float eps, void* out, uint8_t* ws, cudaStream_t stream) {
  const NsSide n{g, f32, M > N ? 1 : 0, std::min(M, N), std::max(M, N)};
  const int chunks = ns_small_chunks(M, N);
  double* qt = reinterpret_cast<double*>(ws);
  double* part = qt + static_cast<int64_t>(E) * kNsSmall * kNsSmall;
  cudaError_t err = cudaFuncSetAttribute(ns_small_steps_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNsStepsSmem);
  if (err == cudaSuccess)
    err = cudaFuncSetAttribute(ns_small_apply_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNsApplySmem);
  if (err != cudaSuccess) return cuda_fail(nm, err);
  ns_small_gram_kernel<<<dim3(chunks, E), kNsThreads, 0, stream>>>(n, part);
  err = cudaGetLastError();
  if (err != cudaSuccess) return cuda_fail(nm, err);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(E, 1, 1);
  cfg.blockDim = dim3(kNsThreads, 1, 1);
  cfg.dynamicSmemBytes = kNsStepsSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  err = cudaLaunchKernelEx(&cfg, ns_small_steps_kernel, static_cast<const double*>(part), chunks, n.side, steps,
                           static_cast<double>(a), static_cast<double>(b), static_cast<double>(c),
                           static_cast<double>(eps), qt);
  if (err != cudaSuccess) return cuda_fail(nm, err);
  cfg.gridDim = dim3((n.len + kNsSmall - 1) / kNsSmall, E, 1);
  cfg.dynamicSmemBytes = kNsApplySmem;
  err = cudaLaunchKernelEx(&cfg, ns_small_apply_kernel, n, static_cast<const double*>(qt),
                           static_cast<__nv_bfloat16*>(out));
  return err == cudaSuccess ? MOE_OK : cuda_fail(nm, err);
}

// ------------------------------------------------------------- larger sides
struct NsLayout {
  int64_t hi[2], lo[2], gram, poly, diag, part, total;
  int ldx, lds, side, chunks;
};

static NsLayout ns_layout(int E, int M, int N) {
  NsLayout L{};
  if (std::min(M, N) <= kNsSmall) {
    L.total = static_cast<int64_t>(E) * (1 + ns_small_chunks(M, N)) * kNsSmall * kNsSmall * 8;
    return L;
  }
  auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b * b; };
  L.side = std::min(M, N);
  // rows begin on 128 bytes: an operand row of 128 bytes is then one line of L2
  L.ldx = static_cast<int>(up(N, 64));
  L.lds = static_cast<int>(up(L.side, 64));
  L.chunks = static_cast<int>(std::min<int64_t>((static_cast<int64_t>(M) * N + 8 * kNsThreads - 1) / (8 * kNsThreads), kNsChunks));
  const int64_t x = up(static_cast<int64_t>(E) * M * L.ldx * 2, 256), s = up(static_cast<int64_t>(E) * L.side * L.lds * 2, 256);
  int64_t off = 0;
  auto take = [&](int64_t n) {
    const int64_t o = off;
    off += up(n, 256);
    return o;
  };
  for (int i = 0; i < 2; ++i) {
    L.hi[i] = take(x);
    L.lo[i] = take(x);
  }
  L.gram = take(s);
  L.poly = take(s);
  L.diag = take(static_cast<int64_t>(E) * L.side * 4);
  L.part = take(static_cast<int64_t>(E) * L.chunks * 8);
  L.total = off;
  return L;
}

struct NsCall {
  const char* nm;
  int E, M, N, steps;
  float a, b, c;
  uint8_t* ws;
  NsLayout L;
  void* out;
  bool direct;  // the result cannot go through a tensor map: rows not a multiple of 16 bytes
  cudaStream_t stream;
};

template <bool kTall, bool kPair>
static int ns_steps(const NsCall& n) {
  const NsLayout& L = n.L;
  const int S = L.side;
  int rc = MOE_OK;
  auto xmap = [&](CUtensorMap* m, int64_t off, int b0, int b1) {
    if (rc == MOE_OK)
      rc = make_map3(m, n.ws + off, Elem::F16, n.N, n.M, n.E, int64_t(L.ldx) * 2, int64_t(n.M) * L.ldx * 2, b0, b1, 1);
  };
  auto smap = [&](CUtensorMap* m, int64_t off, int b0, int b1) {
    if (rc == MOE_OK)
      rc = make_map3(m, n.ws + off, Elem::F16, S, S, n.E, int64_t(L.lds) * 2, int64_t(S) * L.lds * 2, b0, b1, 1);
  };
  // operands are read in boxes of 64 columns, 128 rows (K-major) or 64 (MN-major); pieces are stored, and read
  // beside an accumulator, in boxes of 32 rows
  CUtensorMap x_k[2], x_mn[2], hi32[2], lo32[2], gram_k, gram32, poly_k, poly32, out32;
  for (int i = 0; i < 2; ++i) {
    xmap(&x_k[i], L.hi[i], kGK, 128);
    xmap(&x_mn[i], L.hi[i], 64, kGK);
    xmap(&hi32[i], L.hi[i], 32, 32);
    xmap(&lo32[i], L.lo[i], 32, 32);
  }
  smap(&gram_k, L.gram, kGK, 128);
  smap(&gram32, L.gram, 32, 32);
  smap(&poly_k, L.poly, kGK, 128);
  smap(&poly32, L.poly, 32, 32);
  out32 = hi32[0];
  if (rc == MOE_OK && !n.direct)
    rc = make_map3(&out32, n.out, Elem::Bf16, n.N, n.M, n.E, int64_t(n.N) * 2, int64_t(n.M) * n.N * 2, 32, 32, 1);
  if (rc != MOE_OK) return rc;

  GemmParams base{};
  if ((rc = status_word(n.nm, &base.status)) != MOE_OK) return rc;
  base.wait_ns = kWaitTimeoutNs;
  base.batches = n.E;
  base.a_rows = 128;
  base.store_rows = 32;
  base.side = S;
  base.diag = reinterpret_cast<float*>(n.ws + L.diag);
  base.tall = kTall ? 1 : 0;
  auto tiles = [&](GemmParams* p, int m, int cols, int k) {
    p->m_total = m;
    p->n_total = cols;
    p->m_tiles = (m + tile_m(kPair) - 1) / tile_m(kPair);
    p->n_tiles = (cols + tile_n(kPair) - 1) / tile_n(kPair);
    p->nk = (k + kGK - 1) / kGK;
    return static_cast<int64_t>(n.E) * p->m_tiles * p->n_tiles;
  };
  for (int i = 0; i < n.steps; ++i) {
    const int cur = i & 1, nxt = cur ^ 1;
    const CUtensorMap& x = kTall ? x_mn[cur] : x_k[cur];  // X^T X: both MN-major; X X^T: both K-major
    GemmParams p = base;
    int64_t units = tiles(&p, S, S, kTall ? n.M : n.N);
    p.alpha = 1.0f / (kNsScale * kNsScale);
    rc = launch_tile_gemm<kTall ? Form::TN : Form::NT, Sched::Batch, Epi::Gram, kPair, false>(
        n.nm, GemmMaps{x, x, gram32, gram32, gram32, gram32}, p, units, true, n.stream);
    if (rc != MOE_OK) return rc;
    p = base;
    units = tiles(&p, S, S, S);
    p.alpha = n.c;
    p.beta = n.b;
    p.use_diag = i >= kNsDiagFrom ? 1 : 0;
    rc = launch_tile_gemm<Form::NT, Sched::Batch, Epi::Poly, kPair, false>(
        n.nm, GemmMaps{gram_k, gram_k, poly32, poly32, gram32, gram32}, p, units, true, n.stream);
    if (rc != MOE_OK) return rc;
    p = base;
    units = tiles(&p, n.M, n.N, S);
    p.alpha = n.a;
    p.beta = 1.0f / kNsScale;
    p.use_diag = i >= kNsDiagFrom ? 1 : 0;
    p.last = i + 1 == n.steps ? 1 : 0;
    p.direct = n.direct ? 1 : 0;
    p.out = static_cast<__nv_bfloat16*>(n.out);
    // X B, both K-major (B is symmetric), or B X
    const GemmMaps u{kTall ? x_k[cur] : poly_k, kTall ? poly_k : x_mn[cur], p.last ? out32 : hi32[nxt], lo32[nxt],
                     hi32[cur], lo32[cur]};
    rc = launch_tile_gemm<kTall ? Form::NT : Form::NN, Sched::Batch, Epi::Update, kPair, false>(n.nm, u, p, units, true,
                                                                                               n.stream);
    if (rc != MOE_OK) return rc;
  }
  return MOE_OK;
}

// The longer side: ns_small_gram_kernel steps over it by up to kNsSmallChunks * kNsSmall places in 32 bits, the others
// by less.
constexpr int kNsLongest = 2147483647 - kNsSmallChunks * kNsSmall + 1;

static bool ns_sizes_ok(int E, int M, int N) {
  if (E < 1 || M < 1 || N < 1 || std::max(M, N) > kNsLongest) return false;
  const int64_t tiles = ((int64_t(M) + 63) / 64) * ((int64_t(N) + 63) / 64);
  return E <= 65535 && tiles * E < (int64_t(1) << 31) && int64_t(M) * N < (int64_t(1) << 40);
}

}  // namespace moe

using namespace moe;

extern "C" int64_t moe_orthogonalize_workspace_bytes(int E, int M, int N) {
  return ns_sizes_ok(E, M, N) ? ns_layout(E, M, N).total : -1;
}

extern "C" int moe_orthogonalize(const void* g, int g_dtype, int E, int M, int N, int steps, float a, float b, float c,
                                 float eps, void* out, void* workspace, int64_t workspace_bytes,
                                 moe_stream_t stream) {
  const char* nm = "moe_orthogonalize";
  if (E < 0 || M < 0 || N < 0 || steps < 1)
    return fail(MOE_ERR_INVALID_ARG, "%s: need E, M, N >= 0 and steps >= 1", nm);
  if (g_dtype != MOE_ROWS_BF16 && g_dtype != MOE_ROWS_FP32) return fail(MOE_ERR_UNSUPPORTED, "%s: g must be bf16 or fp32", nm);
  if (!(eps >= 0.0f)) return fail(MOE_ERR_INVALID_ARG, "%s: eps must be >= 0", nm);
  if (!(std::abs(a) <= 64.0f && std::abs(b) <= 64.0f && std::abs(c) <= 64.0f))
    return fail(MOE_ERR_UNSUPPORTED, "%s: coefficients must be within [-64, 64]", nm);
  if (E == 0 || M == 0 || N == 0) return MOE_OK;
  if (!ns_sizes_ok(E, M, N))
    return fail(MOE_ERR_UNSUPPORTED, "%s: too many tiles or a side above 2^31 - 2048", nm);
  if (!g || !out || !workspace) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", nm);
  const int esize = g_dtype == MOE_ROWS_FP32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(g) % esize || reinterpret_cast<uintptr_t>(out) % 2 ||
      reinterpret_cast<uintptr_t>(workspace) % 256)
    return fail(MOE_ERR_ALIGNMENT, "%s: g and out aligned to their element, the workspace to 256 bytes", nm);
  NsCall n{nm, E, M, N, steps, a, b, c, static_cast<uint8_t*>(workspace), ns_layout(E, M, N), out, false,
           reinterpret_cast<cudaStream_t>(stream)};
  if (workspace_bytes < n.L.total)
    return fail(MOE_ERR_WORKSPACE, "%s: workspace %lld bytes < required %lld", nm, (long long)workspace_bytes,
                (long long)n.L.total);
  n.direct = N % 8 != 0 || reinterpret_cast<uintptr_t>(out) % 16 != 0;

  const int64_t mn = int64_t(M) * N;
  const int f32 = g_dtype == MOE_ROWS_FP32 ? 1 : 0;
  if (std::min(M, N) <= kNsSmall && std::max(M, N) <= kNsClusterMax)
    return run_ns_cluster(nm, g, f32, E, M, N, steps, a, b, c, eps, out, n.stream);
  if (std::min(M, N) <= kNsSmall) return run_ns_small(nm, g, f32, E, M, N, steps, a, b, c, eps, out, n.ws, n.stream);
  if (ns_resident_fits(E, M, N)) return run_ns_resident(nm, g, f32, E, M, N, steps, a, b, c, eps, out, n.ws, n.stream);
  const bool al = reinterpret_cast<uintptr_t>(g) % 16 == 0;
  double* part = reinterpret_cast<double*>(n.ws + n.L.part);
  ns_norm_kernel<<<dim3(n.L.chunks, E), kNsThreads, 0, n.stream>>>(g, f32, mn, al && mn % 8 == 0 ? 1 : 0, part);
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return cuda_fail(nm, err);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const int64_t groups = int64_t(M) * (n.L.ldx / 8);
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>((groups + kNsThreads - 1) / kNsThreads, 1024)), E, 1);
  cfg.blockDim = dim3(kNsThreads, 1, 1);
  cfg.stream = n.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  err = cudaLaunchKernelEx(&cfg, ns_init_kernel, g, f32, M, N, n.L.ldx, al && N % 8 == 0 ? 1 : 0,
                           static_cast<const double*>(part), n.L.chunks, static_cast<double>(eps),
                           reinterpret_cast<__half*>(n.ws + n.L.hi[0]), reinterpret_cast<__half*>(n.ws + n.L.lo[0]));
  if (err != cudaSuccess) return cuda_fail(nm, err);
  // tiles of 256 x 256 on CTA pairs where they fill the SMs, else 128 x 128 for four times as many
  const int64_t pairs = int64_t(E) * ((n.L.side + 255) / 256) * ((n.L.side + 255) / 256);
  const bool pair = pairs >= sm_count() / 2;
  if (M > N) return pair ? ns_steps<true, true>(n) : ns_steps<true, false>(n);
  return pair ? ns_steps<false, true>(n) : ns_steps<false, false>(n);
}
