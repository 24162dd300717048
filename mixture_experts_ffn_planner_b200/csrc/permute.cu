// Token rows in expert order and back, and the gradients of both.
//
// With slot(t, j) the place that the planner gave route t*top_k + j in
// sorted_token_ids (none for a route whose expert is outside [0, E)):
//   permute             rows[slot(t, j)] = x[t]
//   permute_backward    grad_x[t]  = sum over j of grad_rows[slot(t, j)]
//   unpermute           out[t]     = sum over j of w[t, j] * y[slot(t, j)]
//   unpermute_backward  grad_y[slot(t, j)] = w[t, j] * grad_out[t]
//                       grad_w[t, j] = <grad_out[t], y[slot(t, j)]>, 0 without a slot
// so two kernels serve all four: a scatter from a token's row to its slots
// (with the dot products riding along) and a gather from the slots to the
// token's row.  Sums run over j in ascending order in fp32 and are rounded
// once, so results do not depend on the launch.  A dot product is summed in
// fp32 by thread, warp and warps in a fixed order.
//
// Both are bound by HBM.  They are token-major -- the threads of one token
// hold its slots in registers and walk the row in vectors -- so every row is
// read once and written once, and the up to 8 rows of a token are 8
// independent streams per thread, which is what keeps enough bytes in flight.
#include <algorithm>
#include <cuda_bf16.h>
#include <initializer_list>
#include <type_traits>

#include "internal.h"

namespace moe {

// Threads a block.  A gather, and a scatter with dot products, hold many rows'
// vectors a thread (80 and 108 registers): blocks of 128 then fill an SM
// better (8192 tokens, top 6, gathered in rows of 8 KB bf16: 78 us, 88 at 256;
// 3000 tokens in rows of 501 fp32: 18 and 27; 8192 tokens of 8 KB, top 8, with
// dot products: 199 and 217).  A scatter without them is ahead with 256 (8192
// tokens of 8 KB, top 8: 118 and 123 us).
constexpr int kPermThreads = 256;
constexpr int kPermGatherThreads = 128;
constexpr int kPermGradThreads = 128;
constexpr int kPermJ = 8;  // routes handled at once (registers); more routes take another turn

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// VB bytes of a row as one access: 16, 8, 4 or 2.
template <int VB>
struct Raw;
template <>
struct Raw<16> { using type = uint4; };
template <>
struct Raw<8> { using type = uint2; };
template <>
struct Raw<4> { using type = uint32_t; };
template <>
struct Raw<2> { using type = uint16_t; };

template <typename T, int VB>
struct Vec {
  static constexpr int n = VB / static_cast<int>(sizeof(T));
  typename Raw<VB>::type raw;
  __device__ __forceinline__ float get(int i) const { return to_f32<T>(reinterpret_cast<const T*>(&raw)[i]); }
  __device__ __forceinline__ void set(int i, float v) { reinterpret_cast<T*>(&raw)[i] = from_f32<T>(v); }
};

// Counts a row's vectors.  An index or an end of a part may lie beyond the row by up to half of it, or by a turn of the
// block: past 2^31 where a row of nearly that many elements is accessed one by one.  (Unsigned for all widths costs
// the gathers of 8-byte vectors a tenth: 8192 tokens of 1004 bf16, top 8, 33 us, unsigned 37.)
template <typename T, int VB>
using RowIndex = std::conditional_t<VB == sizeof(T), uint32_t, int>;

template <typename T, int VB>
__device__ __forceinline__ Vec<T, VB> load_vec(const T* row, RowIndex<T, VB> v) {
  Vec<T, VB> r;
  r.raw = __ldg(reinterpret_cast<const typename Raw<VB>::type*>(row) + v);
  return r;
}
// The same for what nothing reads again (8192 tokens of 8 KB gathered: 104.5 us, 106.5 without the hint).
template <typename T, int VB>
__device__ __forceinline__ Vec<T, VB> load_vec_once(const T* row, RowIndex<T, VB> v) {
  Vec<T, VB> r;
  r.raw = __ldcs(reinterpret_cast<const typename Raw<VB>::type*>(row) + v);
  return r;
}
template <typename T, int VB>
__device__ __forceinline__ void store_vec(T* row, RowIndex<T, VB> v, const Vec<T, VB>& x) {
  reinterpret_cast<typename Raw<VB>::type*>(row)[v] = x.raw;
}

// Vectors of a row that a thread handles at once, a block's width apart: the
// narrow ones of odd row lengths need several to have as many bytes in flight.
// (Four made no odd length faster, and spilled in bf16: 4000 tokens in rows of 250, 23 us, with two 17.)
constexpr int row_unroll(int vb) { return vb == 16 ? 1 : 2; }

struct ScatterParams {
  const void* token;           // (T, K): x, or grad_out
  const void* rows;            // (capacity, K): y (unpermute_backward), else null
  const int32_t* sorted_ids;   // capacity
  const int32_t* ntpp;
  const int32_t* slots;        // (T, top_k)
  const float* weights;        // (T, top_k), or null
  void* row_out;               // (capacity, K)
  float* grad_w;               // (T, top_k), or null
  int64_t capacity;
  int T, top_k, K, tpt, chunks, pad_blocks, pad_step;
  uint32_t span;
};

// Blocks [0, pad_blocks) write zeros into the padding rows below the padded
// total; the others own threads / tpt tokens each, tpt threads a token, or one
// of `chunks` parts (span vectors) of a token's row.
template <typename T, int VB, bool kGrad>
__global__ void __launch_bounds__(kGrad ? kPermGradThreads : kPermThreads) row_scatter_kernel(const ScatterParams p) {
  constexpr int kThreads = kGrad ? kPermGradThreads : kPermThreads;
  constexpr int kU = row_unroll(VB);
  using V = Vec<T, VB>;
  using Ix = RowIndex<T, VB>;
  const Ix nv = p.K / V::n, tpt = p.tpt;
  const int64_t R = static_cast<int64_t>(p.T) * p.top_k;
  if (static_cast<int>(blockIdx.x) < p.pad_blocks) {
    // one warp looks at pad_step (at most 32) places at a time and clears the rows of those that hold no route
    const int lane = threadIdx.x & 31;
    const int64_t total = min(static_cast<int64_t>(max(__ldg(p.ntpp), 0)), p.capacity);
    const int64_t warps = static_cast<int64_t>(p.pad_blocks) * (kThreads / 32);
    for (int64_t p0 = (static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * p.pad_step;
         p0 < total; p0 += warps * p.pad_step) {
      bool pad = false;
      if (lane < p.pad_step && p0 + lane < total) {
        const int id = __ldg(p.sorted_ids + p0 + lane);
        pad = id < 0 || id >= R;
      }
      V zero;
#pragma unroll
      for (int i = 0; i < V::n; ++i) zero.set(i, 0.f);
      for (uint32_t m = __ballot_sync(0xffffffffu, pad); m; m &= m - 1) {
        T* row = static_cast<T*>(p.row_out) + (p0 + __ffs(static_cast<int>(m)) - 1) * p.K;
        for (Ix v = lane; v < nv; v += 32) store_vec<T, VB>(row, v, zero);
      }
    }
    return;
  }
  __shared__ float part[kThreads / 32][kPermJ];
  const int per = kThreads / p.tpt;
  const int sub = threadIdx.x / p.tpt, tid = threadIdx.x - sub * p.tpt;
  const uint32_t place = blockIdx.x - static_cast<uint32_t>(p.pad_blocks), chunks = static_cast<uint32_t>(p.chunks);
  const int64_t t = static_cast<int64_t>(kGrad ? place : place / chunks) * per + sub;  // a dot product takes the whole row
  const Ix span = static_cast<Ix>(p.span), v_lo = kGrad ? 0 : static_cast<Ix>(place % chunks) * span;
  const Ix v_hi = kGrad ? nv : min(nv, v_lo + span);
  const bool live = t < p.T;
  const T* src = static_cast<const T*>(p.token) + t * p.K;
  for (int j0 = 0; j0 < p.top_k; j0 += kPermJ) {
    int64_t at[kPermJ];
    float w[kPermJ], dot[kPermJ];
#pragma unroll
    for (int j = 0; j < kPermJ; ++j) {
      int s = -1;
      w[j] = 1.f;
      dot[j] = 0.f;
      if (live && j0 + j < p.top_k) {
        s = __ldg(p.slots + t * p.top_k + j0 + j);
        if (kGrad && p.weights) w[j] = __ldg(p.weights + t * p.top_k + j0 + j);
      }
      at[j] = s >= 0 && s < p.capacity ? static_cast<int64_t>(s) * p.K : -1;
    }
    if (live) {
      for (Ix v0 = v_lo + tid; v0 < v_hi; v0 += kU * tpt) {
        V x[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (u == 0 || v0 + u * tpt < v_hi) x[u] = load_vec<T, VB>(src, v0 + u * tpt);
        if (kGrad) {
          V y[kU][kPermJ];
#pragma unroll
          for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int j = 0; j < kPermJ; ++j)
              if (at[j] >= 0 && (u == 0 || v0 + u * tpt < v_hi))
                y[u][j] = load_vec<T, VB>(static_cast<const T*>(p.rows) + at[j], v0 + u * tpt);
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            if (u > 0 && v0 + u * tpt >= v_hi) break;
#pragma unroll
            for (int j = 0; j < kPermJ; ++j) {
              if (at[j] < 0) continue;
              V g;
#pragma unroll
              for (int i = 0; i < V::n; ++i) {
                dot[j] = fmaf(x[u].get(i), y[u][j].get(i), dot[j]);
                g.set(i, w[j] * x[u].get(i));
              }
              store_vec<T, VB>(static_cast<T*>(p.row_out) + at[j], v0 + u * tpt, g);
            }
          }
        } else {
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            if (u > 0 && v0 + u * tpt >= v_hi) break;
#pragma unroll
            for (int j = 0; j < kPermJ; ++j)
              if (at[j] >= 0) store_vec<T, VB>(static_cast<T*>(p.row_out) + at[j], v0 + u * tpt, x[u]);
          }
        }
      }
    }
    if (kGrad) {
      // the token's tpt threads: lanes, then (tpt > 32) warps in order
#pragma unroll
      for (int j = 0; j < kPermJ; ++j)
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], d);
      const int warp = threadIdx.x >> 5;
      __syncthreads();
      if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int j = 0; j < kPermJ; ++j) part[warp][j] = dot[j];
      }
      __syncthreads();
      if (live && tid < kPermJ && j0 + tid < p.top_k) {
        float sum = 0.f;
        for (int i = 0; i < p.tpt / 32; ++i) sum += part[sub * (p.tpt / 32) + i][tid];
        p.grad_w[t * p.top_k + j0 + tid] = sum;
      }
    }
  }
}

struct GatherParams {
  const void* rows;      // (n_rows, K)
  const int32_t* slots;  // (T, top_k)
  const float* weights;  // (T, top_k), or null
  void* out;             // (T, K)
  int64_t n_rows;
  int T, top_k, K, tpt;
  uint32_t span;
};

template <typename T, int VB>
__global__ void __launch_bounds__(kPermGatherThreads, 6) row_gather_kernel(const GatherParams p) {
  using V = Vec<T, VB>;
  using Ix = RowIndex<T, VB>;
  const Ix nv = p.K / V::n, tpt = p.tpt;
  const int per = kPermGatherThreads / p.tpt;
  const int sub = threadIdx.x / p.tpt, tid = threadIdx.x - sub * p.tpt;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * per + sub;
  if (t >= p.T) return;
  const Ix span = static_cast<Ix>(p.span), v_lo = static_cast<Ix>(blockIdx.y) * span, v_hi = min(nv, v_lo + span);
  const T* rows = static_cast<const T*>(p.rows);
  T* out = static_cast<T*>(p.out) + t * p.K;
  int64_t at[kPermJ];
  float w[kPermJ];
  auto slots_of = [&](int j0) {
#pragma unroll
    for (int j = 0; j < kPermJ; ++j) {
      int s = -1;
      w[j] = 1.f;
      if (j0 + j < p.top_k) {
        s = __ldg(p.slots + t * p.top_k + j0 + j);
        if (p.weights) w[j] = __ldg(p.weights + t * p.top_k + j0 + j);
      }
      at[j] = s >= 0 && s < p.n_rows ? static_cast<int64_t>(s) * p.K : -1;
    }
  };
  slots_of(0);
  constexpr int kU = row_unroll(VB);
  for (Ix v0 = v_lo + tid; v0 < v_hi; v0 += kU * tpt) {
    float acc[kU][V::n];
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int i = 0; i < V::n; ++i) acc[u][i] = 0.f;
    for (int j0 = 0; j0 < p.top_k; j0 += kPermJ) {
      if (p.top_k > kPermJ) slots_of(j0);
      V y[kU][kPermJ];
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int j = 0; j < kPermJ; ++j)
          if (at[j] >= 0 && (u == 0 || v0 + u * tpt < v_hi)) y[u][j] = load_vec_once<T, VB>(rows + at[j], v0 + u * tpt);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (u > 0 && v0 + u * tpt >= v_hi) break;
#pragma unroll
        for (int j = 0; j < kPermJ; ++j) {
          if (at[j] < 0) continue;
#pragma unroll
          for (int i = 0; i < V::n; ++i) acc[u][i] = fmaf(w[j], y[u][j].get(i), acc[u][i]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (u > 0 && v0 + u * tpt >= v_hi) break;
      V o;
#pragma unroll
      for (int i = 0; i < V::n; ++i) o.set(i, acc[u][i]);
      store_vec<T, VB>(out, v0 + u * tpt, o);
    }
  }
}

__global__ void __launch_bounds__(256)
    route_slots_kernel(const int32_t* __restrict__ sorted_ids, const int32_t* __restrict__ ntpp, int64_t capacity,
                       int64_t R, int32_t* __restrict__ slots) {
  const int64_t total = min(static_cast<int64_t>(max(__ldg(ntpp), 0)), capacity);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int id = __ldg(sorted_ids + i);
    if (id >= 0 && id < R) slots[id] = static_cast<int32_t>(i);
  }
}

// Largest access (bytes) that divides a row and the alignment of every pointer.
static int vector_bytes(int64_t row_bytes, int esize, std::initializer_list<const void*> ptrs) {
  uintptr_t bits = static_cast<uintptr_t>(row_bytes);
  for (const void* p : ptrs) bits |= reinterpret_cast<uintptr_t>(p);
  for (int vb = 16; vb > esize; vb >>= 1)
    if (bits % vb == 0) return vb;
  return esize;
}

// Threads per token: a power of two between a warp and the block, enough for
// one vector each; a short row then shares its block with other tokens.
static int threads_per_token(int64_t nv, int threads) {
  int tpt = 32;
  while (tpt < threads && tpt < nv) tpt <<= 1;
  return tpt;
}

// Parts that a row is split into, of `span` vectors each: while blocks are
// fewer than 4 an SM, so that a thread has fewer vectors to wait for in turn
// (64 tokens of 16 KB, top 8, gathered: 12 -> 8 us).
static int row_chunks(int64_t blocks, int64_t nv, int threads, int tpt, uint32_t* span) {
  int64_t n = 1;
  if (tpt == threads)
    while (blocks * n < static_cast<int64_t>(std::max(1, sm_count())) * 4 && n * tpt < nv) n <<= 1;
  const int64_t s = ((nv + n - 1) / n + tpt - 1) / tpt * tpt;
  *span = static_cast<uint32_t>(s);
  return static_cast<int>((nv + s - 1) / s);
}

// Calls f(type tag, integral constant of the access width).
template <typename F>
static cudaError_t by_access(int dtype, int vb, F f) {
  if (dtype == MOE_ROWS_BF16) {
    switch (vb) {
      case 16: return f(__nv_bfloat16{}, std::integral_constant<int, 16>{});
      case 8: return f(__nv_bfloat16{}, std::integral_constant<int, 8>{});
      case 4: return f(__nv_bfloat16{}, std::integral_constant<int, 4>{});
      default: return f(__nv_bfloat16{}, std::integral_constant<int, 2>{});
    }
  }
  switch (vb) {
    case 16: return f(float{}, std::integral_constant<int, 16>{});
    case 8: return f(float{}, std::integral_constant<int, 8>{});
    default: return f(float{}, std::integral_constant<int, 4>{});
  }
}

static int check_rows(const char* nm, int dtype, int T, int top_k, int K, int64_t capacity) {
  if (T < 0 || top_k < 1 || K < 1 || capacity < 0)
    return fail(MOE_ERR_INVALID_ARG, "%s: need T >= 0, top_k >= 1, K >= 1 and capacity >= 0", nm);
  if (dtype != MOE_ROWS_BF16 && dtype != MOE_ROWS_FP32)
    return fail(MOE_ERR_UNSUPPORTED, "%s: rows must be bf16 or fp32", nm);
  if (static_cast<int64_t>(T) * top_k >= (int64_t(1) << 31) || capacity >= (int64_t(1) << 31))
    return fail(MOE_ERR_UNSUPPORTED, "%s: T * top_k and capacity must be < 2^31", nm);
  return MOE_OK;
}

static bool misaligned(std::initializer_list<const void*> ptrs, int esize) {
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) % esize) return true;
  return false;
}

static int run_scatter(const char* nm, ScatterParams p, int dtype, bool grad, cudaStream_t s) {
  const int esize = dtype == MOE_ROWS_BF16 ? 2 : 4;
  if (misaligned({p.token, p.rows, p.row_out}, esize) ||
      misaligned({p.sorted_ids, p.ntpp, p.slots, p.weights, p.grad_w}, 4))
    return fail(MOE_ERR_ALIGNMENT, "%s: pointers must be aligned to their element", nm);
  const int vb = vector_bytes(static_cast<int64_t>(p.K) * esize, esize, {p.token, p.rows, p.row_out});
  const int threads = grad ? kPermGradThreads : kPermThreads;
  const int64_t nv = static_cast<int64_t>(p.K) * esize / vb;
  p.tpt = threads_per_token(nv, threads);
  const int per = threads / p.tpt;
  int64_t token_blocks = (static_cast<int64_t>(p.T) + per - 1) / per;
  p.chunks = 1;
  if (!grad) {
    p.chunks = row_chunks(token_blocks, nv, threads, p.tpt, &p.span);
    token_blocks *= p.chunks;
  }
  // The padding goes over all SMs, one place a warp while they last: with 32
  // places a warp always, a call of 8 tokens (960 padding rows of 8 KB) took
  // 30 us on 8 blocks.
  const int block_warps = threads / 32;
  const int64_t pad_warps = static_cast<int64_t>(std::max(1, sm_count())) * 4 * block_warps;
  p.pad_step = static_cast<int>(std::min<int64_t>(std::max<int64_t>((p.capacity + pad_warps - 1) / pad_warps, 1), 32));
  const int64_t pad_warps_used = std::min<int64_t>((p.capacity + p.pad_step - 1) / p.pad_step, pad_warps);
  p.pad_blocks = static_cast<int>((pad_warps_used + block_warps - 1) / block_warps);
  const int64_t blocks = token_blocks + p.pad_blocks;
  if (blocks == 0) return MOE_OK;
  const cudaError_t err = by_access(dtype, vb, [&](auto tag, auto width) {
    using T = decltype(tag);
    if (grad)
      row_scatter_kernel<T, decltype(width)::value, true><<<static_cast<unsigned>(blocks), kPermGradThreads, 0, s>>>(p);
    else
      row_scatter_kernel<T, decltype(width)::value, false><<<static_cast<unsigned>(blocks), kPermThreads, 0, s>>>(p);
    return cudaGetLastError();
  });
  return err == cudaSuccess ? MOE_OK : cuda_fail(nm, err);
}

static int run_gather(const char* nm, GatherParams p, int dtype, cudaStream_t s) {
  const int esize = dtype == MOE_ROWS_BF16 ? 2 : 4;
  if (misaligned({p.rows, p.out}, esize) || misaligned({p.slots, p.weights}, 4))
    return fail(MOE_ERR_ALIGNMENT, "%s: pointers must be aligned to their element", nm);
  const int vb = vector_bytes(static_cast<int64_t>(p.K) * esize, esize, {p.rows, p.out});
  const int64_t nv = static_cast<int64_t>(p.K) * esize / vb;
  p.tpt = threads_per_token(nv, kPermGatherThreads);
  const int per = kPermGatherThreads / p.tpt;
  const int64_t blocks = (static_cast<int64_t>(p.T) + per - 1) / per;
  const dim3 grid(static_cast<unsigned>(blocks), row_chunks(blocks, nv, kPermGatherThreads, p.tpt, &p.span));
  const cudaError_t err = by_access(dtype, vb, [&](auto tag, auto width) {
    row_gather_kernel<decltype(tag), decltype(width)::value><<<grid, kPermGatherThreads, 0, s>>>(p);
    return cudaGetLastError();
  });
  return err == cudaSuccess ? MOE_OK : cuda_fail(nm, err);
}

}  // namespace moe

using namespace moe;

extern "C" int moe_route_slots(const int32_t* sorted_token_ids, const int32_t* num_tokens_post_padded,
                               int64_t capacity, int T, int top_k, int32_t* slots, moe_stream_t stream) {
  const char* nm = "moe_route_slots";
  if (int rc = check_rows(nm, MOE_ROWS_BF16, T, top_k, 1, capacity)) return rc;
  if (T == 0) return MOE_OK;
  if (!slots || !num_tokens_post_padded || (capacity > 0 && !sorted_token_ids))
    return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", nm);
  if (misaligned({sorted_token_ids, num_tokens_post_padded, slots}, 4))
    return fail(MOE_ERR_ALIGNMENT, "%s: pointers must be aligned to their element", nm);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int64_t R = static_cast<int64_t>(T) * top_k;
  const cudaError_t err = cudaMemsetAsync(slots, 0xFF, static_cast<size_t>(R) * sizeof(int32_t), s);
  if (err != cudaSuccess) return cuda_fail(nm, err);
  if (capacity > 0) {
    const int64_t blocks = std::min<int64_t>((capacity + 255) / 256, static_cast<int64_t>(std::max(1, sm_count())) * 8);
    route_slots_kernel<<<static_cast<unsigned>(blocks), 256, 0, s>>>(sorted_token_ids, num_tokens_post_padded, capacity,
                                                                    R, slots);
  }
  const cudaError_t lerr = cudaGetLastError();
  return lerr == cudaSuccess ? MOE_OK : cuda_fail(nm, lerr);
}

extern "C" int moe_permute(const void* x, int rows_dtype, const int32_t* sorted_token_ids,
                           const int32_t* num_tokens_post_padded, const int32_t* slots, int64_t capacity, int T,
                           int top_k, int K, void* rows, moe_stream_t stream) {
  const char* nm = "moe_permute";
  if (int rc = check_rows(nm, rows_dtype, T, top_k, K, capacity)) return rc;
  if (T == 0 && capacity == 0) return MOE_OK;
  if ((T > 0 && (!x || !slots)) || (capacity > 0 && (!sorted_token_ids || !rows)) || !num_tokens_post_padded)
    return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", nm);
  ScatterParams p{};
  p.token = x;
  p.sorted_ids = sorted_token_ids;
  p.ntpp = num_tokens_post_padded;
  p.slots = slots;
  p.row_out = rows;
  p.capacity = capacity;
  p.T = T; p.top_k = top_k; p.K = K;
  return run_scatter(nm, p, rows_dtype, false, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int moe_permute_backward(const void* grad_rows, int rows_dtype, const int32_t* slots, int64_t capacity,
                                    int T, int top_k, int K, void* grad_x, moe_stream_t stream) {
  const char* nm = "moe_permute_backward";
  if (int rc = check_rows(nm, rows_dtype, T, top_k, K, capacity)) return rc;
  if (T == 0) return MOE_OK;
  if (!slots || !grad_x || (capacity > 0 && !grad_rows)) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", nm);
  GatherParams p{};
  p.rows = grad_rows;
  p.slots = slots;
  p.out = grad_x;
  p.n_rows = capacity;
  p.T = T; p.top_k = top_k; p.K = K;
  return run_gather(nm, p, rows_dtype, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int moe_unpermute(const void* y, int rows_dtype, const int32_t* slots, const float* topk_weights,
                             int64_t capacity, int T, int top_k, int K, void* out, moe_stream_t stream) {
  const char* nm = "moe_unpermute";
  if (int rc = check_rows(nm, rows_dtype, T, top_k, K, capacity)) return rc;
  if (T == 0) return MOE_OK;
  if (!slots || !topk_weights || !out || (capacity > 0 && !y)) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", nm);
  GatherParams p{};
  p.rows = y;
  p.slots = slots;
  p.weights = topk_weights;
  p.out = out;
  p.n_rows = capacity;
  p.T = T; p.top_k = top_k; p.K = K;
  return run_gather(nm, p, rows_dtype, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int moe_unpermute_backward(const void* grad_out, const void* y, int rows_dtype,
                                      const int32_t* sorted_token_ids, const int32_t* num_tokens_post_padded,
                                      const int32_t* slots, const float* topk_weights, int64_t capacity, int T,
                                      int top_k, int K, void* grad_y, float* grad_weights, moe_stream_t stream) {
  const char* nm = "moe_unpermute_backward";
  if (int rc = check_rows(nm, rows_dtype, T, top_k, K, capacity)) return rc;
  if (T == 0 && capacity == 0) return MOE_OK;
  if ((T > 0 && (!grad_out || !slots || !topk_weights || !grad_weights)) ||
      (capacity > 0 && (!sorted_token_ids || !y || !grad_y)) || !num_tokens_post_padded)
    return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", nm);
  ScatterParams p{};
  p.token = grad_out;
  p.rows = y;
  p.sorted_ids = sorted_token_ids;
  p.ntpp = num_tokens_post_padded;
  p.slots = slots;
  p.weights = topk_weights;
  p.row_out = grad_y;
  p.grad_w = grad_weights;
  p.capacity = capacity;
  p.T = T; p.top_k = top_k; p.K = K;
  return run_scatter(nm, p, rows_dtype, true, reinterpret_cast<cudaStream_t>(stream));
}
