// A persistent tcgen05 product of 16-bit operands, tile by tile, for the
// training operators: D (128 x TN, fp32 in TMEM) = A . B over a contraction
// cut into chunks of 64, in the three forms that a layer's forward pass and
// its two gradients need,
//   NT   D[i][j] = sum_k A[i][k] B[j][k]    both operands K-major
//   NN   D[i][j] = sum_k A[i][k] B[k][j]    B is MN-major
//   TN   D[i][j] = sum_k A[k][i] B[k][j]    both are MN-major
// The tensor cores read either layout from shared memory (a bit each in the
// instruction descriptor), so no operand is ever transposed in memory.
//
// One CTA per SM walks the tiles.  Warp 0 copies operand chunks by TMA into a
// ring of stages, warp 1 issues the MMAs (one lane), warps 2-9 take a finished
// accumulator out of TMEM (two of them alternate, so the epilogue of a tile
// runs beside the next tile's MMAs), apply the epilogue and store it by TMA
// from a swizzled staging buffer of 4 KB a warp.  Every wait is bounded.
//
// What a tile is (Sched):
//   Blocks   a planner block of rows by TN columns of that block's expert;
//   Experts  128 x TN of one expert's weight gradient, contracted over the
//            expert's rows (a run of planner blocks; the rows behind the last
//            routed one are cleared in shared memory, whatever they hold);
//   Batch    128 x TN of one matrix of a batch.
#pragma once

#include <atomic>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"

namespace moe {

enum class Form { NT, NN, TN };
enum class Sched { Blocks, Experts, Batch };
enum class Epi {
  Rows,        // bf16 rows of a block
  GateUp,      // h = [gate | up] and silu(gate) * up, bf16
  SwigluGrad,  // D is the gradient of act: bf16 gradients of gate and up
  Weights,     // a weight gradient, bf16 or fp32, the latter optionally added to what is there
  Gram,        // alpha * D, fp16
  Poly,        // b * C + c * D, fp16, optionally with its diagonal taken out into fp32
  Update       // coefficient * (hi + lo / 2048) + D: the next iterate's hi and lo, or the result in bf16
};

constexpr int kGM = 128;
constexpr int kGK = 64;
constexpr int kGRow = 128;  // bytes of an operand row in a stage
constexpr int kGEpiWarps = 8;
constexpr int kGThreads = 32 * (2 + kGEpiWarps);
constexpr int kGStaging = 4096;  // bytes a warp
constexpr int kGSmemLimit = 232448;
constexpr float kLoScale = 2048.0f;  // lo = fp16(2048 * (value - hi)): 11 more bits

template <int TN>
struct GemmShape {
  static constexpr int a_bytes = kGM * kGRow, b_bytes = TN * kGRow;
  static constexpr int stage = a_bytes + b_bytes;
  static constexpr int stages = TN == 256 ? 4 : 6;
  static constexpr int staging = stages * stage;  // offset
  static constexpr int ctrl = staging + kGEpiWarps * kGStaging;
  static constexpr int smem = 1024 + ctrl + 256;
  static_assert(smem <= kGSmemLimit, "shared memory");
};

struct GemmParams {
  // planner (Blocks, Experts)
  const int32_t* sorted_ids;
  const int32_t* expert_ids;
  const int32_t* ntpp;
  int bm, max_blocks, E;
  // tiles
  int m_tiles, n_tiles, batches;
  int m_total, n_total;  // rows (Experts, Batch) and columns of D
  int nk;                // chunks of the contraction (Blocks, Batch)
  int a_rows;            // rows of A's box (K-major A)
  int store_rows;        // rows of the store boxes
  // SwigluGrad
  const __nv_bfloat16* h;
  // Weights
  int out_f32, accumulate;
  // Gram, Poly, Update (read past L1: the launches are chained and reuse buffers)
  float alpha, beta;
  int use_diag, tall, last, direct;
  float* diag;           // (batches, side)
  int side;
  const __half* c0;      // Poly: the Gram matrix; Update: hi
  const __half* c1;      // Update: lo
  int64_t ldc, zc;       // row and matrix strides of c0 and c1, elements
  __nv_bfloat16* out;    // Update, last, direct: (batches, m_total, n_total)
  int* status;
  unsigned long long wait_ns;
};

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_b16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack_b16(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 unpack_f16(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

struct Tile {
  int z, m0, n0;
  int nk;      // chunks; 0: a weight gradient without rows; < 0: nothing to do
  int p0;      // Experts: first row of the contraction
  int rows;    // Experts: its routed rows
};

// First of the n ascending ids that is >= e (warp-collective; 32 probes a round).
__device__ __forceinline__ int warp_lower_bound(const int32_t* ids, int n, int e, int lane) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const int below = __popc(__ballot_sync(0xffffffffu, lane * step < hi - lo && __ldg(ids + min(i, n - 1)) < e));
    if (below == 0) break;
    hi = min(hi, lo + below * step);
    lo += (below - 1) * step + 1;
  }
  return lo;
}

// The tiles of one role, in the order that every role walks them.
template <Sched kSched, Epi kEpi, int TN>
struct Walk {
  const GemmParams& p;
  const int lane;
  int blocks, units;
  int z_seen = -1, seg_lo = 0, seg_rows = 0;

  __device__ __forceinline__ Walk(const GemmParams& p_) : p(p_), lane(static_cast<int>(lane_id())) {
    blocks = 0;
    if (kSched != Sched::Batch) {
      const int n = __ldg(p.ntpp) / p.bm;
      blocks = n < 0 ? 0 : min(n, p.max_blocks);
    }
    units = kSched == Sched::Blocks ? blocks * p.n_tiles : p.batches * p.m_tiles * p.n_tiles;
  }

  __device__ __forceinline__ Tile at(int u) {
    Tile t{};
    constexpr int kCols = kEpi == Epi::GateUp ? TN / 2 : TN;
    if (kSched == Sched::Blocks) {
      const int b = u / p.n_tiles;
      t.z = __ldg(p.expert_ids + b);
      t.m0 = b * p.bm;
      t.n0 = (u - b * p.n_tiles) * kCols;
      t.nk = t.z >= 0 && t.z < p.E ? p.nk : -1;
      return t;
    }
    const int per = p.m_tiles * p.n_tiles;
    t.z = u / per;
    const int r = u - t.z * per, mi = r / p.n_tiles;
    t.m0 = mi * kGM;
    t.n0 = (r - mi * p.n_tiles) * kCols;
    t.nk = p.nk;
    if (kSched == Sched::Experts) {
      if (t.z != z_seen) {  // warp-uniform
        z_seen = t.z;
        seg_lo = warp_lower_bound(p.expert_ids, blocks, t.z, lane);
        const int n = warp_lower_bound(p.expert_ids + seg_lo, blocks - seg_lo, t.z + 1, lane);
        seg_rows = 0;
        if (n > 0) {  // whole blocks, and the routed rows that the last one begins with
          const int64_t at = static_cast<int64_t>(seg_lo + n - 1) * p.bm;
          int last = 0;
          for (int q = 0; q < p.bm; q += 32) {
            bool v = false;
            if (q + lane < p.bm) {
              const int id = __ldg(p.sorted_ids + at + q + lane);
              v = id >= 0;
            }
            last += __popc(__ballot_sync(0xffffffffu, v));
          }
          seg_rows = (n - 1) * p.bm + last;
        }
      }
      t.p0 = seg_lo * p.bm;
      t.rows = seg_rows;
      t.nk = (seg_rows + kGK - 1) / kGK;
    }
    return t;
  }
};

template <Form kForm, Sched kSched, Epi kEpi, int TN, bool kBf16>
__global__ void __launch_bounds__(kGThreads, 1)
    tile_gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                     const __grid_constant__ CUtensorMap tm_d, const __grid_constant__ CUtensorMap tm_d2,
                     const __grid_constant__ GemmParams p) {
  using S = GemmShape<TN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::ctrl);
  uint64_t* empty = full + S::stages;
  uint64_t* acc_full = empty + S::stages;
  uint64_t* acc_empty = acc_full + 2;
  uint32_t* tmem_base_sm = reinterpret_cast<uint32_t*>(acc_empty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base_sm + 1);
  constexpr uint32_t kTmemCols = 2 * TN;
  constexpr bool kAMn = kForm == Form::TN, kBMn = kForm != Form::NT;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], kGEpiWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tm_a);
    prefetch_tmap(&tm_b);
    prefetch_tmap(&tm_d);
  }
  if (warp == 1) {
    tmem_alloc(tmem_base_sm, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_base_sm;
  pdl_wait();  // what a chained launch before this one wrote is read below
  Walk<kSched, kEpi, TN> walk(p);

  if (warp == 0) {
    // ------------------------------------------------ TMA producer
    const uint64_t pol = policy_evict_normal();
    const uint32_t tx = static_cast<uint32_t>((kAMn ? kGM : p.a_rows) * kGRow + S::b_bytes);
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < walk.units && ok; u += gridDim.x) {
      const Tile t = walk.at(u);
      const int za = kSched == Sched::Batch ? t.z : 0;
      const int zb = kSched == Sched::Experts ? 0 : t.z;
      for (int kc = 0; kc < t.nk; ++kc) {
        if (lane == 0) {
          ok = mbar_wait(&empty[s], ph ^ 1u, abort_flag, p.status, p.wait_ns);
          if (ok) {
            uint8_t* a = smem + s * S::stage;
            uint8_t* b = a + S::a_bytes;
            const int k0 = t.p0 + kc * kGK;
            mbar_arrive_expect_tx(&full[s], tx);
            if (kAMn) {
#pragma unroll
              for (int i = 0; i < kGM / 64; ++i)
                tma_load_3d(a + i * 64 * kGRow, &tm_a, &full[s], t.m0 + 64 * i, k0, za, pol);
            } else {
              tma_load_3d(a, &tm_a, &full[s], k0, t.m0, za, pol);
            }
            if (kBMn) {
#pragma unroll
              for (int i = 0; i < TN / 64; ++i)
                tma_load_3d(b + i * 64 * kGRow, &tm_b, &full[s], t.n0 + 64 * i, k0, zb, pol);
            } else if (kEpi == Epi::GateUp) {
              tma_load_3d(b, &tm_b, &full[s], k0, t.n0, 2 * zb, pol);
              tma_load_3d(b + S::b_bytes / 2, &tm_b, &full[s], k0, t.n0, 2 * zb + 1, pol);
            } else {
              tma_load_3d(b, &tm_b, &full[s], k0, t.n0, zb, pol);
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (++s == S::stages) { s = 0; ph ^= 1u; }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer
    constexpr uint32_t kIdesc = idesc_f16(kGM, TN, kBf16, kAMn, kBMn);
    int s = 0, acc_it = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < walk.units && ok; u += gridDim.x) {
      const Tile t = walk.at(u);
      if (t.nk <= 0) continue;
      const int buf = acc_it & 1;
      if (lane == 0)
        ok = mbar_wait(&acc_empty[buf], ((acc_it >> 1) & 1) ^ 1u, abort_flag, p.status, p.wait_ns);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tbase + static_cast<uint32_t>(buf) * TN;
      for (int kc = 0; kc < t.nk; ++kc) {
        uint8_t* a = smem + s * S::stage;
        uint8_t* b = a + S::a_bytes;
        if (lane == 0) ok = mbar_wait(&full[s], ph, abort_flag, p.status, p.wait_ns);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        int kk_end = kGK / 16;
        if (kSched == Sched::Experts) {
          // the last chunk may reach past the expert's routed rows: what
          // padding or another expert left there becomes zeros (a product
          // with zero would keep a NaN), and whole steps of it are left out
          const int rem = t.rows - kc * kGK;
          if (rem < kGK) {
            kk_end = (rem + 15) / 16;
            __syncwarp();
            const int gap = kk_end * 16 - rem;  // < 16 rows
            constexpr int kBoxes = kGM / 64 + TN / 64;
            for (int i = lane; i < kBoxes * gap * 8; i += 32) {
              const int box = i / (gap * 8), r = i - box * (gap * 8);
              *reinterpret_cast<uint4*>(a + box * 64 * kGRow + (rem + r / 8) * kGRow + (r & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
        }
        if (lane == 0) {
          tc_fence_after();
          const uint64_t ad = kAMn ? sdesc_sw128_mn(smem_u32(a), 64 * kGRow) : sdesc_sw128(smem_u32(a));
          const uint64_t bd = kBMn ? sdesc_sw128_mn(smem_u32(b), 64 * kGRow) : sdesc_sw128(smem_u32(b));
#pragma unroll
          for (int kk = 0; kk < kGK / 16; ++kk) {
            if (kSched == Sched::Experts && kk >= kk_end) break;
            // 16 contraction indices: 32 bytes of a K-major row, 16 rows of an MN-major one
            mma_f16(d, ad + (kAMn ? 128u : 2u) * kk, bd + (kBMn ? 128u : 2u) * kk, kIdesc, (kc | kk) != 0);
          }
          tc_commit(&empty[s]);
        }
        __syncwarp();
        if (++s == S::stages) { s = 0; ph ^= 1u; }
      }
      if (ok && lane == 0) tc_commit(&acc_full[buf]);
      ++acc_it;
    }
  } else {
    // ------------------------------------------------ epilogue
    // Warp w reads TMEM lanes 32 (w % 4) .. + 31, a row a thread, and half of
    // the tile's columns.
    const int q = warp & 3, hf = (warp - 2) >> 2;
    const int r = 32 * q + lane;
    const uint32_t stg = smem_u32(smem + S::staging + (warp - 2) * kGStaging);
    // 16 bytes of this thread's row of a staging tile, swizzled as its tensor
    // map says: 128-byte rows (64 16-bit columns), or 64-byte rows (32 columns)
    auto put128 = [&](int i, uint4 v) {
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stg + lane * 128 + ((i ^ (lane & 7)) << 4)),
                   "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                   : "memory");
    };
    auto put64 = [&](int tile, int i, uint4 v) {
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stg + tile * 2048 + lane * 64 +
                                                                  ((i ^ ((lane >> 1) & 3)) << 4)),
                   "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                   : "memory");
    };
    auto staging_free = [&] {
      if (lane == 0) bulk_wait_read();
      __syncwarp();
    };
    auto staged = [&] {
      fence_proxy_async_smem();
      __syncwarp();
    };
    // rows of this warp's 32 that are stored: those of the block, or of the matrix
    auto store = [&](const CUtensorMap* map, int tile_off, int row_bytes, int m0, int limit, int c0, int c1_or_row,
                     int z, bool row_last, bool add) {
      if (lane == 0) {
        for (int i = 0; i < 32; i += p.store_rows) {
          if (32 * q + i >= limit) break;
          const uint32_t src = stg + tile_off + i * row_bytes;
          const int row = m0 + 32 * q + i;
          if (add)
            tma_add_3d(map, src, c0, row, z);
          else if (row_last)
            tma_store_3d(map, src, c0, c1_or_row, row);
          else
            tma_store_3d(map, src, c0, row, z);
        }
        bulk_commit();
      }
    };
    int acc_it = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < walk.units && ok; u += gridDim.x) {
      const Tile t = walk.at(u);
      if (t.nk < 0 || (t.nk == 0 && p.accumulate)) continue;
      // rows of the tile that belong to the output, and whether this thread's carries a value
      const int limit = kSched == Sched::Blocks ? p.bm : min(kGM, p.m_total - t.m0);
      bool mine = r < limit;
      if (kSched == Sched::Blocks && mine) {
        const int id = __ldg(p.sorted_ids + static_cast<int64_t>(t.m0) + r);
        mine = id >= 0;
      }
      const int half = p.n_total;  // GateUp, SwigluGrad: columns of gate (and of up)
      uint4 hg[4], hu[4];
      auto load_h = [&](int col) {  // 32 columns of gate and up of this thread's row
        const __nv_bfloat16* row = p.h + (static_cast<int64_t>(t.m0) + r) * 2 * half + col;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          hg[i] = hu[i] = make_uint4(0, 0, 0, 0);
          if (mine && col + 8 * i < half) {
            hg[i] = __ldg(reinterpret_cast<const uint4*>(row) + i);
            hu[i] = __ldg(reinterpret_cast<const uint4*>(row + half) + i);
          }
        }
      };
      if (kEpi == Epi::SwigluGrad) load_h(t.n0 + hf * (TN / 2));
      const int buf = acc_it & 1;
      if (t.nk > 0) {
        ok = mbar_wait(&acc_full[buf], (acc_it >> 1) & 1, abort_flag, p.status, p.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
      }
      const uint32_t tacc = tbase + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(buf) * TN;
      if (32 * q < limit) {  // warp-uniform
        if (kEpi == Epi::GateUp) {
          const int col = t.n0 + 64 * hf;
          if (col < half) {
#pragma unroll 1
            for (int part = 0; part < 2; ++part) {  // gate, then up, into h
              staging_free();
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                uint32_t v[32];
                tmem_ld32(tacc + part * (TN / 2) + 64 * hf + 32 * c, v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  uint32_t w[4];
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                    w[j] = mine ? pack_b16(__uint_as_float(v[8 * i + 2 * j]), __uint_as_float(v[8 * i + 2 * j + 1])) : 0u;
                  put128(4 * c + i, make_uint4(w[0], w[1], w[2], w[3]));
                }
              }
              staged();
              store(&tm_d, 0, 128, t.m0, limit, col, part, 0, true, false);
            }
            staging_free();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t g[32], up[32];
              tmem_ld32(tacc + 64 * hf + 32 * c, g);
              tmem_ld32(tacc + TN / 2 + 64 * hf + 32 * c, up);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const int e = 8 * i + 2 * j;
                  w[j] = mine ? pack_b16(silu_f32(__uint_as_float(g[e])) * __uint_as_float(up[e]),
                                         silu_f32(__uint_as_float(g[e + 1])) * __uint_as_float(up[e + 1]))
                              : 0u;
                }
                put128(4 * c + i, make_uint4(w[0], w[1], w[2], w[3]));
              }
            }
            staged();
            store(&tm_d2, 0, 128, t.m0, limit, col, 0, 0, false, false);
          }
        } else if (kEpi == Epi::SwigluGrad) {
          // act = gate s(gate) up, s the sigmoid: d act / d gate = up s (1 + gate (1 - s)), d act / d up = gate s
#pragma unroll 1
          for (int c = 0; c < TN / 64; ++c) {
            const int col = t.n0 + hf * (TN / 2) + 32 * c;
            if (col >= half) break;
            uint32_t v[32];
            tmem_ld32(tacc + hf * (TN / 2) + 32 * c, v);
            tmem_ld_wait();
            staging_free();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t gw[4] = {hg[i].x, hg[i].y, hg[i].z, hg[i].w};
              const uint32_t uw[4] = {hu[i].x, hu[i].y, hu[i].z, hu[i].w};
              uint32_t og[4], ou[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 g2 = unpack_b16(gw[j]), u2 = unpack_b16(uw[j]);
                float dg[2], du[2];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                  const float g = b ? g2.y : g2.x, up = b ? u2.y : u2.x;
                  const float ga = __uint_as_float(v[8 * i + 2 * j + b]);
                  const float sg = __fdividef(1.0f, 1.0f + __expf(-g));
                  dg[b] = ga * up * sg * fmaf(g, 1.0f - sg, 1.0f);
                  du[b] = ga * g * sg;
                }
                og[j] = mine ? pack_b16(dg[0], dg[1]) : 0u;
                ou[j] = mine ? pack_b16(du[0], du[1]) : 0u;
              }
              put64(0, i, make_uint4(og[0], og[1], og[2], og[3]));
              put64(1, i, make_uint4(ou[0], ou[1], ou[2], ou[3]));
            }
            if (c + 1 < TN / 64) load_h(col + 32);
            staged();
            store(&tm_d, 0, 64, t.m0, limit, col, 0, 0, true, false);
            store(&tm_d, 2048, 64, t.m0, limit, col, 1, 0, true, false);
          }
        } else if (kEpi == Epi::Update) {
          const __half* hi_row = p.c0 + t.z * p.zc + (static_cast<int64_t>(t.m0) + r) * p.ldc;
          const __half* lo_row = p.c1 + t.z * p.zc + (static_cast<int64_t>(t.m0) + r) * p.ldc;
          const float* diag = p.diag + static_cast<int64_t>(t.z) * p.side;
          float coef = p.alpha;
          if (p.use_diag && !p.tall && mine) coef += __ldcg(diag + t.m0 + r);
#pragma unroll 1
          for (int c = 0; c < TN / 64; ++c) {
            const int col = t.n0 + hf * (TN / 2) + 32 * c;
            if (col >= p.n_total) break;
            uint4 hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              hi[i] = lo[i] = make_uint4(0, 0, 0, 0);
              if (mine && col + 8 * i < p.n_total) {  // rows are padded to 8 elements
                hi[i] = __ldcg(reinterpret_cast<const uint4*>(hi_row + col) + i);
                lo[i] = __ldcg(reinterpret_cast<const uint4*>(lo_row + col) + i);
              }
            }
            uint32_t v[32];
            tmem_ld32(tacc + hf * (TN / 2) + 32 * c, v);
            tmem_ld_wait();
            float y[32];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t hw[4] = {hi[i].x, hi[i].y, hi[i].z, hi[i].w};
              const uint32_t lw[4] = {lo[i].x, lo[i].y, lo[i].z, lo[i].w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 h2 = unpack_f16(hw[j]), l2 = unpack_f16(lw[j]);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                  const int e = 8 * i + 2 * j + b;
                  float cf = coef;
                  if (p.use_diag && p.tall) cf += __ldcg(diag + min(col + e, p.side - 1));
                  const float x = fmaf(b ? l2.y : l2.x, 1.0f / kLoScale, b ? h2.y : h2.x);
                  y[e] = fmaf(cf, x, __uint_as_float(v[e]));
                }
              }
            }
            if (!p.last) {
              staging_free();
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t wh[4], wl[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const int e = 8 * i + 2 * j;
                  wh[j] = pack_f16(y[e], y[e + 1]);
                  const float2 h2 = unpack_f16(wh[j]);
                  wl[j] = pack_f16((y[e] - h2.x) * kLoScale, (y[e + 1] - h2.y) * kLoScale);
                }
                put64(0, i, make_uint4(wh[0], wh[1], wh[2], wh[3]));
                put64(1, i, make_uint4(wl[0], wl[1], wl[2], wl[3]));
              }
              staged();
              store(&tm_d, 0, 64, t.m0, limit, col, 0, t.z, false, false);
              store(&tm_d2, 2048, 64, t.m0, limit, col, 0, t.z, false, false);
            } else if (p.direct) {
              __nv_bfloat16* dst =
                  p.out + (static_cast<int64_t>(t.z) * p.m_total + t.m0 + r) * p.n_total + col;
              if (mine) {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (col + e < p.n_total) dst[e] = __float2bfloat16_rn(y[e] * p.beta);
              }
            } else {
              staging_free();
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  w[j] = pack_b16(y[8 * i + 2 * j] * p.beta, y[8 * i + 2 * j + 1] * p.beta);
                put64(0, i, make_uint4(w[0], w[1], w[2], w[3]));
              }
              staged();
              store(&tm_d, 0, 64, t.m0, limit, col, 0, t.z, false, false);
            }
          }
        } else if (kEpi == Epi::Weights && p.out_f32) {
#pragma unroll 1
          for (int c = 0; c < TN / 64; ++c) {
            const int col = t.n0 + hf * (TN / 2) + 32 * c;
            if (col >= p.n_total) break;
            uint32_t v[32];
            if (t.nk > 0) {
              tmem_ld32(tacc + hf * (TN / 2) + 32 * c, v);
              tmem_ld_wait();
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = 0;
            }
            staging_free();
#pragma unroll
            for (int i = 0; i < 8; ++i) put128(i, make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
            staged();
            store(&tm_d, 0, 128, t.m0, limit, col, 0, t.z, false, p.accumulate != 0);
          }
        } else {  // Rows, Weights in bf16, Gram, Poly: 64 columns at a time
          const __half* c_row = nullptr;
          if (kEpi == Epi::Poly) c_row = p.c0 + t.z * p.zc + (static_cast<int64_t>(t.m0) + r) * p.ldc;
#pragma unroll 1
          for (int c = 0; c < TN / 128; ++c) {
            const int col = t.n0 + hf * (TN / 2) + 64 * c;
            if (col >= p.n_total) break;
            uint32_t w[32];
#pragma unroll
            for (int s2 = 0; s2 < 2; ++s2) {
              uint32_t v[32];
              if (kSched != Sched::Experts || t.nk > 0) {
                tmem_ld32(tacc + hf * (TN / 2) + 64 * c + 32 * s2, v);
                tmem_ld_wait();
              } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0;
              }
              if (kEpi == Epi::Poly) {
                uint4 g[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  g[i] = make_uint4(0, 0, 0, 0);
                  if (mine && col + 32 * s2 + 8 * i < p.n_total)
                    g[i] = __ldcg(reinterpret_cast<const uint4*>(c_row + col + 32 * s2) + i);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const uint32_t gw[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    const float2 g2 = unpack_f16(gw[j]);
                    float o[2];
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                      const int e = 8 * i + 2 * j + b;
                      o[b] = fmaf(p.beta, b ? g2.y : g2.x, p.alpha * __uint_as_float(v[e]));
                      if (p.use_diag && col + 32 * s2 + e == t.m0 + r && mine) {
                        p.diag[static_cast<int64_t>(t.z) * p.side + t.m0 + r] = o[b];
                        o[b] = 0.f;
                      }
                    }
                    w[16 * s2 + 4 * i + j] = pack_f16(o[0], o[1]);
                  }
                }
              } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const float a = __uint_as_float(v[2 * i]), b = __uint_as_float(v[2 * i + 1]);
                  w[16 * s2 + i] = kEpi == Epi::Gram ? pack_f16(p.alpha * a, p.alpha * b) : mine ? pack_b16(a, b) : 0u;
                }
              }
            }
            staging_free();
#pragma unroll
            for (int i = 0; i < 8; ++i) put128(i, make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
            staged();
            store(&tm_d, 0, 128, t.m0, limit, col, 0, kSched == Sched::Blocks ? 0 : t.z, false, false);
          }
        }
      }
      if (t.nk > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[buf]);
        ++acc_it;
      }
    }
    if (lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // copies and MMAs issued before a wait gave up may still be landing; they
    // finish within microseconds
    const unsigned long long t0 = globaltimer();
    while (globaltimer() - t0 < 100000ull) __nanosleep(1000);
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, kTmemCols);
  }
}

// ------------------------------------------------------------------ host side
// 3-D tensor map over 16-bit (or fp32) elements: dims d0 (contiguous), d1, d2
// with strides s1, s2 in bytes, box b0 x b1 x 1 or, for row_last, b0 x 1 x b1.
// row_bytes of the box: 128 or 64, which also names the swizzle.
enum class Elem { Bf16, F16, F32 };
inline int make_map3(CUtensorMap* m, const void* base, Elem el, int64_t d0, int64_t d1, int64_t d2, int64_t s1,
                     int64_t s2, int b0, int b1, int b2) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (!enc) return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled entry point not available");
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d0), static_cast<cuuint64_t>(d1), static_cast<cuuint64_t>(d2)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(s1), static_cast<cuuint64_t>(s2)};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(b0), static_cast<cuuint32_t>(b1), static_cast<cuuint32_t>(b2)};
  const cuuint32_t estr[3] = {1, 1, 1};
  const int esize = el == Elem::F32 ? 4 : 2;
  const CUtensorMapDataType dt = el == Elem::Bf16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                 : el == Elem::F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                   : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  const CUresult r = enc(m, dt, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         b0 * esize == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
  return MOE_OK;
}

// Launches one product; pdl: chained to the launch before it.
template <Form kForm, Sched kSched, Epi kEpi, int TN, bool kBf16>
int launch_tile_gemm(const char* nm, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& d,
                     const CUtensorMap& d2, const GemmParams& p, int64_t max_units, bool pdl, cudaStream_t stream) {
  auto kernel = tile_gemm_kernel<kForm, kSched, kEpi, TN, kBf16>;
  constexpr int smem = GemmShape<TN>::smem;
  static std::atomic<bool> attr_set[kMaxDevices];  // per device; setting it twice is harmless
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cuda_fail("cudaGetDevice");
  if (dev >= kMaxDevices || !attr_set[dev].load(std::memory_order_relaxed)) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return cuda_fail(nm, e);
    if (dev < kMaxDevices) attr_set[dev].store(true, std::memory_order_relaxed);
  }
  const int nsm = sm_count();
  if (nsm <= 0) return cuda_fail("cudaDeviceGetAttribute(SM count)");
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(static_cast<unsigned>(max_units < nsm ? max_units : nsm), 1, 1);
  c.blockDim = dim3(kGThreads, 1, 1);
  c.dynamicSmemBytes = smem;
  c.stream = stream;
  c.attrs = attr;
  c.numAttrs = pdl ? 1 : 0;
  const cudaError_t err = cudaLaunchKernelEx(&c, kernel, a, b, d, d2, p);
  return err == cudaSuccess ? MOE_OK : cuda_fail(nm, err);
}

}  // namespace moe
