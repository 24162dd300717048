// Newton-Schulz steps on matrices of a shorter side of 65 to 256 and a longer
// one of at most 512 (1024 for a side up to 128): one launch, a cluster of up to
// 8 CTAs a matrix, with one barrier of the cluster a step instead of three
// launches (128 x 128: 32 us, 79 launched; 256 x 256: 78 and 87; 28 of them: 83
// and 107).
//
// CTA r of a cluster owns 64 (128) places of the longer side, its share of X, in
// fp32 registers from the first step to the last.  Only X's fp16 operand is
// shared: every CTA writes its part of it to memory, S x 64, and after the
// barrier reads all of it (K-major, whichever way the matrix lies) for
//   A = X X^T                   every CTA all of it: S x S in TMEM, then fp16 in shared memory
//   B = b A + c A A             from there, replaced in place
//   X <- (a + d) X + B X        its own places; d: B's diagonal, from step kNsDiagFrom on
// Computing A and B on every CTA costs tensor time that nobody else could use
// (4 thousand cycles each of a step's 24 at 256 x 256, where the barrier and the
// reads of X take 5 and the three accumulators' ways out of TMEM 9), and saves
// two exchanges through memory and two barriers.  Two CTAs sharing it, each
// storing its half of A and B into both, took 96 us at 256 x 256: rows of 16
// bytes a lane go slowly to another CTA's shared memory.
//
// The warps work in turn: warp 0 copies, warp 1 issues the MMAs, and all eight
// take the accumulators, 32 rows each (warp & 3), either all columns of one of
// two halves of 128 rows, or every second piece of 32 columns.
#pragma once

#include "tile_gemm.cuh"

namespace moe {

constexpr int kNrThreads = 256;
constexpr int kNrSide = 256, kNrMaxCtas = 8;
// Places of the longer side a CTA: as many as its threads' 64 registers hold, or fewer on more CTAs.
__host__ __device__ constexpr int nr_places(int side, int len) { return side <= 128 && len > 64 * kNrMaxCtas ? 128 : 64; }
constexpr int kNrMat = 4 * 32768;       // A, then B: blocks of 64 columns, 256 rows of 128 bytes
constexpr int kNrShare = 256 * 128;     // X's own share as an operand: S rows of 64 places, or two blocks of 128 rows
constexpr int kNrHalf = 128 * 128;       // 64 places of 128 rows of X
constexpr int kNrStages = 4;            // of one half each, or 2 of both
constexpr int kNrTotal = 112;  // CTAs a call
constexpr int kNrCtrl = kNrMat + kNrShare + kNrStages * kNrHalf;
constexpr int kNrSmem = 1024 + kNrCtrl + 128 + 4 * kNrSide;
static_assert(kNrSmem + 256 <= 232448, "shared memory");

struct NsResident {
  const void* g;
  int f32, side, len, tall, steps, ldx;
  float a, b, c;
  double eps;
  __half* x[2];  // (E, side, ldx): X's operand, by turns
  __nv_bfloat16* out;
  int* status;
  unsigned long long wait_ns;
};

__global__ void __launch_bounds__(kNrThreads, 1)
    ns_resident_kernel(const __grid_constant__ CUtensorMap map0, const __grid_constant__ CUtensorMap map1,
                       const __grid_constant__ NsResident p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ double warps[kNrThreads / 32];
  __shared__ double norm2;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *mat = smem, *share = smem + kNrMat, *ring = share + kNrShare;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kNrCtrl);
  uint64_t* empty = full + kNrStages;
  uint64_t* acc = empty + kNrStages;
  uint32_t* tmem_sm = reinterpret_cast<uint32_t*>(acc + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_sm + 1);
  float* diag = reinterpret_cast<float*>(smem + kNrCtrl + 128);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int S = p.side, halves = S > 128 ? 2 : 1, kblocks = (S + 63) / 64, nk = (p.len + 63) / 64;
  const int group = warp >> 2, half = halves == 2 ? group : 0;
  const int row = half * 128 + 32 * (warp & 3) + lane;
  const int places = nr_places(S, p.len);
  const int pieces = halves * places / 64;              // of 32 places: this thread's, from c0 of the CTA's on
  const int c0 = halves == 2 ? 0 : places / 2 * group;
  const int stages = kNrStages / halves;
  const int64_t z = blockIdx.y;
  const int l0 = static_cast<int>(cluster_ctarank()) * places + c0;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.status, p.wait_ns));
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < kNrStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&map0);
    prefetch_tmap(&map1);
  }
  if (warp == 1) {
    tmem_alloc(tmem_sm, 512);
    tmem_relinquish();
  }

  // The share of G, and the norm over the cluster.  Matrices come and go through `mat`, its places a row of X,
  // so that the lanes' accesses to memory are consecutive whichever way the matrix lies (each thread its own row, one
  // after another: 8 us at 128 x 128, and as much for the result).
  auto stage = [&](int i, int l) -> float& { return reinterpret_cast<float*>(mat)[i * (places + 1) + l]; };
  // Turn k of a thread: row i_lo + k i_by of X, place l_lo + k l_by of the CTA's.
  const int first = l0 - c0;
  const int wrap = halves == 2 ? 1 : 2;  // turns of 128 rows go to two threads each
  const int i_lo = p.tall ? static_cast<int>(threadIdx.x) % (128 * halves) : static_cast<int>(threadIdx.x) / places;
  const int l_lo = p.tall ? static_cast<int>(threadIdx.x) / (128 * halves) : static_cast<int>(threadIdx.x) % places;
  const int i_by = p.tall ? 0 : kNrThreads / places, l_by = p.tall ? wrap : 0;
  const int turns = p.tall ? places / wrap : (S + i_by - 1) / i_by;
  const int64_t by_i = p.tall ? 1 : p.len, by_l = p.tall ? S : 1;
  const int64_t base = z * S * p.len + first * by_l;
  auto row_of = [&](int k) { return i_lo + k * i_by; };
  auto place_of = [&](int k) { return l_lo + k * l_by; };
  auto index_of = [&](int i, int l) { return base + i * by_i + l * by_l; };
  // sixteen at once, from clamped places and without a condition: behind one each, loads are waited for one by one
  auto take = [&](auto load) {
#pragma unroll 1
    for (int k0 = 0; k0 < turns; k0 += 16) {
      float v[16];
#pragma unroll
      for (int u = 0; u < 16; ++u)
        v[u] = load(index_of(min(row_of(k0 + u), S - 1), min(place_of(k0 + u), p.len - 1 - first)));
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        const int i = row_of(k0 + u), l = place_of(k0 + u);
        if (i < S && l < places) stage(i, l) = v[u];
      }
    }
  };
  if (p.f32)
    take([&](int64_t at) { return __ldg(static_cast<const float*>(p.g) + at); });
  else
    take([&](int64_t at) { return __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(p.g) + at)); });
  __syncthreads();
  float x[2][32];
  double sum = 0.0;
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      x[k][j] = k < pieces && row < S && l0 + 32 * k + j < p.len ? stage(row, c0 + 32 * k + j) : 0.f;
      sum += static_cast<double>(x[k][j]) * static_cast<double>(x[k][j]);
    }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (lane == 0) warps[warp] = sum;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = __shfl_sync(0xffffffffu, *tmem_sm, 0);
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int w = 0; w < kNrThreads / 32; ++w) s += warps[w];
    norm2 = s;
  }
  __syncwarp();
  cluster_sync();
  double total = 0.0;
  for (uint32_t q = 0; q < cluster_nctarank(); ++q) {
    double v;
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(cluster_addr(&norm2, q)) : "memory");
    total += v;
  }
  const NsFactors scale = ns_factors(sqrt(total) + p.eps);
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int j = 0; j < 32; ++j) x[k][j] = x[k][j] * scale.pre * scale.post;

  // X's share in fp16: to the next operand in memory, and as the own one in shared memory (MN-major, 64 places a row)
  auto publish = [&](int buf) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k >= pieces) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = pack_f16(x[k][8 * i + 2 * j], x[k][8 * i + 2 * j + 1]);
        const uint4 v = make_uint4(w[0], w[1], w[2], w[3]);
        const int chunk = (c0 + 32 * k) / 8 + i;
        *reinterpret_cast<uint4*>(share + (chunk >> 3) * kNrHalf + row * 128 + (((chunk & 7) ^ (row & 7)) << 4)) = v;
        if (row < S) *reinterpret_cast<uint4*>(p.x[buf] + (z * S + row) * p.ldx + l0 + 32 * k + 8 * i) = v;
      }
    }
  };
  publish(0);

  // the accumulator's pieces of 32 columns that this thread's warp takes, and where they lie in `mat`
  auto for_pieces = [&](auto f) {
#pragma unroll 1
    for (int c = halves == 2 ? 0 : group; c < 2 * kblocks; c += halves == 2 ? 1 : 2) f(32 * c);
  };
  auto mat_at = [&](int col, int i) {
    return mat + (col / 64) * 32768 + row * 128 + ((((col % 64) / 8 + i) ^ (row & 7)) << 4);
  };
  const uint32_t lanes = tbase + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + static_cast<uint32_t>(half) * 256;
  auto piece_of = [&](int col, uint32_t (&v)[32]) {
    tmem_ld32(lanes + col, v);
    tmem_ld_wait();
    if (col + 32 > S) {  // columns behind the side: nothing was summed there
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (col + e >= S) v[e] = 0;
    }
  };
  const int n16 = (S + 15) / 16 * 16;
  const uint32_t idesc = idesc_f16(128, n16, false, false, false);
  uint32_t acc_ph = 0;
  int slot = 0;       // of the ring, warps 0 and 1
  uint32_t ph = 0;
  auto accumulated = [&] {
    wait(acc, acc_ph);
    acc_ph ^= 1u;
    tc_fence_after();
  };
  auto operands_written = [&] {
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  };

  for (int step = 0; step < p.steps; ++step) {
    // every CTA's part of X is in memory, and in its own shared memory
    fence_proxy_async_all();
    tc_fence_before();
    __syncwarp();
    cluster_sync();
    tc_fence_after();
    if (warp == 0) {
      fence_proxy_async_all();
      const CUtensorMap* map = step & 1 ? &map1 : &map0;
      const uint64_t pol = policy_evict_normal();
      bool ok = true;
      for (int kc = 0; kc < nk && ok; ++kc) {
        ok = wait(&empty[slot], ph ^ 1u);
        if (!ok) break;
        uint8_t* dst = ring + slot * halves * kNrHalf;
        if (elect_one()) {
          mbar_arrive_expect_tx(&full[slot], halves * kNrHalf);
          for (int h = 0; h < halves; ++h)
            tma_load_3d(dst + h * kNrHalf, map, &full[slot], 64 * kc, 128 * h, static_cast<int>(z), pol);
        }
        __syncwarp();
        if (++slot == stages) { slot = 0; ph ^= 1u; }
      }
    } else if (warp == 1) {
      bool ok = true;
      for (int kc = 0; kc < nk && ok; ++kc) {
        ok = wait(&full[slot], ph);
        if (!ok) break;
        tc_fence_after();
        const uint32_t b = smem_u32(ring + slot * halves * kNrHalf);
#pragma unroll 1
        for (int h = 0; h < halves; ++h)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f16_one(tbase + 256 * h, sdesc_sw128(b + h * kNrHalf) + 2 * kk, sdesc_sw128(b) + 2 * kk, idesc,
                        (kc | kk) != 0);
        tc_commit_one(&empty[slot]);
        __syncwarp();
        if (++slot == stages) { slot = 0; ph ^= 1u; }
      }
      tc_commit_one(acc);
    }
    accumulated();
    for_pieces([&](int col) {
      uint32_t v[32];
      piece_of(col, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = 8 * i + 2 * j;
          constexpr float alpha = 1.0f / (kNsScale * kNsScale);
          w[j] = pack_f16(alpha * __uint_as_float(v[e]), alpha * __uint_as_float(v[e + 1]));
        }
        *reinterpret_cast<uint4*>(mat_at(col, i)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    });
    operands_written();
    if (warp == 1) {
      const uint32_t m = smem_u32(mat);
#pragma unroll 1
      for (int h = 0; h < halves; ++h)
#pragma unroll 1
        for (int kb = 0; kb < kblocks; ++kb)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f16_one(tbase + 256 * h, sdesc_sw128(m + kb * 32768 + h * 16384) + 2 * kk,
                        sdesc_sw128(m + kb * 32768) + 2 * kk, idesc, (kb | kk) != 0);
      tc_commit_one(acc);
    }
    accumulated();
    const bool use_diag = step >= kNsDiagFrom;
    for_pieces([&](int col) {
      uint32_t v[32];
      piece_of(col, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 old = *reinterpret_cast<const uint4*>(mat_at(col, i));
        const uint32_t aw[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 a2 = unpack_f16(aw[j]);
          const int e = 8 * i + 2 * j;
          v[e] = __float_as_uint(fmaf(p.b, a2.x, p.c * __uint_as_float(v[e])));
          v[e + 1] = __float_as_uint(fmaf(p.b, a2.y, p.c * __uint_as_float(v[e + 1])));
        }
      }
      const bool on_diag = use_diag && col == row - lane;  // lane e's is element e of this piece
      if (on_diag) {
        uint32_t pick[16];  // element `lane`, by halving
#pragma unroll
        for (int e = 0; e < 16; ++e) pick[e] = lane & 16 ? v[e + 16] : v[e];
#pragma unroll
        for (int n = 8; n > 0; n >>= 1)
#pragma unroll
          for (int e = 0; e < n; ++e) pick[e] = lane & n ? pick[e + n] : pick[e];
        diag[row] = __uint_as_float(pick[0]);
      }
      const uint32_t keep = lane & 1 ? 0x0000FFFFu : 0xFFFF0000u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          w[j] = pack_f16(__uint_as_float(v[8 * i + 2 * j]), __uint_as_float(v[8 * i + 2 * j + 1]));
          w[j] &= on_diag && (lane >> 1) == 4 * i + j ? keep : 0xFFFFFFFFu;
        }
        *reinterpret_cast<uint4*>(mat_at(col, i)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    });
    operands_written();
    if (warp == 1) {
      const uint32_t m = smem_u32(mat), own = smem_u32(share);
#pragma unroll 1
      for (int h = 0; h < halves; ++h)
#pragma unroll 1
        for (int kb = 0; kb < kblocks; ++kb)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f16_one(tbase + 256 * h, sdesc_sw128(m + kb * 32768 + h * 16384) + 2 * kk,
                        sdesc_sw128_mn(own + kb * 8192, kNrHalf) + 128 * kk, idesc_f16(128, places, false, false, true),
                        (kb | kk) != 0);
      tc_commit_one(acc);
    }
    accumulated();
    const float coef = p.a + (use_diag && row < S ? diag[row] : 0.f);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k >= pieces) break;
      uint32_t v[32];
      tmem_ld32(lanes + c0 + 32 * k, v);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 32; ++j) x[k][j] = fmaf(coef, x[k][j], __uint_as_float(v[j]));
    }
    if (step + 1 < p.steps) publish((step + 1) & 1);
  }
  if (row < S) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (k >= pieces) break;
#pragma unroll
      for (int j = 0; j < 32; ++j) stage(row, c0 + 32 * k + j) = x[k][j] * (1.0f / kNsScale);
    }
  }
  __syncthreads();
#pragma unroll 4
  for (int k = 0; k < turns; ++k) {
    const int i = row_of(k), l = place_of(k);
    if (i < S && l < places && first + l < p.len) p.out[index_of(i, l)] = __float2bfloat16_rn(stage(i, l));
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {  // copies issued before a wait gave up may still be landing
    const unsigned long long t0 = globaltimer();
    while (globaltimer() - t0 < 100000ull) __nanosleep(1000);
  }
  __syncwarp();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// Clusters that a GPU has room for at once limit it to few matrices: with more, the chained launches share the SMs better.
inline bool ns_resident_fits(int E, int M, int N) {
  const int side = M < N ? M : N, len = M < N ? N : M;
  return side <= kNrSide && len <= kNrMaxCtas * nr_places(side, len) &&
         static_cast<int64_t>(E) * ((len + nr_places(side, len) - 1) / nr_places(side, len)) <= kNrTotal;
}

static int run_ns_resident(const char* nm, const void* g, int f32, int E, int M, int N, int steps, float a, float b,
                           float c, float eps, void* out, uint8_t* ws, cudaStream_t stream) {
  NsResident p{};
  p.g = g;
  p.f32 = f32;
  p.side = M < N ? M : N;
  p.len = M < N ? N : M;
  p.tall = M > N ? 1 : 0;
  p.steps = steps;
  p.ldx = (p.len + 127) / 128 * 128;  // whole shares
  p.a = a; p.b = b; p.c = c;
  p.eps = eps;
  // within the workspace's four buffers of iterates (len * ns_layout's pitch each, or side * it): two of side * ldx,
  // ldx < len + 128 and len > 64
  const int64_t bytes = (static_cast<int64_t>(E) * p.side * p.ldx * 2 + 255) / 256 * 256;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.wait_ns = kWaitTimeoutNs;
  if (int rc = status_word(nm, &p.status)) return rc;
  CUtensorMap map[2];
  for (int i = 0; i < 2; ++i) {
    p.x[i] = reinterpret_cast<__half*>(ws + i * bytes);
    if (int rc = make_map3(&map[i], p.x[i], Elem::F16, p.len, p.side, E, int64_t(p.ldx) * 2, int64_t(p.side) * p.ldx * 2,
                           64, 128, 1))
      return rc;
  }
  cudaError_t err = cudaFuncSetAttribute(ns_resident_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNrSmem);
  if (err != cudaSuccess) return cuda_fail(nm, err);
  const int places = nr_places(p.side, p.len), ctas = (p.len + places - 1) / places;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, E, 1);
  cfg.blockDim = dim3(kNrThreads, 1, 1);
  cfg.dynamicSmemBytes = kNrSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  err = cudaLaunchKernelEx(&cfg, ns_resident_kernel, map[0], map[1], p);
  return err == cudaSuccess ? MOE_OK : cuda_fail(nm, err);
}

}  // namespace moe
