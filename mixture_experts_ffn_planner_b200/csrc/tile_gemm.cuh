// A persistent tcgen05 product of 16-bit operands, tile by tile, for the
// training operators: D (fp32 in TMEM) = A . B over a contraction cut into
// chunks of 64, in the three forms that a layer's forward pass and its two
// gradients need,
//   NT   D[i][j] = sum_k A[i][k] B[j][k]    both operands K-major
//   NN   D[i][j] = sum_k A[i][k] B[k][j]    B is MN-major
//   TN   D[i][j] = sum_k A[k][i] B[k][j]    both are MN-major
// The tensor cores read either layout from shared memory (a bit each in the
// instruction descriptor), so no operand is ever transposed in memory.
//
// Tiles.  kPair: two CTAs of a cluster work on one 256 x 256 tile with
// cta_group::2 MMAs: each loads half of A's rows and half of B's, 32 KB a
// chunk, and takes half of D's rows out of its own TMEM.  That is 128 flop a
// byte from L2, where one CTA on a 128 x 256 tile has 85.  At 8192 tokens on 64
// experts (K = N = 2048, cold L2) the gate/up product takes 434 us by itself on a
// GPU that was idle, where one CTA took 484, and 540 to 550 among others of its
// kind; the tensor pipe is busy 82 % of the time at the 1.44 GHz that the power
// limit leaves, of which an eighth goes to rows behind an expert's last in
// 256-row tiles.  Otherwise one CTA works on 128 x 128: for experts with too
// few rows to fill 256, where the weights' bytes bound the call and 148 CTAs
// stream more of them at once.
//
// One CTA per SM walks the tiles.  Warp 0 copies operand chunks by TMA into a
// ring of 5 or 6 stages (the same product: 543 us with 3, 485 with 4, 471 with
// 5, all else as it was then), warp 1 (of the even CTA of a pair) issues the
// MMAs; warps 2-9 take a finished accumulator out of TMEM (two of them
// alternate, so the epilogue of a tile runs beside the next tile's MMAs) and
// store it by TMA from two swizzled staging buffers a warp, 32 columns of bf16
// at a time.  What an epilogue reads beside the accumulator (h, the iterate,
// the Gram matrix) is loaded by TMA into the staging buffer that its result
// then replaces, one piece ahead: read by each thread from its own row, as the
// accumulator lies, those loads took longer than the product.  The roles' warps
// stay converged, and one elected lane issues: behind a branch on the lane, an
// instruction's operands are moved over one by one, and the issue of a chunk's
// four MMAs took 520 cycles, more than the MMAs.  Every wait is bounded.
//
// What a tile is (Sched):
//   Blocks   rows of one expert (consecutive planner blocks, whatever block_m
//            is) by columns of that expert's weights;
//   Experts  a part of one expert's weight gradient, contracted over the
//            expert's rows (where they begin is looked up once, into shared
//            memory: searched for by every role at every tile, it made tiles of
//            few rows cost 5.8 us); what lies behind the last routed one in a
//            chunk is cleared in shared memory by warp 10, whatever it holds;
//   Batch    a part of one matrix of a batch; of a symmetric one (Gram, Poly)
//            the tiles on and above the diagonal, each stored as it is and
//            transposed.
#pragma once

#include <atomic>
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"
#include "segments.h"

namespace moe {

enum class Form { NT, NN, TN };
enum class Sched { Blocks, Experts, Batch };
enum class Epi {
  Rows,        // bf16 rows of an expert
  GateUp,      // h = [gate | up] and silu(gate) * up, bf16
  SwigluGrad,  // D is the gradient of act: bf16 gradients of gate and up
  Weights,     // a weight gradient, bf16 or fp32, the latter optionally added to what is there
  Gram,        // alpha * D, fp16
  Poly,        // beta * C + alpha * D, fp16, optionally with its diagonal taken out into fp32
  Update       // coefficient * (hi + lo / 2048) + D: the next iterate's hi and lo, or the result in bf16
};

constexpr int kGK = 64;     // contraction indices a chunk
constexpr int kGRow = 128;  // bytes of an operand row in a stage
constexpr int kGHalf = 128 * kGRow;   // bytes of a CTA's A, and of its B, a chunk
constexpr int kGStage = 2 * kGHalf;
constexpr int kGEpiWarps = 8;
constexpr int kGPatchWarp = 2 + kGEpiWarps;
constexpr int kGThreads = 32 * (3 + kGEpiWarps);
constexpr int kGTile = 32 * 64;  // bytes of a staging tile: 32 rows of 64
// epilogues that read a second operand
constexpr bool epi_side(Epi e) { return e == Epi::SwigluGrad || e == Epi::Poly || e == Epi::Update; }
constexpr int gemm_stages(Sched s, Epi e) { return epi_side(e) || s == Sched::Experts ? 5 : 6; }
constexpr int gemm_buf(Epi e) { return (epi_side(e) ? 2 : 1) * kGTile; }  // bytes of a staging buffer; two a warp
constexpr int gemm_ctrl(Sched s, Epi e) { return gemm_stages(s, e) * kGStage + kGEpiWarps * 2 * gemm_buf(e); }
constexpr int kGCtrlBytes = 512;
constexpr int gemm_smem(Sched s, Epi e) {
  return 1024 + gemm_ctrl(s, e) + kGCtrlBytes + (s == Sched::Experts ? 4 * (kMaxExperts + 1) : 0);
}
static_assert(gemm_smem(Sched::Blocks, Epi::Rows) <= 232448 && gemm_smem(Sched::Batch, Epi::Update) <= 232448 &&
                  gemm_smem(Sched::Experts, Epi::Weights) <= 232448,
              "shared memory");
constexpr float kLoScale = 2048.0f;  // lo = fp16(2048 * (value - hi)): 11 more bits

constexpr int tile_m(bool pair) { return pair ? 256 : 128; }
constexpr int tile_n(bool pair) { return pair ? 256 : 128; }

struct GemmParams {
  // planner (Blocks, Experts)
  const int32_t* sorted_ids;
  const int32_t* expert_ids;
  const int32_t* ntpp;
  int bm, max_blocks, E;
  // tiles
  int m_tiles, n_tiles, batches;
  int m_total, n_total;  // rows (Experts, Batch) and columns of D; GateUp, SwigluGrad: columns of act
  int nk;                // chunks of the contraction (Blocks, Batch)
  int a_rows;            // rows of A's boxes (A K-major): 128, or 32 where tiles have few rows
  int store_rows;        // rows of the store (and side) boxes
  // Weights
  int out_f32, accumulate;
  // Gram, Poly, Update (scalars read past L1: the launches are chained and reuse buffers)
  float alpha, beta;
  int use_diag, tall, last, direct;
  float* diag;           // (batches, side)
  int side;
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
  int z;       // expert or matrix
  int m0, n0;  // this CTA's first row of A, the tile's first column
  int total;   // rows of the tile that belong to the output
  int limit;   // those of this CTA's half (<= 0: none)
  int nk;      // chunks; 0: a weight gradient without rows
  bool mirror; // symmetric: the transposed tile is stored too
  int p0;      // Experts: first row of the contraction
  int rows;    // Experts: its routed rows
};

// first[e], e <= E: the first of the plan's blocks whose expert is >= e (by all threads; segments.h).
// Two blocks have the same entry only where ids do not ascend: both CTAs of a pair take the least all the same.
__device__ __forceinline__ void find_segments(const GemmParams& p, int blocks, int* first) {
  for (int e = static_cast<int>(threadIdx.x); e <= p.E; e += kGThreads) first[e] = blocks;
  __syncthreads();
  for (int b = static_cast<int>(threadIdx.x); b <= blocks; b += kGThreads) {
    const SegmentEntries s = segment_entries(b, blocks, p.E, b == 0 ? -1 : __ldg(p.expert_ids + b - 1),
                                             b == blocks ? p.E : __ldg(p.expert_ids + b));
    for (int e = s.lo; e <= s.hi; ++e) atomicMin(&first[e], b);
  }
}

// The tiles of one role, in the order that every role walks them: tile numbers
// `from`, from + stride, ... (warp-collective).
template <Sched kSched, Epi kEpi, bool kPair>
struct Walk {
  static constexpr int kCols = kEpi == Epi::GateUp ? tile_n(kPair) / 2 : tile_n(kPair);
  static constexpr bool kSym = kEpi == Epi::Gram || kEpi == Epi::Poly;  // square tiles, m_tiles == n_tiles
  const GemmParams& p;
  const int lane, rank, stride;
  const int blocks;
  int u, units, per_z;
  // Blocks: a window of 32 blocks and those in it that begin a tile of their expert
  int win = 0, before = 0, carry = 0, prev = -1, id = -1;
  uint32_t heads = 0;
  // Experts: the segments, and the order's ids in the last block of the next tile's expert, 32 an element
  const int* first;
  int z_next = -1;
  int last_ids[4];

  __device__ __forceinline__ Walk(const GemmParams& p_, int rank_, int from, int stride_, int blocks_, const int* first_)
      : p(p_), lane(static_cast<int>(lane_id())), rank(rank_), stride(stride_), blocks(blocks_), u(from), first(first_) {
    per_z = kSym ? p.m_tiles * (p.m_tiles + 1) / 2 : p.m_tiles * p.n_tiles;
    units = p.batches * per_z;
    if (kSched == Sched::Blocks) look(0);
    if (kSched == Sched::Experts) peek();
  }

  // Starts the loads of last_ids for tile u, a tile ahead of their use.
  __device__ __forceinline__ void peek() {
    if (u >= units || u / per_z == z_next) return;
    z_next = u / per_z;
    const int end = first[z_next + 1];
    if (segment_blocks(first[z_next], end) <= 0) return;
    // (no value is chosen here: that would wait for the loads)
    const int32_t* block = p.sorted_ids + static_cast<int64_t>(end - 1) * p.bm;
#pragma unroll
    for (int i = 0; i < 4; ++i) last_ids[i] = __ldg(block + min(32 * i + lane, p.bm - 1));
  }

  // The window from block `at` on: a tile begins every tile_m / bm blocks of an expert's run.
  __device__ __forceinline__ void look(int at) {
    win = at;
    const int per = tile_m(kPair) / p.bm;
    id = at + lane < blocks ? __ldg(p.expert_ids + at + lane) : -1;
    const int left = __shfl_up_sync(0xffffffffu, id, 1);
    const uint32_t starts = __ballot_sync(0xffffffffu, id != (lane ? left : prev));
    const uint32_t mine = starts & (0xffffffffu >> (31 - lane));
    const int pos = mine ? lane - (31 - __clz(static_cast<int>(mine))) : lane + carry;  // place in the run
    heads = __ballot_sync(0xffffffffu, id >= 0 && id < p.E && pos % per == 0);
    carry = __shfl_sync(0xffffffffu, pos, 31) + 1;
    prev = __shfl_sync(0xffffffffu, id, 31);
  }

  __device__ __forceinline__ bool next(Tile* t) {
    if (kSched == Sched::Blocks) {
      const int want = u / p.n_tiles;
      while (want - before >= __popc(heads)) {
        if (win + 32 >= blocks) return false;
        before += __popc(heads);
        look(win + 32);
      }
      // the head that has want - before others ahead of it in the window
      const int ahead = __popc(heads & ((1u << lane) - 1u));
      const int at = __ffs(static_cast<int>(__ballot_sync(0xffffffffu, (heads >> lane & 1u) && ahead == want - before))) - 1;
      const int b = win + at;
      t->z = __shfl_sync(0xffffffffu, id, at);
      t->n0 = (u - want * p.n_tiles) * kCols;
      // blocks of the tile: those from b on with its expert (id is -1 behind the last), read again where the window ends
      const int per = tile_m(kPair) / p.bm;
      uint32_t same = __ballot_sync(0xffffffffu, id == t->z) >> at;
      if (at + per > 32)
        same = __ballot_sync(0xffffffffu, b + lane < blocks && __ldg(p.expert_ids + min(b + lane, blocks - 1)) == t->z);
      const int run = min(per, same == 0xffffffffu ? 32 : __ffs(static_cast<int>(~same)) - 1);
      t->m0 = b * p.bm + rank * 128;
      t->total = run * p.bm;
      t->limit = min(128, t->total - rank * 128);
      t->nk = p.nk;
      t->p0 = t->rows = 0;
      t->mirror = false;
      u += stride;
      return true;
    }
    if (u >= units) return false;
    t->z = u / per_z;
    int mi = 0, ni = u - t->z * per_z;
    if (kSym) {
      while (ni >= p.n_tiles - mi) ni -= p.n_tiles - mi++;
      ni += mi;
      t->mirror = ni != mi;
    } else {
      mi = ni / p.n_tiles;
      ni -= mi * p.n_tiles;
      t->mirror = false;
    }
    t->m0 = mi * tile_m(kPair) + rank * 128;
    t->n0 = ni * kCols;
    t->total = p.m_total - mi * tile_m(kPair);
    t->limit = min(128, p.m_total - t->m0);
    t->nk = p.nk;
    t->p0 = t->rows = 0;
    if (kSched == Sched::Experts) {
      const int lo = first[t->z], n = segment_blocks(lo, first[t->z + 1]);
      t->p0 = lo * p.bm;
      if (n > 0) {  // whole blocks, and the routed rows that the last one begins with
        t->rows = (n - 1) * p.bm;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          t->rows += __popc(__ballot_sync(0xffffffffu, 32 * i + lane < p.bm && last_ids[i] >= 0));
      }
      t->nk = (t->rows + kGK - 1) / kGK;
      u += stride;
      peek();
      return true;
    }
    u += stride;
    return true;
  }
};

// What a chunk of a weight gradient's contraction holds beyond the expert's
// routed rows: from row `rem` of 64 on; 64 or more: nothing.
__device__ __forceinline__ bool ragged(const Tile& t, int kc) { return t.rows - kc * kGK < kGK; }

// A thread's view of its CTA: the shared memory's parts and its place.
struct TileCta {
  uint8_t* smem;
  uint64_t *full, *empty;
  uint64_t* part;       // ragged chunks: landed, not yet cleared
  uint64_t *acc_full, *acc_empty;
  uint64_t* side_full;  // [kGEpiWarps][2]
  uint32_t* tmem_base_sm;
  volatile int* abort_flag;
  int warp, lane;
  uint32_t rank, tbase;
};

// Shared memory's layout, barriers, TMEM; the CTA's other set-up may follow before tile_cta_ready.
template <int kStages, int kBuf, bool kPair>
__device__ __forceinline__ void tile_cta_setup(TileCta* c, uint8_t* smem_raw) {
  c->smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  c->full = reinterpret_cast<uint64_t*>(c->smem + kStages * kGStage + kGEpiWarps * 2 * kBuf);
  c->empty = c->full + kStages;
  c->part = c->empty + kStages;
  c->acc_full = c->part + kStages;
  c->acc_empty = c->acc_full + 2;
  c->side_full = c->acc_empty + 2;
  c->tmem_base_sm = reinterpret_cast<uint32_t*>(c->side_full + 2 * kGEpiWarps);
  c->abort_flag = reinterpret_cast<volatile int*>(c->tmem_base_sm + 1);
  // by shuffle, so that the compiler knows them to be the same in all lanes, and the roles' operands to be uniform
  c->warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  c->lane = threadIdx.x & 31;
  c->rank = kPair ? cluster_ctarank() : 0u;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      // pair: the even CTA's twice, for the copies of both, or warp 10 of each
      mbar_init(&c->full[s], kPair ? 2 : 1);
      mbar_init(&c->empty[s], 1);
      mbar_init(&c->part[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&c->acc_full[a], 1);
      mbar_init(&c->acc_empty[a], kPair ? 2 * kGEpiWarps : kGEpiWarps);
    }
    for (int i = 0; i < 2 * kGEpiWarps; ++i) mbar_init(&c->side_full[i], 1);
    *c->abort_flag = 0;
    fence_mbar_init();
  }
  if (c->warp == 1) {
    if (kPair) {
      tmem_alloc_pair(c->tmem_base_sm, 2 * tile_n(kPair));
      tmem_relinquish_pair();
    } else {
      tmem_alloc(c->tmem_base_sm, 2 * tile_n(kPair));
      tmem_relinquish();
    }
  }
}
template <bool kPair>
__device__ __forceinline__ void tile_cta_ready(TileCta* c) {
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync();  // the other CTA's barriers are ready
  tc_fence_after();
  c->tbase = __shfl_sync(0xffffffffu, *c->tmem_base_sm, 0);
}
template <bool kPair>
__device__ __forceinline__ void tile_cta_leave(const TileCta& c) {
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*c.abort_flag) {
    // copies and MMAs issued before a wait gave up may still be landing; they
    // finish within microseconds
    const unsigned long long t0 = globaltimer();
    while (globaltimer() - t0 < 100000ull) __nanosleep(1000);
  }
  __syncwarp();
  if (kPair) cluster_sync();  // neither CTA leaves while the other may still read or signal it
  if (c.warp == 1) {
    tc_fence_after();
    if (kPair)
      tmem_dealloc_pair(c.tbase, 2 * tile_n(kPair));
    else
      tmem_dealloc(c.tbase, 2 * tile_n(kPair));
  }
}

// The product: every warp in its role over the tiles of `walk`.
template <Form kForm, Sched kSched, Epi kEpi, bool kPair, bool kBf16, int kStages, int kBuf>
__device__ __forceinline__ void tile_product(const TileCta& c, Walk<kSched, kEpi, kPair>& walk, const CUtensorMap* tm_a,
                                             const CUtensorMap* tm_b, const CUtensorMap* tm_d, const CUtensorMap* tm_d2,
                                             const CUtensorMap* tm_c, const CUtensorMap* tm_c2, const GemmParams& p) {
  constexpr int kN = tile_n(kPair);
  constexpr bool kAMn = kForm == Form::TN, kBMn = kForm != Form::NT;
  constexpr int kStaging = kStages * kGStage;
  // side tiles of 32 columns, one or two at once
  constexpr bool kSide = epi_side(kEpi);
  constexpr int kSideTiles = kEpi == Epi::Poly ? 1 : 2;
  uint8_t* const smem = c.smem;
  uint64_t *const full = c.full, *const empty = c.empty, *const part = c.part;
  uint64_t *const acc_full = c.acc_full, *const acc_empty = c.acc_empty, *const side_full = c.side_full;
  volatile int* const abort_flag = c.abort_flag;
  const int warp = c.warp, lane = c.lane;
  const uint32_t rank = c.rank, tbase = c.tbase;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return mbar_wait(bar, parity, abort_flag, p.status, p.wait_ns);
  };
  // a barrier that threads of the other CTA arrive on.  Cluster scope is dear: an acquire of it for every chunk, with
  // a releasing arrival from the other CTA, made a chunk of 256 x 256 x 64 cost 1.06 us.  So it is for the barriers
  // that need it: an accumulator's, once a tile, and a chunk's whose last rows warp 10 of either CTA has cleared.
  auto wait_cluster = [&](uint64_t* bar, uint32_t parity) {
    return mbar_wait<kPair>(bar, parity, abort_flag, p.status, p.wait_ns);
  };
  Tile t;

  if (warp == 0) {
    // ------------------------------------------------ TMA producer
    const uint64_t pol = policy_evict_normal();
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    while (ok && walk.next(&t)) {
      const int za = kSched == Sched::Batch ? t.z : 0;
      const int zb = kSched == Sched::Experts ? 0 : t.z;
      const int r = static_cast<int>(rank);
      // rows behind the tile's last are not loaded: what is in shared memory there reaches no row that is stored
      const int boxes = kAMn ? 0 : t.limit > 0 ? (t.limit + p.a_rows - 1) / p.a_rows : 0;
      const uint32_t mine = kGHalf + (kAMn ? kGHalf : boxes * p.a_rows * kGRow);
      const uint32_t bytes = !kPair ? mine : 2 * kGHalf + (kAMn || t.total > 128 ? 2 * kGHalf : kGHalf);
      for (int kc = 0; kc < t.nk; ++kc) {
        ok = __all_sync(0xffffffffu, wait(&empty[s], ph ^ 1u));
        if (!ok) break;
        uint8_t* a = smem + s * kGStage;
        uint8_t* b = a + kGHalf;
        const int k0 = t.p0 + kc * kGK;
        const bool held = kSched == Sched::Experts && ragged(t, kc);
        const uint32_t bar = held || !kPair ? smem_u32(held ? &part[s] : &full[s]) : cluster_addr(&full[s], 0);
        if (elect_one()) {
          if (held) {
            mbar_arrive_expect_tx(&part[s], mine);
          } else if (rank == 0) {  // the odd CTA's copies complete on the even one's barrier
            mbar_arrive_expect_tx(&full[s], bytes);
            if (kPair) mbar_arrive(&full[s]);
          }
          auto load = [&](void* dst, const CUtensorMap* map, int c0, int c1, int c2) {
            if (kPair)
              tma_load_3d_pair(dst, map, bar, c0, c1, c2, pol);
            else
              tma_load_3d(dst, map, held ? &part[s] : &full[s], c0, c1, c2, pol);
          };
          if (kAMn) {
            load(a, tm_a, t.m0, k0, za);
            load(a + kGHalf / 2, tm_a, t.m0 + 64, k0, za);
          } else {
            for (int i = 0; i < boxes; ++i) load(a + i * p.a_rows * kGRow, tm_a, k0, t.m0 + i * p.a_rows, za);
          }
          if (kBMn) {
            load(b, tm_b, t.n0 + 128 * r, k0, zb);
            load(b + kGHalf / 2, tm_b, t.n0 + 128 * r + 64, k0, zb);
          } else if (kEpi == Epi::GateUp) {
            if (kPair) {  // the even CTA holds the gate columns, the odd one the up columns
              load(b, tm_b, k0, t.n0, 2 * zb + r);
            } else {
              load(b, tm_b, k0, t.n0, 2 * zb);
              load(b + kGHalf / 2, tm_b, k0, t.n0, 2 * zb + 1);
            }
          } else {
            load(b, tm_b, k0, t.n0 + 128 * r, zb);
          }
        }
        __syncwarp();
        if (++s == kStages) { s = 0; ph ^= 1u; }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer
    constexpr uint32_t kIdesc = idesc_f16(tile_m(kPair), kN, kBf16, kAMn, kBMn);
    int s = 0, acc_it = 0;
    uint32_t ph = 0;
    bool ok = rank == 0;
    bool more = ok && walk.next(&t);
    while (more) {
      const Tile now = t;
      if (now.nk == 0) {
        more = walk.next(&t);
        continue;
      }
      const int buf = acc_it & 1;
      ok = __all_sync(0xffffffffu, wait_cluster(&acc_empty[buf], ((acc_it >> 1) & 1) ^ 1u));
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tbase + static_cast<uint32_t>(buf) * kN;
      for (int kc = 0; kc < now.nk; ++kc) {
        const bool cut = kSched == Sched::Experts && ragged(now, kc);
        ok = __all_sync(0xffffffffu, cut ? wait_cluster(&full[s], ph) : wait(&full[s], ph));
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = smem_u32(smem + s * kGStage), b = a + kGHalf;
        const uint64_t ad = kAMn ? sdesc_sw128_mn(a, kGHalf / 2) : sdesc_sw128(a);
        const uint64_t bd = kBMn ? sdesc_sw128_mn(b, kGHalf / 2) : sdesc_sw128(b);
        // whole steps without a routed row are left out
        const int steps = cut ? (now.rows - kc * kGK + 15) / 16 : kGK / 16;
        // 16 contraction indices: 32 bytes of a K-major row, 16 rows of an MN-major one.  A predicated issue is the
        // faster one for single CTAs (a chunk of 128 x 128 in 232 cycles of this warp, behind a branch 344), but not
        // for pairs, whose MMAs take longer than their issue (up, 8192 tokens on 64 experts: 454 us, 440 behind it).
        constexpr uint32_t kStepA = kAMn ? 128 : 2, kStepB = kBMn ? 128 : 2;
        if (kPair) {
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kGK / 16; ++kk)
              if (kSched != Sched::Experts || kk < steps)
                mma_f16_pair(d, ad + kStepA * kk, bd + kStepB * kk, kIdesc, (kc | kk) != 0);
            tc_commit_pair(&empty[s]);
            if (kc + 1 == now.nk) tc_commit_pair(&acc_full[buf]);
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < kGK / 16; ++kk)
            if (kSched != Sched::Experts || kk < steps)
              mma_f16_one(d, ad + kStepA * kk, bd + kStepB * kk, kIdesc, (kc | kk) != 0);
          tc_commit_one(&empty[s]);
          if (kc + 1 == now.nk) tc_commit_one(&acc_full[buf]);
        }
        __syncwarp();
        if (++s == kStages) { s = 0; ph ^= 1u; }
        if (kc == 0) more = walk.next(&t);  // beside the MMAs
      }
      if (!ok) break;
      ++acc_it;
    }
  } else if (warp == kGPatchWarp) {
    // ------------------------------------------------ rows behind the routed ones
    // Padding, or another expert's rows, in an expert's last chunk become
    // zeros (a product with zero would keep a NaN), up to the MMA's next 16.
    if (kSched == Sched::Experts) {
      int count = 0;      // chunks so far
      uint32_t seen = 0;  // parity of part[s], one bit a stage
      bool ok = true;
      while (ok && walk.next(&t)) {
        if (t.nk > 0 && ragged(t, t.nk - 1)) {
          const int s = (count + t.nk - 1) % kStages;
          ok = wait(&part[s], (seen >> s) & 1u);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          seen ^= 1u << s;
          const int rem = t.rows - (t.nk - 1) * kGK;
          const int gap = (rem + 15) / 16 * 16 - rem;
          uint8_t* base = smem + s * kGStage;  // A, B: two boxes each of 64 rows of 128 bytes
          for (int i = lane; i < 4 * gap * 8; i += 32) {
            const int box = i / (gap * 8), r = i - box * (gap * 8);
            *reinterpret_cast<uint4*>(base + box * (kGHalf / 2) + (rem + r / 8) * kGRow + (r & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (kPair)
              mbar_arrive_release(cluster_addr(&full[s], 0));
            else
              mbar_arrive(&full[s]);
          }
        }
        count += t.nk;
      }
    }
  } else {
    // ------------------------------------------------ epilogue
    // Warp w reads TMEM lanes 32 (w % 4) .. + 31, a row a thread, and half of
    // the tile's columns, in pieces that fill a staging buffer.
    const int q = warp & 3, hf = (warp - 2) >> 2;
    const int r = 32 * q + lane;
    constexpr int kHalfCols = kN / 2;
    const uint32_t stg0 = smem_u32(smem + kStaging + (warp - 2) * 2 * kBuf);
    uint64_t* side = side_full + (warp - 2) * 2;
    int piece = 0;  // pieces so far; piece % 2 is the buffer
    auto buffer = [&] { return stg0 + static_cast<uint32_t>(piece & 1) * kBuf; };
    // 16 bytes of this thread's row of a staging tile, swizzled as its tensor map says
    auto at64 = [&](int tile, int i) { return buffer() + tile * kGTile + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4); };
    auto put = [&](uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
    };
    auto get = [&](uint32_t at, uint32_t (&v)[4]) {
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                   : "r"(at)
                   : "memory");
    };
    // a 32 x 32 piece in fp16 (w: this row's pairs) into a tile of the buffer, transposed: lanes 2i and
    // 2i + 1 exchange halves and write a pair each, to rows 2j and 2j + 1, without bank conflicts
    auto put_transposed = [&](int tile, const uint32_t (&w)[16]) {
      const bool odd = lane & 1;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const uint32_t other = __shfl_xor_sync(0xffffffffu, w[j], 1);
        const uint32_t pair = odd ? __byte_perm(other, w[j], 0x7632) : __byte_perm(w[j], other, 0x5410);
        const uint32_t at = buffer() + tile * kGTile + (2 * j + (odd ? 1 : 0)) * 64 + (((lane >> 3) ^ (j & 3)) << 4) + ((lane >> 1) & 3) * 4;
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(pair) : "memory");
      }
    };
    // the buffer about to be filled was last stored from two pieces ago
    auto buffer_free = [&] {
      if (lane == 0) bulk_wait_read<1>();
      __syncwarp();
    };
    // a tile of the buffer to `map`: this warp's rows below the limit, boxes of store_rows
    auto store = [&](const CUtensorMap* map, int tile, int c0, int c1, bool row_last) {
      for (int i = 0; i < 32; i += p.store_rows) {
        if (32 * q + i >= t.limit) break;
        const uint32_t src = buffer() + tile * kGTile + i * 64;
        const int row = t.m0 + 32 * q + i;
        if (kEpi == Epi::Weights && p.accumulate)
          tma_add_3d(map, src, c0, row, c1);
        else if (row_last)
          tma_store_3d(map, src, c0, c1, row);
        else
          tma_store_3d(map, src, c0, row, c1);
      }
    };
    auto stored = [&](auto f) {  // fills done by the lanes; f: the stores, by one
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        f();
        bulk_commit();
      }
      ++piece;
    };
    // Side tiles of the 32-column piece `col` into buffer b: from tm_c and tm_c2,
    // except h, whose gate and up halves are two planes of one map.
    auto side_load = [&](int b, int col) {
      if (lane == 0) {
        bulk_wait_read<0>();
        int boxes = 0;
        for (int i = 0; i < 32 && 32 * q + i < t.limit; i += p.store_rows) ++boxes;
        mbar_arrive_expect_tx(&side[b], boxes * p.store_rows * 64 * kSideTiles);
        const uint64_t pol = policy_evict_normal();
        for (int i = 0; i < boxes; ++i) {
          const int row = t.m0 + 32 * q + i * p.store_rows;
          uint8_t* dst = smem + kStaging + (warp - 2) * 2 * kBuf + b * kBuf + i * p.store_rows * 64;
          if (kEpi == Epi::SwigluGrad) {
            tma_load_3d(dst, tm_c, &side[b], col, 0, row, pol);
            tma_load_3d(dst + kGTile, tm_c, &side[b], col, 1, row, pol);
          } else {
            tma_load_3d(dst, tm_c, &side[b], col, row, t.z, pol);
            if (kSideTiles == 2) tma_load_3d(dst + kGTile, tm_c2, &side[b], col, row, t.z, pol);
          }
        }
      }
      __syncwarp();
    };
    int acc_it = 0;
    uint32_t side_ph = 0;  // parity of side[b], a bit each
    bool ok = true;
    while (ok && walk.next(&t)) {
      if (t.nk == 0 && p.accumulate) continue;
      const bool rows_here = 32 * q < t.limit;  // warp-uniform
      const int col0 = t.n0 + (kEpi == Epi::GateUp ? hf * (kHalfCols / 2) : hf * kHalfCols);
      bool mine = r < t.limit;  // this thread's row carries a value (a padding row: zeros)
      if (kSched == Sched::Blocks && mine) mine = __ldg(p.sorted_ids + static_cast<int64_t>(t.m0) + r) >= 0;
      // the first piece, while the MMAs run, or both of a single CTA (of a pair a second one only adds to the load:
      // 228 us an update of 16 x 2048 x 2048, 212 without)
      if (kSide && rows_here) {
        if (col0 < p.n_total) side_load(piece & 1, col0);
        if (!kPair && col0 + 32 < p.n_total) side_load((piece & 1) ^ 1, col0 + 32);
      }
      const int buf = acc_it & 1;
      if (t.nk > 0) {
        ok = wait(&acc_full[buf], (acc_it >> 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
      }
      const uint32_t tacc = tbase + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(buf) * kN;
      auto acc32 = [&](int col, uint32_t (&v)[32]) {  // 32 columns of the accumulator, zeros without one
        if (kSched != Sched::Experts || t.nk > 0) {
          tmem_ld32(tacc + col, v);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0;
        }
      };
      if (rows_here) {
        if (kEpi == Epi::GateUp) {
#pragma unroll 1
          for (int c = 0; c < kHalfCols / 64; ++c) {
            const int col = col0 + 32 * c, ac = hf * (kHalfCols / 2) + 32 * c;
            if (col >= p.n_total) break;
            uint32_t g[32], up[32];
            tmem_ld32(tacc + ac, g);
            tmem_ld32(tacc + kN / 2 + ac, up);
            tmem_ld_wait();
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              buffer_free();
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const int e = 8 * i + 2 * j;
                  w[j] = mine ? pack_b16(__uint_as_float(half ? up[e] : g[e]), __uint_as_float(half ? up[e + 1] : g[e + 1])) : 0u;
                }
                put(at64(0, i), w[0], w[1], w[2], w[3]);
              }
              stored([&] { store(tm_d, 0, col, half, true); });
            }
            buffer_free();
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
              put(at64(0, i), w[0], w[1], w[2], w[3]);
            }
            stored([&] { store(tm_d2, 0, col, 0, false); });
          }
        } else if (kSide) {
#pragma unroll 1
          for (int c = 0; c < kHalfCols / 32; ++c) {
            const int col = col0 + 32 * c;
            if (col >= p.n_total) break;
            const int b = piece & 1;
            if ((kPair || c > 0) && c + 1 < kHalfCols / 32 && col + 32 < p.n_total) side_load(b ^ 1, col + 32);
            uint32_t v[32];
            acc32(hf * kHalfCols + 32 * c, v);
            ok = mbar_wait(&side[b], (side_ph >> b) & 1u, abort_flag, p.status, p.wait_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            side_ph ^= 1u << b;
            if (kEpi == Epi::SwigluGrad) {
              // act = gate s(gate) up, s the sigmoid: d act / d gate = up s (1 + gate (1 - s)), d act / d up = gate s
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t gw[4], uw[4], og[4], ou[4];
                get(at64(0, i), gw);
                get(at64(1, i), uw);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float2 g2 = unpack_b16(gw[j]), u2 = unpack_b16(uw[j]);
                  float dg[2], du[2];
#pragma unroll
                  for (int k = 0; k < 2; ++k) {
                    const float g = k ? g2.y : g2.x, up = k ? u2.y : u2.x;
                    const float ga = __uint_as_float(v[8 * i + 2 * j + k]);
                    const float sg = __fdividef(1.0f, 1.0f + __expf(-g));
                    dg[k] = ga * up * sg * fmaf(g, 1.0f - sg, 1.0f);
                    du[k] = ga * g * sg;
                  }
                  og[j] = mine ? pack_b16(dg[0], dg[1]) : 0u;
                  ou[j] = mine ? pack_b16(du[0], du[1]) : 0u;
                }
                put(at64(0, i), og[0], og[1], og[2], og[3]);
                put(at64(1, i), ou[0], ou[1], ou[2], ou[3]);
              }
              stored([&] {
                store(tm_d, 0, col, 0, true);
                store(tm_d, 1, col, 1, true);
              });
            } else if (kEpi == Epi::Poly) {
              uint32_t w[16];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t cw[4];
                get(at64(0, i), cw);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float2 c2 = unpack_f16(cw[j]);
                  float o[2];
#pragma unroll
                  for (int k = 0; k < 2; ++k) {
                    const int e = 8 * i + 2 * j + k;
                    o[k] = fmaf(p.beta, k ? c2.y : c2.x, p.alpha * __uint_as_float(v[e]));
                    if (p.use_diag && col + e == t.m0 + r) {
                      if (mine) p.diag[static_cast<int64_t>(t.z) * p.side + t.m0 + r] = o[k];
                      o[k] = 0.f;
                    }
                  }
                  w[4 * i + j] = pack_f16(o[0], o[1]);
                }
                put(at64(0, i), w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
              }
              if (t.mirror) put_transposed(1, w);
              stored([&] {
                store(tm_d, 0, col, t.z, false);
                if (t.mirror) tma_store_3d(tm_d, buffer() + kGTile, t.m0 + 32 * q, col, t.z);
              });
            } else {
              const float* diag = p.diag + static_cast<int64_t>(t.z) * p.side;
              float coef = p.alpha;
              if (p.use_diag && !p.tall && mine) coef += __ldcg(diag + t.m0 + r);
              // column col + lane's term of the tall form, handed round below
              const float dcol = p.use_diag && p.tall ? __ldcg(diag + min(col + lane, p.side - 1)) : 0.f;
              float y[32];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t hw[4], lw[4];
                get(at64(0, i), hw);
                get(at64(1, i), lw);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float2 h2 = unpack_f16(hw[j]), l2 = unpack_f16(lw[j]);
#pragma unroll
                  for (int k = 0; k < 2; ++k) {
                    const int e = 8 * i + 2 * j + k;
                    const float x = fmaf(k ? l2.y : l2.x, 1.0f / kLoScale, k ? h2.y : h2.x);
                    y[e] = fmaf(coef + __shfl_sync(0xffffffffu, dcol, e), x, __uint_as_float(v[e]));
                  }
                }
              }
              if (p.last && p.direct) {
                __nv_bfloat16* dst = p.out + (static_cast<int64_t>(t.z) * p.m_total + t.m0 + r) * p.n_total + col;
                if (mine) {
#pragma unroll
                  for (int e = 0; e < 32; ++e)
                    if (col + e < p.n_total) dst[e] = __float2bfloat16_rn(y[e] * p.beta);
                }
                __syncwarp();  // the buffer is loaded into again
                ++piece;
              } else if (p.last) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  uint32_t w[4];
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                    w[j] = pack_b16(y[8 * i + 2 * j] * p.beta, y[8 * i + 2 * j + 1] * p.beta);
                  put(at64(0, i), w[0], w[1], w[2], w[3]);
                }
                stored([&] { store(tm_d, 0, col, t.z, false); });
              } else {
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
                  put(at64(0, i), wh[0], wh[1], wh[2], wh[3]);
                  put(at64(1, i), wl[0], wl[1], wl[2], wl[3]);
                }
                stored([&] {
                  store(tm_d, 0, col, t.z, false);
                  store(tm_d2, 1, col, t.z, false);
                });
              }
            }
          }
        } else if (kEpi == Epi::Weights && p.out_f32) {
#pragma unroll 1
          for (int c = 0; c < kHalfCols / 32; ++c) {
            const int col = col0 + 32 * c;
            if (col >= p.n_total) break;
            uint32_t v[32];
            acc32(hf * kHalfCols + 32 * c, v);
#pragma unroll
            for (int half = 0; half < 2; ++half) {  // 16 columns of fp32 a tile
              if (col + 16 * half >= p.n_total) break;
              buffer_free();
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int e = 16 * half + 4 * i;
                put(at64(0, i), v[e], v[e + 1], v[e + 2], v[e + 3]);
              }
              stored([&] { store(tm_d, 0, col + 16 * half, t.z, false); });
            }
          }
        } else if (kEpi == Epi::Gram) {
#pragma unroll 1
          for (int c = 0; c < kHalfCols / 32; ++c) {
            const int col = col0 + 32 * c;
            if (col >= p.n_total) break;
            uint32_t v[32], w[16];
            acc32(hf * kHalfCols + 32 * c, v);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              w[i] = pack_f16(p.alpha * __uint_as_float(v[2 * i]), p.alpha * __uint_as_float(v[2 * i + 1]));
            buffer_free();
#pragma unroll
            for (int i = 0; i < 4; ++i) put(at64(0, i), w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            stored([&] { store(tm_d, 0, col, t.z, false); });
            if (t.mirror) {
              buffer_free();
              put_transposed(0, w);
              stored([&] { tma_store_3d(tm_d, buffer(), t.m0 + 32 * q, col, t.z); });
            }
          }
        } else {  // Rows, Weights in bf16
#pragma unroll 1
          for (int c = 0; c < kHalfCols / 32; ++c) {
            const int col = col0 + 32 * c;
            if (col >= p.n_total) break;
            uint32_t v[32];
            acc32(hf * kHalfCols + 32 * c, v);
            buffer_free();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int e = 8 * i + 2 * j;
                w[j] = mine ? pack_b16(__uint_as_float(v[e]), __uint_as_float(v[e + 1])) : 0u;
              }
              put(at64(0, i), w[0], w[1], w[2], w[3]);
            }
            stored([&] { store(tm_d, 0, col, kSched == Sched::Blocks ? 0 : t.z, false); });
          }
        }
        if (!ok) break;
      }
      if (t.nk > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (kPair)
            mbar_arrive_relaxed(cluster_addr(&acc_empty[buf], 0));
          else
            mbar_arrive(&acc_empty[buf]);
        }
        ++acc_it;
      }
    }
    if (lane == 0) bulk_wait_all();
  }
}


template <Form kForm, Sched kSched, Epi kEpi, bool kPair, bool kBf16>
__global__ void __launch_bounds__(kGThreads, 1)
    tile_gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                     const __grid_constant__ CUtensorMap tm_d, const __grid_constant__ CUtensorMap tm_d2,
                     const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_c2,
                     const __grid_constant__ GemmParams p) {
  constexpr int kStages = gemm_stages(kSched, kEpi), kBuf = gemm_buf(kEpi);
  extern __shared__ uint8_t smem_raw[];
  TileCta c;
  pdl_launch_dependents();
  tile_cta_setup<kStages, kBuf, kPair>(&c, smem_raw);
  if (threadIdx.x == 0) {
    prefetch_tmap(&tm_a);
    prefetch_tmap(&tm_b);
    prefetch_tmap(&tm_d);
    if (epi_side(kEpi)) prefetch_tmap(&tm_c);
  }
  int* first = reinterpret_cast<int*>(c.smem + gemm_ctrl(kSched, kEpi) + kGCtrlBytes);
  int blocks = 0;
  if (kSched != Sched::Batch) {  // the plan, which no launch that this one may overlap has written
    const int n = __ldg(p.ntpp) / p.bm;
    blocks = n < 0 ? 0 : min(n, p.max_blocks);
    if (kSched == Sched::Experts) find_segments(p, blocks, first);
  }
  tile_cta_ready<kPair>(&c);
  if (kSched == Sched::Batch) pdl_wait();  // what a chained launch before this one wrote is read below
  const int at = static_cast<int>(blockIdx.x), of = static_cast<int>(gridDim.x);
  Walk<kSched, kEpi, kPair> walk(p, static_cast<int>(c.rank), kPair ? at / 2 : at, kPair ? of / 2 : of, blocks, first);
  tile_product<kForm, kSched, kEpi, kPair, kBf16, kStages, kBuf>(c, walk, &tm_a, &tm_b, &tm_d, &tm_d2, &tm_c, &tm_c2, p);
  // a weight gradient runs beside the product launched before it, which it does not depend on, but does not end
  // before it: what follows on the stream waits for both
  if (kSched == Sched::Experts) pdl_wait();
  tile_cta_leave<kPair>(c);
}

// ------------------------------------------------------------------ host side
// 3-D tensor map over 16-bit (or fp32) elements: dims d0 (contiguous), d1, d2
// with strides s1, s2 in bytes.  A box row of 128 or 64 bytes names the swizzle.
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

struct GemmMaps {
  CUtensorMap a, b, d, d2, c, c2;
};

// Launches one product of at most max_tiles tiles; pdl: chained to the launch before it.
template <Form kForm, Sched kSched, Epi kEpi, bool kPair, bool kBf16>
int launch_tile_gemm(const char* nm, const GemmMaps& m, const GemmParams& p, int64_t max_tiles, bool pdl,
                     cudaStream_t stream) {
  auto kernel = tile_gemm_kernel<kForm, kSched, kEpi, kPair, kBf16>;
  static std::atomic<bool> attr_set[kMaxDevices];  // per device; setting it twice is harmless
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cuda_fail("cudaGetDevice");
  if (dev >= kMaxDevices || !attr_set[dev].load(std::memory_order_relaxed)) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, gemm_smem(kSched, kEpi));
    if (e != cudaSuccess) return cuda_fail(nm, e);
    if (dev < kMaxDevices) attr_set[dev].store(true, std::memory_order_relaxed);
  }
  const int nsm = sm_count();
  if (nsm <= 0) return cuda_fail("cudaDeviceGetAttribute(SM count)");
  const int64_t slots = kPair ? nsm / 2 : nsm;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (kPair) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = 2;
    attr[n].val.clusterDim.y = 1;
    attr[n++].val.clusterDim.z = 1;
  }
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(static_cast<unsigned>((max_tiles < slots ? max_tiles : slots) * (kPair ? 2 : 1)), 1, 1);
  c.blockDim = dim3(kGThreads, 1, 1);
  c.dynamicSmemBytes = gemm_smem(kSched, kEpi);
  c.stream = stream;
  c.attrs = attr;
  c.numAttrs = n;
  const cudaError_t err = cudaLaunchKernelEx(&c, kernel, m.a, m.b, m.d, m.d2, m.c, m.c2, p);
  return err == cudaSuccess ? MOE_OK : cuda_fail(nm, err);
}

}  // namespace moe
