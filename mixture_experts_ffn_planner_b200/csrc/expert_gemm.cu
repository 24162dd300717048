// The experts' products of a training step on rows in the planner's order, and
// their gradients (tile_gemm.cuh does the tiles):
//   up             h = rows w1[e]^T (N columns: gate, then up), act = silu(gate) * up       NT
//   down           y = act w2[e]^T                                                          NT
//   down_backward  grad_act = grad_y w2[e] (never stored), grad_h from it and h             NN
//                  grad_w2[e] = sum over e's rows of grad_y^T act                           TN
//   up_backward    grad_rows = grad_h w1[e]                                                 NN
//                  grad_w1[e] = sum over e's rows of grad_h^T rows                          TN
// All operands are bf16, all sums fp32 in TMEM; act and grad_h come from the
// fp32 accumulators, rounded once.
#include <algorithm>
#include <initializer_list>

#include "tile_gemm.cuh"

namespace moe {

// Pairs of CTAs take tiles of 256 x 256, single ones 128 x 128 with twice the
// bytes from L2 a flop, but four times as many tiles that end four times as
// soon.  So pairs are for tiles that are many, filled well and long.  Single
// and pair, us, each forced, on 40 experts: up at K = N = 2048, 122 and 102 with
// 192 rows an expert, 638 and 476 with 1536; down at K = 512, N = 1024 (a
// contraction of 512, 160 tiles), 24 and 25 with 384 rows, 38 and 35 with 768;
// down at K = 4096, N = 512 (256, but 1280 tiles), 72 and 64 with 384 rows.  On 8
// experts: down at K = N = 2048, 21 and 21 with 256 rows; up at K = 4096, N = 1024
// (32 tiles), 41 and 35 with 256.  On 16: up at K = 1024, N = 2048, 32 and 29 with
// 192.  The rule is a grid drawn through such points and misses some between
// them: up at K = 960, N = 2048 on 16 experts, 31 and 27 with 192 rows, 45 and 42
// with 384, runs on single CTAs until 410 rows.
// Where a row's pitch is no multiple of 128 bytes, every 128 of an operand lie
// in two lines of L2 and the bytes count for more: down at K = 1992, N = 1360,
// 56 and 47 with 128 rows, 89 and 68 with 256; up at K = 1000, N = 720, 42 and 33
// with 192; on 12 experts, down at K = 1000, N = 1360, 18 and 17 with 256; on 8, up
// at K = 1000, N = 1008, 24 and 19 with 300.
static bool pairs_for_rows(int64_t tiles, int64_t rows, int64_t contraction, bool lines) {
  if (tiles < 32 || rows < (lines ? 192 : 128)) return false;
  const int64_t least = !lines ? 80 : tiles >= 512 ? 96 : contraction >= 1000 ? 187 : 384;
  return rows * contraction >= least * 1024;
}
// Weight gradients, whose contraction is the rows, from 24 tiles' elements on; whole
// calls: up_backward at K = 4096, N = 1024 on 40 experts, 173 and 164 us with 64
// rows, 230 and 213 with 192; down_backward at K = 512, N = 1024 on 8 experts, 15
// and 15 with 64, 40 and 37 with 1536.  The elements stand for the tiles: a
// gradient that fills its tiles badly takes pairs all the same and is up to an
// eighth slower on them (up_backward at K = 4096, N = 16 on 64 experts of 256
// rows, 96 and 107; down_backward at K = 264, N = 1040 on 24 of 128, 25 and 27).
static bool pairs_for_weights(int64_t E, int64_t m, int64_t n) { return E * m * n >= 24 * 65536; }

struct ExpertCall {
  const char* nm;
  const int32_t* sorted_ids;
  const int32_t* expert_ids;
  const int32_t* ntpp;
  int64_t capacity;
  int K, N, E, bm;
  cudaStream_t stream;
};

static bool aligned16(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) % 16) return false;
  return true;
}

// Checks shared by the four calls.  `tensors`: every row and weight buffer.
static int check_expert(const ExpertCall& c, std::initializer_list<const void*> rows,
                        std::initializer_list<const void*> weights) {
  if (c.capacity < 0 || c.K <= 0 || c.N <= 0 || c.E < 1)
    return fail(MOE_ERR_INVALID_ARG, "%s: need capacity >= 0, K > 0, N > 0 and E >= 1", c.nm);
  if (!valid_block_m(c.bm)) return fail(MOE_ERR_UNSUPPORTED, "%s: block_m must be 16, 32, 64 or 128", c.nm);
  if (c.E > kMaxExperts) return fail(MOE_ERR_UNSUPPORTED, "%s: E must be <= %d", c.nm, kMaxExperts);
  if (c.K % 8 != 0 || c.N % 16 != 0)
    return fail(MOE_ERR_UNSUPPORTED, "%s: K %% 8 == 0 and N %% 16 == 0 required (K=%d N=%d)", c.nm, c.K, c.N);
  if (c.capacity >= (int64_t(1) << 31)) return fail(MOE_ERR_UNSUPPORTED, "%s: capacity must be < 2^31", c.nm);
  const int64_t tiles = (static_cast<int64_t>(std::max(c.K, c.N)) + 63) / 64;
  if (c.capacity / c.bm * tiles >= (int64_t(1) << 31) || c.E * tiles * tiles >= (int64_t(1) << 31))
    return fail(MOE_ERR_UNSUPPORTED, "%s: too many tiles", c.nm);
  bool null = !c.ntpp || (c.capacity > 0 && (!c.sorted_ids || !c.expert_ids));
  for (const void* p : weights) null |= !p;
  if (c.capacity > 0)
    for (const void* p : rows) null |= !p;
  if (null) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", c.nm);
  if (!aligned16(rows) || !aligned16(weights))
    return fail(MOE_ERR_ALIGNMENT, "%s: tensors must be 16-byte aligned", c.nm);
  if ((reinterpret_cast<uintptr_t>(c.sorted_ids) | reinterpret_cast<uintptr_t>(c.expert_ids) |
       reinterpret_cast<uintptr_t>(c.ntpp)) % 4)
    return fail(MOE_ERR_ALIGNMENT, "%s: the planner's outputs must be 4-byte aligned", c.nm);
  return MOE_OK;
}

static int base_params(const ExpertCall& c, GemmParams* p) {
  *p = GemmParams{};
  if (int rc = status_word(c.nm, &p->status)) return rc;
  p->wait_ns = kWaitTimeoutNs;
  p->sorted_ids = c.sorted_ids;
  p->expert_ids = c.expert_ids;
  p->ntpp = c.ntpp;
  p->bm = c.bm;
  p->E = c.E;
  p->max_blocks = static_cast<int>(c.capacity / c.bm);
  return MOE_OK;
}

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Row buffer (capacity, width) bf16 as an operand or an output: boxes of
// `cols` x `rows`.
static int rows_map(CUtensorMap* m, const ExpertCall& c, const void* base, int64_t width, int cols, int rows) {
  return make_map3(m, base, Elem::Bf16, width, c.capacity, 1, width * 2, c.capacity * width * 2, cols, rows, 1);
}
// The same with its halves (gate and up) apart, so that a tile that overhangs
// the gate half writes nothing into the up half.
static int halves_map(CUtensorMap* m, const ExpertCall& c, const void* base, int64_t half, int cols, int rows) {
  return make_map3(m, base, Elem::Bf16, half, 2, c.capacity, half * 2, half * 4, cols, 1, rows);
}
static int weights_map(CUtensorMap* m, const void* base, Elem el, int64_t cols, int64_t rows, int64_t n, int b0, int b1) {
  const int64_t es = el == Elem::F32 ? 4 : 2;
  return make_map3(m, base, el, cols, rows, n, cols * es, cols * rows * es, b0, b1, 1);
}

// Routed rows an expert has on average, at most: the planner's capacity is
// routes + E (block_m - 1).
static int64_t mean_rows(const ExpertCall& c) {
  return std::max<int64_t>(0, c.capacity - static_cast<int64_t>(c.E) * (c.bm - 1)) / c.E;
}

// rows of `width_in` times the expert's weights, into rows of width_out.
template <Form kForm, Epi kEpi, bool kPair>
static int blocks_tiled(const ExpertCall& c, const void* in, int64_t width_in, const void* w, int64_t w_cols,
                        int64_t w_rows, int64_t width_out, void* out, void* out2, const void* h) {
  GemmParams p;
  if (int rc = base_params(c, &p)) return rc;
  constexpr int kCols = kEpi == Epi::GateUp ? tile_n(kPair) / 2 : tile_n(kPair);
  p.n_total = static_cast<int>(width_out);
  p.n_tiles = static_cast<int>(ceil_div(width_out, kCols));
  p.nk = static_cast<int>(ceil_div(width_in, kGK));
  p.store_rows = std::min(c.bm, 32);
  GemmMaps m;
  p.a_rows = kPair ? 128 : 32;
  int rc = rows_map(&m.a, c, in, width_in, kGK, p.a_rows);
  if (rc == MOE_OK) {
    if (kForm == Form::NN)
      rc = weights_map(&m.b, w, Elem::Bf16, w_cols, w_rows, c.E, 64, kGK);
    else if (kEpi == Epi::GateUp)
      rc = weights_map(&m.b, w, Elem::Bf16, w_cols, w_rows / 2, 2 * static_cast<int64_t>(c.E), kGK, kPair ? 128 : 64);
    else
      rc = weights_map(&m.b, w, Elem::Bf16, w_cols, w_rows, c.E, kGK, 128);
  }
  if (rc == MOE_OK) {
    if (kEpi == Epi::Rows)
      rc = rows_map(&m.d, c, out, width_out, 32, p.store_rows);
    else
      rc = halves_map(&m.d, c, out, width_out, 32, p.store_rows);
  }
  m.d2 = m.c = m.c2 = m.d;
  if (rc == MOE_OK && kEpi == Epi::GateUp) rc = rows_map(&m.d2, c, out2, width_out, 32, p.store_rows);
  if (rc == MOE_OK && kEpi == Epi::SwigluGrad) rc = halves_map(&m.c, c, h, width_out, 32, p.store_rows);
  if (rc != MOE_OK) return rc;
  return launch_tile_gemm<kForm, Sched::Blocks, kEpi, kPair, true>(
      c.nm, m, p, static_cast<int64_t>(p.max_blocks) * p.n_tiles, false, c.stream);
}

// cols: columns of the product.
template <Form kForm, Epi kEpi, typename... Args>
static int run_blocks(const ExpertCall& c, int64_t cols, const void* in, int64_t width_in, Args... args) {
  if (c.capacity / c.bm == 0) return MOE_OK;
  const int64_t rows = mean_rows(c);
  const bool lines = width_in % 64 == 0 && (kForm != Form::NN || cols % 64 == 0);
  return pairs_for_rows(c.E * ceil_div(rows, 256) * ceil_div(cols, 256), rows, width_in, lines)
             ? blocks_tiled<kForm, kEpi, true>(c, in, width_in, args...)
             : blocks_tiled<kForm, kEpi, false>(c, in, width_in, args...);
}

// grad[e] (m x n) = sum over e's rows of a^T b, a (capacity, m), b (capacity, n).  Launched to run beside the rows'
// gradient before it (which is launched where there is a block): its CTAs take the SMs that run out of tiles there.
template <bool kPair>
static int weights_tiled(const ExpertCall& c, const void* a, int64_t m, const void* b, int64_t n, void* grad, int f32,
                         int accumulate) {
  GemmParams p;
  if (int rc = base_params(c, &p)) return rc;
  p.batches = c.E;
  p.m_total = static_cast<int>(m);
  p.n_total = static_cast<int>(n);
  p.m_tiles = static_cast<int>(ceil_div(m, tile_m(kPair)));
  p.n_tiles = static_cast<int>(ceil_div(n, tile_n(kPair)));
  p.store_rows = 32;
  p.out_f32 = f32;
  p.accumulate = accumulate;
  GemmMaps t;
  ExpertCall one = c;  // a tensor map needs at least one row; without capacity no row is read
  one.capacity = std::max<int64_t>(c.capacity, 1);
  int rc = rows_map(&t.a, one, c.capacity ? a : grad, m, 64, kGK);
  if (rc == MOE_OK) rc = rows_map(&t.b, one, c.capacity ? b : grad, n, 64, kGK);
  if (rc == MOE_OK) rc = weights_map(&t.d, grad, f32 ? Elem::F32 : Elem::Bf16, n, m, c.E, f32 ? 16 : 32, 32);
  if (rc != MOE_OK) return rc;
  t.d2 = t.c = t.c2 = t.d;
  return launch_tile_gemm<Form::TN, Sched::Experts, Epi::Weights, kPair, true>(
      c.nm, t, p, static_cast<int64_t>(c.E) * p.m_tiles * p.n_tiles, c.capacity / c.bm > 0, c.stream);
}

static int run_weights(const ExpertCall& c, const void* a, int64_t m, const void* b, int64_t n, void* grad, int f32,
                       int accumulate) {
  return pairs_for_weights(c.E, m, n)
             ? weights_tiled<true>(c, a, m, b, n, grad, f32, accumulate)
             : weights_tiled<false>(c, a, m, b, n, grad, f32, accumulate);
}

static int check_grad(const ExpertCall& c, int dtype, int accumulate) {
  if (dtype != MOE_ROWS_BF16 && dtype != MOE_ROWS_FP32)
    return fail(MOE_ERR_UNSUPPORTED, "%s: a weight gradient must be bf16 or fp32", c.nm);
  if (accumulate && dtype != MOE_ROWS_FP32)
    return fail(MOE_ERR_UNSUPPORTED, "%s: accumulating needs an fp32 weight gradient", c.nm);
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" int moe_expert_up(const void* rows, const void* w1, const int32_t* sorted_token_ids,
                             const int32_t* expert_ids, const int32_t* num_tokens_post_padded, int64_t capacity,
                             int K, int N, int E, int block_m, void* h, void* act, moe_stream_t stream) {
  const ExpertCall c{"moe_expert_up", sorted_token_ids, expert_ids, num_tokens_post_padded, capacity, K, N, E, block_m,
                     reinterpret_cast<cudaStream_t>(stream)};
  if (int rc = check_expert(c, {rows, h, act}, {w1})) return rc;
  return run_blocks<Form::NT, Epi::GateUp>(c, N, rows, K, w1, K, N, N / 2, h, act, nullptr);
}

extern "C" int moe_expert_down(const void* act, const void* w2, const int32_t* sorted_token_ids,
                               const int32_t* expert_ids, const int32_t* num_tokens_post_padded, int64_t capacity,
                               int K, int N, int E, int block_m, void* y, moe_stream_t stream) {
  const ExpertCall c{"moe_expert_down", sorted_token_ids, expert_ids, num_tokens_post_padded, capacity, K, N, E,
                     block_m, reinterpret_cast<cudaStream_t>(stream)};
  if (int rc = check_expert(c, {act, y}, {w2})) return rc;
  return run_blocks<Form::NT, Epi::Rows>(c, K, act, N / 2, w2, N / 2, K, K, y, nullptr, nullptr);
}

extern "C" int moe_expert_down_backward(const void* grad_y, const void* h, const void* act, const void* w2,
                                        const int32_t* sorted_token_ids, const int32_t* expert_ids,
                                        const int32_t* num_tokens_post_padded, int64_t capacity, int K, int N, int E,
                                        int block_m, void* grad_h, void* grad_w2, int grad_dtype, int accumulate,
                                        moe_stream_t stream) {
  const ExpertCall c{"moe_expert_down_backward", sorted_token_ids, expert_ids, num_tokens_post_padded, capacity, K, N,
                     E, block_m, reinterpret_cast<cudaStream_t>(stream)};
  if (int rc = check_grad(c, grad_dtype, accumulate)) return rc;
  if (int rc = check_expert(c, {grad_y, h, act, grad_h}, {w2, grad_w2})) return rc;
  if (int rc = run_blocks<Form::NN, Epi::SwigluGrad>(c, N / 2, grad_y, K, w2, N / 2, K, N / 2, grad_h, nullptr, h))
    return rc;
  return run_weights(c, grad_y, K, act, N / 2, grad_w2, grad_dtype == MOE_ROWS_FP32, accumulate);
}

extern "C" int moe_expert_up_backward(const void* grad_h, const void* rows, const void* w1,
                                      const int32_t* sorted_token_ids, const int32_t* expert_ids,
                                      const int32_t* num_tokens_post_padded, int64_t capacity, int K, int N, int E,
                                      int block_m, void* grad_rows, void* grad_w1, int grad_dtype, int accumulate,
                                      moe_stream_t stream) {
  const ExpertCall c{"moe_expert_up_backward", sorted_token_ids, expert_ids, num_tokens_post_padded, capacity, K, N, E,
                     block_m, reinterpret_cast<cudaStream_t>(stream)};
  if (int rc = check_grad(c, grad_dtype, accumulate)) return rc;
  if (int rc = check_expert(c, {grad_h, rows, grad_rows}, {w1, grad_w1})) return rc;
  if (int rc = run_blocks<Form::NN, Epi::Rows>(c, K, grad_h, N, w1, K, N, K, grad_rows, nullptr, nullptr)) return rc;
  return run_weights(c, grad_h, N, rows, K, grad_w1, grad_dtype == MOE_ROWS_FP32, accumulate);
}
