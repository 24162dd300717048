// Where each expert's blocks begin in a plan's expert_ids, as arithmetic alone
// (no CUDA, so that it can be compiled and checked on any host).
//
// first[e], 0 <= e <= E, is the first used block whose expert is >= e: the least
// b whose entries (below) hold e.  The ids of a plan ascend, and each e is then
// among the entries of one block.  Whatever else they hold, every e is among
// some block's, so first[e] is within [0, blocks] and the same wherever it is
// computed (by the CTAs of a pair, say), and an expert has no fewer than no blocks.
#pragma once

#ifdef __CUDACC__
#define MOE_SEGMENTS_FN __host__ __device__ __forceinline__
#else
#define MOE_SEGMENTS_FN inline
#endif

namespace moe {

// Entries lo .. hi of `first` that block b (0 <= b <= blocks) may be the value of: `before`
// is the id of block b - 1 (b > 0), `here` that of block b (b < blocks).
struct SegmentEntries {
  int lo, hi;
};
MOE_SEGMENTS_FN SegmentEntries segment_entries(int b, int blocks, int E, int before, int here) {
  SegmentEntries s;
  s.lo = b == 0 ? 0 : (before < -1 ? -1 : before < E ? before : E) + 1;
  s.hi = b == blocks ? E : here < E ? here : E;
  return s;
}

// Blocks of an expert whose first is `lo` and whose successor's first is `hi`.
MOE_SEGMENTS_FN int segment_blocks(int lo, int hi) { return hi > lo ? hi - lo : 0; }

}  // namespace moe
