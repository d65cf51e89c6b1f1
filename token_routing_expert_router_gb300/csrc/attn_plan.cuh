// The order of a ragged batch's tiles (attn_plan.cu), for the kernels that take them.
#pragma once

#include "attn.cuh"

namespace moe {
namespace attn {

struct TileEntry {
  int q0, n, k0, m;  // the sequence's rows
  int start;         // the tile's first query or key
  int lo, hi;        // its inner tiles
  int cut;           // 0: whole; else a piece: first place of its pieces << 16 | its number << 8 | their count
};
struct TilePlan {
  int count, pad[7];
  TileEntry tile[1];
};
inline size_t plan_bytes(int64_t tiles) { return align_up(32 + (size_t)tiles * sizeof(TileEntry), 256); }

struct PlanJob {
  int keys;          // tiles of 128 keys (dk, dv), or of `rows` queries
  int rows;
  int inner, packs;  // keys: queries of an inner tile, packs of heads
  int heads;         // what the tiles are done for: packs of heads, or key heads
  int pieces;        // 0, or cut tiles so that about this many pieces come of all heads' tiles
  int most;          // entries that there is room for, without the cuts
  TilePlan* plan;
  int* first;        // [B + 1]: tiles of the sequences before
};
struct StatsJob {
  int pack;
  float *neg_lse, *neg_delta;  // [Hq / pack][Tq][pack]
};
cudaError_t launch_plan(const AttnArgs& a, const PlanJob& j, cudaStream_t s);
cudaError_t launch_plan_backward(const AttnArgs& a, const PlanJob& dq, const PlanJob& dkv, const StatsJob& st, cudaStream_t s);

// Block id -> the tile's place in the order and the head: chunks of heads whose operands stay in L2 one
// behind the other, in a chunk every head's longest tile, then every head's next.
struct Place {
  int rank, head;
};
__device__ __forceinline__ Place place_of(int id, int tiles, int heads, int chunk) {
  const int c = id / (chunk * tiles), r = id - c * chunk * tiles, in = min(chunk, heads - c * chunk);
  return Place{r / in, c * chunk + r % in};
}
inline int head_chunk(int64_t bytes, int heads) {
  const int64_t n = ((int64_t)64 << 20) / (bytes > 0 ? bytes : 1);
  return (int)(n < 1 ? 1 : n > heads ? heads : n);
}

}  // namespace attn
}  // namespace moe
