// What the attention kernels share (attn_*.cu): the arguments as the device sees them, a sequence's rows,
// and the map from a block to the tile of a ragged batch.
#pragma once

#include "step.cuh"

namespace moe {
namespace attn {

struct AttnArgs {
  int Tq, Tk, B, Hq, Hkv, D, group;  // group: query heads of a key head
  int causal, max_q;
  float scale;
  int64_t ld_q, ld_k, ld_v, ld_o;
  const void *q, *k, *v;
  const int32_t *q_start, *k_start, *k_len;
  void* o;
  float* lse;
  // backward
  const void* d_o;
  void *dq, *dk, *dv;
  float* delta;  // [Hq, Tq]: do . o of every query row and head
  DeviceStatus* status;
};

struct Seq {
  int q0, n;  // query rows [q0, q0 + n)
  int k0, m;  // key rows [k0, k0 + m)
};

// Sequence b, with what is out of range left out: no rows for query rows that are not inside q or
// more than max_q, no keys for key rows that are not inside k.
__device__ __forceinline__ Seq load_seq(const AttnArgs& a, int b, bool report) {
  Seq s;
  s.q0 = __ldg(a.q_start + b);
  const int q1 = __ldg(a.q_start + b + 1);
  bool bad = s.q0 < 0 || q1 < s.q0 || q1 > a.Tq || q1 - s.q0 > a.max_q;
  s.n = bad ? 0 : q1 - s.q0;
  if (a.k_start) {
    s.k0 = __ldg(a.k_start + b);
    s.m = __ldg(a.k_len + b);
    const bool bad_k = s.k0 < 0 || s.m < 0 || s.k0 > a.Tk || s.m > a.Tk - s.k0;
    if (bad_k) s.k0 = s.m = 0;
    bad |= bad_k;
  } else {
    s.k0 = s.q0;
    s.m = s.n;
  }
  if (bad && report) set_status(a.status, MOE_ERR_DEVICE_BAD_INPUT, b);
  return s;
}

// The backward writes every key's gradient once: of the sequences in range, one whose keys begin before
// those of another in front of it end has none. end: of those in front, then of s too. True: s has lost its keys.
__device__ __forceinline__ int keys_end(const Seq& s) { return s.m > 0 ? s.k0 + s.m : 0; }
__device__ __forceinline__ bool hold_apart(Seq& s, int& end) {
  const bool lost = s.m > 0 && s.k0 < end;
  end = max(end, keys_end(s));
  if (lost) s.k0 = s.m = 0;
  return lost;
}

// The largest v (>= 0) of the threads in front of this one, and of all. Every thread calls it.
// scratch: THREADS / 32 words of shared memory, read until the next barrier.
struct Largest {
  int before, all;
};
template <int THREADS>
__device__ __forceinline__ Largest largest_before(int v, int* scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v = max(v, o);
  }
  if (lane == 31) scratch[warp] = v;
  Largest l{__shfl_up_sync(0xffffffffu, v, 1), 0};
  if (lane == 0) l.before = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) l.before = max(l.before, scratch[w]);
    l.all = max(l.all, scratch[w]);
  }
  return l;
}

struct Tile {
  int b;      // sequence, or -1: no such tile
  int index;  // of its tiles, from 0
  int count;  // of the sequence's tiles
  Seq s;
};

// The block's tile `want` of all sequences' tiles of `rows` query rows (KEYS: key rows), one after
// the other. Every thread calls it. Each thread takes the sequences of an equal share of B, the
// block scans the shares' tiles (APART: after the ends of their keys), and the thread whose share holds
// the wanted one walks it. Up to 256 sequences that is one load and two exchanges, and one more. The sums
// are 64 bits wide: sequences whose rows overlap (which is reported) may have more tiles than 32 bits count.
// The loops over the sequences are not unrolled: unrolled, they take registers and code from the short kernels
// behind them (backward of 256 tokens in fp32: 30.8 for 29.5 us).
template <int THREADS>
constexpr int kFindWords = 3 * (THREADS / 32) + 7;
template <int THREADS, bool KEYS, bool APART>
__device__ Tile find_tile(const AttnArgs& a, int64_t want, int rows, bool report, int (&scratch)[kFindWords<THREADS>]) {
  int64_t* sWarp = reinterpret_cast<int64_t*>(scratch);
  volatile int* sTile = scratch + 3 * (THREADS / 32);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int share = (a.B + THREADS - 1) / THREADS;
  const int b0 = min(a.B, tid * share), b1 = min(a.B, b0 + share);
  const Seq own = b0 < b1 ? load_seq(a, b0, report) : Seq{};  // the share's first; most often all of it
  int front = 0;  // where the keys in front of the share end
  if constexpr (APART) {
    int end = keys_end(own);
#pragma unroll 1
    for (int b = b0 + 1; b < b1; ++b) end = max(end, keys_end(load_seq(a, b, false)));
    front = largest_before<THREADS>(end, scratch + 2 * (THREADS / 32)).before;
  }
  auto tiles = [&](Seq& s, int b, int& end, bool tell) {
    s = b == b0 ? own : load_seq(a, b, tell);
    if (APART && hold_apart(s, end) && tell) set_status(a.status, MOE_ERR_DEVICE_BAD_INPUT, b);
    return ((KEYS ? s.m : s.n) + rows - 1) / rows;
  };
  int64_t mine = 0;
  int end = front;
  Seq s;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) mine += tiles(s, b, end, report);
  int64_t inc = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += o;
  }
  if (lane == 31) sWarp[warp] = inc;
  if (tid == 0) sTile[0] = -1;
  __syncthreads();
  int64_t before = inc - mine;
  for (int w = 0; w < warp; ++w) before += sWarp[w];
  if (want >= before && want < before + mine) {
    int left = (int)(want - before);
    end = front;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      const int n = tiles(s, b, end, false);
      if (left < n) {
        sTile[0] = b, sTile[1] = left, sTile[2] = n;
        sTile[3] = s.q0, sTile[4] = s.n, sTile[5] = s.k0, sTile[6] = s.m;
        break;
      }
      left -= n;
    }
  }
  __syncthreads();
  return Tile{sTile[0], sTile[1], sTile[2], Seq{sTile[3], sTile[4], sTile[5], sTile[6]}};
}

// Keys that query row i of a sequence sees: [0, visible).
__device__ __forceinline__ int visible(const AttnArgs& a, const Seq& s, int i) {
  return a.causal ? min(s.m, i + 1 + s.m - s.n) : s.m;  // may be <= 0
}

// ---- launchers of the variants
bool tc_rows(const AttnArgs& a, bool backward);  // bf16 tensors' rows are multiples of 16 bytes
struct TilePlan;  // attn_plan.cuh
// plan: room for the tiles' order; first: for B + 1 words; queue: two words of the workspace's head
cudaError_t launch_tc(const AttnArgs& a, TilePlan* plan, int* first, int* queue, cudaStream_t s);
// Few rows over many keys: one CTA an SM, each with two places for parts of lines.
constexpr int kMaxStreamCtas = 160;
inline int stream_ctas() { return tc::num_sms() < kMaxStreamCtas ? tc::num_sms() : kMaxStreamCtas; }
struct StreamSpace {
  uint32_t* tickets;  // in the workspace's head
  float2* stat;
  float* part;
};
bool stream_rule(const AttnArgs& a);
cudaError_t launch_stream(const AttnArgs& a, const StreamSpace& w, cudaStream_t s);
// Few rows over many keys, fp32: parts of lines, a line being 16 rows of a sequence and key head.
constexpr int kFewParts = 304, kMostSplits = 64;  // parts wanted of all lines, two for every SM (in turn, at 128 channels); of one, at most
constexpr int kMostFewParts = 2 * kFewParts;      // where lines are cut at all
bool few_rule(const AttnArgs& a);
cudaError_t launch_few(const AttnArgs& a, float2* stat, float* part, cudaStream_t s);
cudaError_t launch_simt(const AttnArgs& a, bool bf16, cudaStream_t s);
// What the backward keeps in the workspace beside the statistics.
struct BackwardSpace {
  TilePlan *dq_plan, *dkv_plan;
  int* first;         // [2][B + 1]
  float *neg_lse, *neg_delta;
  float* part;        // [kMostPieces][2][128][DP]: dk and dv of pieces of a tile
  uint32_t* tickets;  // [kMostPieces], zero between calls
};
constexpr int kPieces = 228;               // a cut tile of dk and dv has at most this share of all their work
constexpr int kMostPieces = 2 * kPieces;   // of tiles that are cut
cudaError_t launch_tc_backward(const AttnArgs& a, const BackwardSpace& w, cudaStream_t s);
// Entries of the plans.
int64_t forward_tiles(const AttnArgs& a);
int64_t dq_tiles(const AttnArgs& a);
int64_t dkv_tiles(const AttnArgs& a);
cudaError_t launch_simt_backward(const AttnArgs& a, bool bf16, cudaStream_t s);
cudaError_t launch_delta(const AttnArgs& a, bool bf16, cudaStream_t s);

}  // namespace attn
}  // namespace moe
