// Token embedding and its gradient.
//   out[t] = scale * table[token[t]]                          (a negative token: a zero row)
//   dtable[v] = scale * sum over t with token[t] = v of dout[t], positions ascending
//
// The gradient has no atomics, so its bits do not depend on timing. The positions are sorted
// by (token, position): blocks sort 2048 tokens each in shared memory as one 32-bit key
// (token << 11 | position in the block), then every element of a run of blocks finds its place as
// its own index plus, by binary search, the number of smaller keys in each other block, and runs
// of those are merged eight at a time in the same way. (Every block against every other in one
// launch is quadratic: the whole gradient of 131072 tokens of 8 channels took 131 us, of 4 million
// 31.9 ms.)
// The sums then go over equal chunks of the sorted positions, whatever the tokens' frequencies:
// a token whose run lies inside a chunk is written at once, one that crosses chunks leaves one
// partial sum per chunk, and join_kernel adds those in order. Rows of tokens that do not occur
// are zeroed by further blocks of the same launch. Everything is bound by DRAM: dout is read
// once, dtable written once.
#include <algorithm>
#include <type_traits>

#include "step.cuh"

namespace moe {
namespace {

constexpr int kSortBlock = 2048;  // tokens sorted by one block
constexpr int kSortThreads = 256;
constexpr int kPosBits = 11;
constexpr uint32_t kNoKey = 0xffffffffu;

template <typename T, int VEC>
struct Vec;
template <>
struct Vec<float, 8> {
  uint4 a, b;
  __device__ void add_to(float (&f)[8]) const {
    f[0] += __uint_as_float(a.x), f[1] += __uint_as_float(a.y), f[2] += __uint_as_float(a.z), f[3] += __uint_as_float(a.w);
    f[4] += __uint_as_float(b.x), f[5] += __uint_as_float(b.y), f[6] += __uint_as_float(b.z), f[7] += __uint_as_float(b.w);
  }
  __device__ static Vec of(const float (&f)[8]) {
    return {make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])),
            make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]))};
  }
};
template <>
struct Vec<__nv_bfloat16, 8> {
  uint4 a;
  __device__ void add_to(float (&f)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] += __uint_as_float(w[i] << 16);
      f[2 * i + 1] += __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static Vec of(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return {make_uint4(w[0], w[1], w[2], w[3])};
  }
};
template <>
struct Vec<float, 4> {
  uint4 a;
  __device__ void add_to(float (&f)[4]) const {
    f[0] += __uint_as_float(a.x), f[1] += __uint_as_float(a.y), f[2] += __uint_as_float(a.z), f[3] += __uint_as_float(a.w);
  }
  __device__ static Vec of(const float (&f)[4]) {
    return {make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]))};
  }
};
template <>
struct Vec<__nv_bfloat16, 4> {
  uint2 a;
  __device__ void add_to(float (&f)[4]) const {
    f[0] += __uint_as_float(a.x << 16), f[1] += __uint_as_float(a.x & 0xffff0000u);
    f[2] += __uint_as_float(a.y << 16), f[3] += __uint_as_float(a.y & 0xffff0000u);
  }
  __device__ static Vec of(const float (&f)[4]) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(f[0], f[1]), q = __floats2bfloat162_rn(f[2], f[3]);
    return {make_uint2(*reinterpret_cast<const uint32_t*>(&p), *reinterpret_cast<const uint32_t*>(&q))};
  }
};
template <>
struct Vec<float, 1> {
  float a;
  __device__ void add_to(float (&f)[1]) const { f[0] += a; }
  __device__ static Vec of(const float (&f)[1]) { return {f[0]}; }
};
template <>
struct Vec<__nv_bfloat16, 1> {
  __nv_bfloat16 a;
  __device__ void add_to(float (&f)[1]) const { f[0] += __bfloat162float(a); }
  __device__ static Vec of(const float (&f)[1]) { return {__float2bfloat16_rn(f[0])}; }
};

// blockIdx.x: token, blockIdx.y: slab of blockDim.x pieces of its row.
template <typename T, int VEC>
__global__ void __launch_bounds__(256)
    embed_kernel(const T* table, const int32_t* token, T* out, int H, int V, float scale, DeviceStatus* st) {
  using P = Vec<T, VEC>;
  const int nvec = H / VEC, c = blockIdx.y * blockDim.x + threadIdx.x;
  const int64_t t = blockIdx.x;
  const int32_t v = __ldg(token + t);
  if (v >= V && threadIdx.x == 0 && blockIdx.y == 0) set_status(st, MOE_ERR_DEVICE_BAD_INPUT, (int32_t)t);
  if (c >= nvec) return;
  float f[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) f[e] = 0.0f;
  if (v >= 0 && v < V) {
    reinterpret_cast<const P*>(table)[(int64_t)v * nvec + c].add_to(f);
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] *= scale;
  }
  reinterpret_cast<P*>(out)[t * nvec + c] = P::of(f);
}

// Sorts block b's tokens [2048 b, 2048 b + 2048): keys [T rounded up to 2048] (tokens that do
// not count, and the places past T, become kNoKey and sort last). With one block the order is
// final: stoken and spos are written. The number of tokens that count goes to block_count[b],
// or to *count. A bitonic network with 8 consecutive keys per thread: strides below 8 stay in
// registers, below 256 in a warp's shuffles, and only 6 of the 66 stages need a barrier (with
// every stage in shared memory the sort of 16384 tokens took 10.9 us).
constexpr int kKeys = kSortBlock / kSortThreads;
static_assert(kKeys == 8, "the stages below");

template <int STRIDE>
__device__ __forceinline__ void sort_in_thread(uint32_t (&k)[kKeys], int size) {
#pragma unroll
  for (int i = 0; i < kKeys; ++i) {
    if (i & STRIDE) continue;
    const uint32_t a = k[i], b = k[i | STRIDE];
    const bool up = ((threadIdx.x * kKeys + i) & size) == 0;
    k[i] = up ? min(a, b) : max(a, b);
    k[i | STRIDE] = up ? max(a, b) : min(a, b);
  }
}

__global__ void __launch_bounds__(kSortThreads)
    sort_blocks_kernel(const int32_t* token, int T, int V, uint32_t* keys, int32_t* block_count,
                       int32_t* stoken, int32_t* spos, int32_t* count, DeviceStatus* st) {
  __shared__ __align__(16) uint32_t other[2][kSortBlock];
  __shared__ int32_t counted;
  let_next_begin();
  const int64_t base = (int64_t)blockIdx.x * kSortBlock;
  const int first = threadIdx.x * kKeys;  // this thread's first place in the block
  if (threadIdx.x == 0) counted = 0;
  __syncthreads();
  uint32_t k[kKeys];
  int32_t mine = 0;
#pragma unroll
  for (int i = 0; i < kKeys; ++i) {
    k[i] = kNoKey;
    if (base + first + i < T) {
      const int32_t v = __ldg(token + base + first + i);
      if (v >= V) set_status(st, MOE_ERR_DEVICE_BAD_INPUT, (int32_t)(base + first + i));
      if (v >= 0 && v < V) k[i] = (uint32_t)v << kPosBits | (uint32_t)(first + i), ++mine;
    }
  }
  if (mine) atomicAdd(&counted, mine);
  const int live = (int)min((int64_t)kSortBlock, T - base);
  int n = kKeys;  // sorted length: a power of two that holds every live element
  while (n < live) n <<= 1;
  int turn = 0;
  for (int size = 2; size <= n; size <<= 1) {
    int stride = size >> 1;
    for (; stride >= 32 * kKeys; stride >>= 1) {  // across warps
      uint4* out = reinterpret_cast<uint4*>(other[turn] + first);
      out[0] = make_uint4(k[0], k[1], k[2], k[3]);
      out[1] = make_uint4(k[4], k[5], k[6], k[7]);
      __syncthreads();
      const uint4* in = reinterpret_cast<const uint4*>(other[turn] + (first ^ stride));
      const uint4 a = in[0], b = in[1];
      const uint32_t p[kKeys] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      const bool low = ((first & stride) == 0) == ((first & size) == 0);
#pragma unroll
      for (int i = 0; i < kKeys; ++i) k[i] = low ? min(k[i], p[i]) : max(k[i], p[i]);
      turn ^= 1;  // the next exchange writes the other buffer, whose readers are a barrier behind
    }
    for (; stride >= kKeys; stride >>= 1) {
      const bool low = ((first & stride) == 0) == ((first & size) == 0);
#pragma unroll
      for (int i = 0; i < kKeys; ++i) {
        const uint32_t p = __shfl_xor_sync(0xffffffffu, k[i], stride / kKeys);
        k[i] = low ? min(k[i], p) : max(k[i], p);
      }
    }
    if (size >= 8) sort_in_thread<4>(k, size);
    if (size >= 4) sort_in_thread<2>(k, size);
    sort_in_thread<1>(k, size);
  }
  const bool single = gridDim.x == 1;
  if (!single) {
    uint4* out = reinterpret_cast<uint4*>(keys + base + first);
    out[0] = make_uint4(k[0], k[1], k[2], k[3]);
    out[1] = make_uint4(k[4], k[5], k[6], k[7]);
  } else {
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      if (k[i] == kNoKey) continue;
      stoken[first + i] = (int32_t)(k[i] >> kPosBits);
      spos[first + i] = (int32_t)(k[i] & (kSortBlock - 1));
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) *(single ? count : block_count + blockIdx.x) = counted;
}

// The place of every key among the run_blocks blocks of its run: its index in its own block, plus
// the number of keys of the same or a smaller token in the blocks before, and of a smaller token
// in those after. One thread per key; the blocks' keys pass through shared memory four blocks at a
// time (searched in L2 the 11 dependent steps took 10.6 us for 16384 tokens). Block 0 also adds up
// the blocks' counts. With more than one run the tokens that do not count are placed too, last.
// Up to 32 blocks are one run; more are runs of 16 (the whole gradient of 65536 tokens of 8
// channels: 82 us, and 87 with two runs to merge; of 131072: 119 with runs of 32, 108 with 16).
int run_blocks_of(int blocks) { return blocks <= 32 ? 32 : 16; }
constexpr int kRankBlocks = 4;
__global__ void __launch_bounds__(256)
    rank_kernel(const uint32_t* keys, const int32_t* block_count, int blocks, int run_blocks, int32_t* stoken,
                int32_t* spos, int32_t* count) {
  __shared__ __align__(16) uint32_t sk[kRankBlocks][kSortBlock];
  let_next_begin();
  after_previous();
  if (blockIdx.x == 0) {
    __shared__ int32_t total;
    if (threadIdx.x == 0) total = 0;
    __syncthreads();
    int32_t mine = 0;
    for (int b = threadIdx.x; b < blocks; b += 256) mine += block_count[b];
    if (mine) atomicAdd(&total, mine);
    __syncthreads();
    if (threadIdx.x == 0) *count = total;
  }
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int own = (int)(i / kSortBlock);
  const int run0 = own / run_blocks * run_blocks, run1 = min(blocks, run0 + run_blocks);
  const uint32_t key = keys[i], token = key >> kPosBits;
  const uint32_t own_bound = key == kNoKey ? 0 : key;
  int rank = run0 * kSortBlock;
  for (int b0 = run0; b0 < run1; b0 += kRankBlocks) {
    const int here = min(kRankBlocks, run1 - b0);
    const uint4* src = reinterpret_cast<const uint4*>(keys + (int64_t)b0 * kSortBlock);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kRankBlocks * kSortBlock / 4 / 256; ++j) {
      const int at = threadIdx.x + j * 256;
      if (at < here * (kSortBlock / 4)) reinterpret_cast<uint4*>(sk)[at] = src[at];
    }
    __syncthreads();
    int at[kRankBlocks];  // number of keys below the bound
    uint32_t bound[kRankBlocks];
#pragma unroll
    for (int u = 0; u < kRankBlocks; ++u) {
      const int b = b0 + u;
      bound[u] = u >= here ? 0u : b == own ? own_bound : (b < own ? token + 1 : token) << kPosBits;
      at[u] = 0;
    }
#pragma unroll
    for (int s = kSortBlock / 2; s > 0; s >>= 1)
#pragma unroll
      for (int u = 0; u < kRankBlocks; ++u)
        if (sk[u][at[u] + s - 1] < bound[u]) at[u] += s;
#pragma unroll
    for (int u = 0; u < kRankBlocks; ++u) {
      if (at[u] == kSortBlock - 1 && sk[u][at[u]] < bound[u]) ++at[u];
      rank += at[u];
    }
  }
  if (key == kNoKey) {
    if (blocks <= run_blocks) return;
    // the bounds of the blocks before wrapped to 0: all of those, and the places before it in its own
    rank += (own - run0) * kSortBlock + (int)(i % kSortBlock);
  }
  stoken[rank] = (int32_t)token;
  spos[rank] = own * kSortBlock + (int)(key & (kSortBlock - 1));
}

// Merges kMerge sorted runs of `run` places (a power of two) into one, of [0, n): the place of an
// element is its index in its own run plus the number of the same or smaller tokens in the runs
// before and of smaller ones in those after. The tokens are in L2, and a warp's 32 neighbours walk
// nearly the same way through them.
constexpr int kMerge = 8;
__global__ void __launch_bounds__(256)
    merge_kernel(const int32_t* token, const int32_t* pos, int n, int run, int32_t* token_out, int32_t* pos_out) {
  let_next_begin();
  after_previous();
  const int i = blockIdx.x * 256 + threadIdx.x;  // n is a multiple of 256
  const int64_t base = (int64_t)i / ((int64_t)run * kMerge) * ((int64_t)run * kMerge);
  const int own = (int)((i - base) / run);
  const int32_t v = token[i];
  int at[kMerge];  // places of the run with a token below the bound
#pragma unroll
  for (int u = 0; u < kMerge; ++u) at[u] = 0;
  for (int s = run; s > 0; s >>= 1)
#pragma unroll
    for (int u = 0; u < kMerge; ++u) {
      const int64_t first = base + (int64_t)u * run;
      if (u != own && at[u] + s <= run && first + at[u] + s <= n &&
          token[first + at[u] + s - 1] < v + (u < own ? 1 : 0))
        at[u] += s;
    }
  int64_t rank = base + (i - base) % run;
#pragma unroll
  for (int u = 0; u < kMerge; ++u) rank += at[u];
  token_out[rank] = v;
  pos_out[rank] = pos[i];
}

struct EmbedBwd {
  const int32_t *stoken, *spos, *count;
  const void* dout;
  void* dtable;
  float* part;  // [chunks][2][H]: the sums of a run that came from the chunk before, and of one that goes on
  int H, V, chunk, chunks, zero_rows, zero_lanes_log, accumulate;
  float scale;
};

template <typename G, int VEC>
__device__ __forceinline__ void write_row(const EmbedBwd& p, int32_t v, int c, const float (&acc)[VEC]) {
  using Q = Vec<G, VEC>;
  Q* dst = static_cast<Q*>(p.dtable) + (int64_t)v * (p.H / VEC) + c;
  float f[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) f[e] = acc[e] * p.scale;
  if (p.accumulate) dst->add_to(f);
  *dst = Q::of(f);
}

// blockIdx.x < chunks: the sums of one chunk of sorted positions; the further blocks zero the
// rows of tokens that do not occur, zero_rows tokens each. blockIdx.y: slab of 256 pieces.
constexpr int kMaxChunk = 256;
template <typename T, typename G, int VEC>
__global__ void __launch_bounds__(256) embed_sum_kernel(const EmbedBwd p) {
  using P = Vec<T, VEC>;
  __shared__ int32_t ids[kMaxChunk + 2];  // ids[i + 1] = token of the chunk's place i, with both neighbours
  __shared__ int32_t pos[kMaxChunk];
  let_next_begin();
  after_previous();
  const int nvec = p.H / VEC, c = blockIdx.y * 256 + threadIdx.x;
  const int n = *p.count;
  if ((int)blockIdx.x < p.chunks) {
    const int64_t s = (int64_t)blockIdx.x * p.chunk;
    if (s >= n) return;
    const int len = (int)min((int64_t)p.chunk, n - s);
    for (int i = threadIdx.x; i < len + 2; i += 256) {
      const int64_t at = s + i - 1;
      ids[i] = at >= 0 && at < n ? p.stoken[at] : -1;
      if (i >= 1 && i <= len) pos[i - 1] = p.spos[at];
    }
    __syncthreads();
    if (c >= nvec) return;
    const P* dout = static_cast<const P*>(p.dout) + c;
    float acc[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = 0.0f;
    bool started = ids[0] != ids[1];  // the current run begins inside this chunk
    constexpr int kAhead = 8;  // loads in flight
    P buf[kAhead];
    for (int i0 = 0; i0 < len; i0 += kAhead) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (i0 + u < len) buf[u] = dout[(int64_t)pos[i0 + u] * nvec];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u;
        if (i >= len) break;
        buf[u].add_to(acc);
        const bool ends = ids[i + 2] != ids[i + 1];
        if (ends || i + 1 == len) {
          if (started && ends) {
            write_row<G, VEC>(p, ids[i + 1], c, acc);
          } else {
            float* q = p.part + ((int64_t)blockIdx.x * 2 + (started ? 1 : 0)) * p.H + (int64_t)c * VEC;
#pragma unroll
            for (int e = 0; e < VEC; ++e) q[e] = acc[e];
          }
#pragma unroll
          for (int e = 0; e < VEC; ++e) acc[e] = 0.0f;
          started = true;
        }
      }
    }
  } else {
    // the tokens [v0, v1) that do not occur: walk the sorted tokens from the first >= v0
    const int v0 = ((int)blockIdx.x - p.chunks) * p.zero_rows, v1 = min(p.V, v0 + p.zero_rows);
    __shared__ uint32_t seen[kMaxChunk / 32];
    for (int i = threadIdx.x; i < kMaxChunk / 32; i += 256) seen[i] = 0;
    // The first place after lo with a token >= v, which is in (lo, n]. Every warp: the lanes try a
    // place each, 32 times closer per step.
    auto first_from = [&](int lo, int v) {
      int hi = n;
      while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + (int)(threadIdx.x % 32 + 1) * step;
        const bool less = at < hi && p.stoken[at] < v;
        const int k = __popc(__ballot_sync(0xffffffffu, less));  // sorted: the places below v are the first k
        hi = min(hi, lo + (k + 1) * step);
        lo += k * step;
      }
      return hi;
    };
    int at = first_from(-1, v0);
    __syncthreads();
    // A token that fills 4096 places is left behind by a search (walked to its end, one token in half
    // of 1048576 positions of 8 channels made the gradient 968 us, 549 so).
    while (at < n) {
      const int first = p.stoken[at], end = min(at + 4096, n), last = p.stoken[end - 1];
      for (int i = at + threadIdx.x; i < end; i += 256) {
        const int v = p.stoken[i];
        if (v >= v1) break;
        atomicOr(&seen[(v - v0) >> 5], 1u << ((v - v0) & 31));
      }
      if (last >= v1) break;
      __syncwarp();
      at = first == last && end < n ? first_from(end - 1, last + 1) : end;
    }
    __syncthreads();
    using W = typename std::conditional<(VEC > 1), uint4, G>::type;  // rows of whole 16-byte words, or of elements
    const int words = p.H * (int)sizeof(G) / (int)sizeof(W);
    W* row = static_cast<W*>(p.dtable) + (int64_t)v0 * words;
    auto absent = [&](int v) { return !(seen[v >> 5] >> (v & 31) & 1); };
    if (words < 256) {  // 2^k threads to a row
      const int k = p.zero_lanes_log, at = threadIdx.x & ((1 << k) - 1);
      if (at >= words) return;
#pragma unroll 4
      for (int v = threadIdx.x >> k; v < v1 - v0; v += 256 >> k)
        if (absent(v)) row[v * words + at] = W{};
    } else if constexpr (VEC > 1) {
      for (int v = 0; v < v1 - v0; ++v, row += words)
        if (absent(v))
          for (int i = blockIdx.y * 256 + threadIdx.x; i < words; i += gridDim.y * 256) row[i] = W{};
    } else {
      if (c >= nvec) return;
      for (int v = 0; v < v1 - v0; ++v, row += words)
        if (absent(v)) row[c] = W{};
    }
  }
}

// One warp per chunk whose last run goes on: adds the run's partial sums in the order of the
// chunks, 32 pieces wide (blockIdx.y).
template <typename G, int VEC>
__global__ void __launch_bounds__(256) embed_join_kernel(const EmbedBwd p) {
  const int chunk = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  after_previous();
  const int n = *p.count;
  const int64_t e = ((int64_t)chunk + 1) * p.chunk, s = e - p.chunk;  // the chunk's places [s, e)
  if (e >= n) return;
  const int32_t v = p.stoken[e - 1];
  const int32_t next = p.stoken[e], at_s = p.stoken[s], before = s > 0 ? p.stoken[s - 1] : -1;
  if (next != v || (at_s == v && before == v)) return;  // it ends here, or began in an earlier chunk
  // the chunk of the run's last place: the 32 lanes try a place each, 32 times closer per step
  int64_t lo = e, hi = n;  // place lo belongs to the run, place hi does not
  while (hi - lo > 1) {
    const int64_t step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
    const bool in = at < hi && p.stoken[at] == v;
    const int k = __popc(__ballot_sync(0xffffffffu, in));  // sorted: the places in the run are the first k
    const int64_t nhi = lo + (int64_t)(k + 1) * step;
    lo += k * step;
    hi = nhi < hi ? nhi : hi;
  }
  const int last = (int)(lo / p.chunk);
  const int nvec = p.H / VEC, c = blockIdx.y * 32 + lane;
  if (c >= nvec) return;
  float acc[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
  // slot 1 of the first chunk, slot 0 of the further ones
  using P = Vec<float, VEC>;
  const P* part = reinterpret_cast<const P*>(p.part) + c;
  part[((int64_t)chunk * 2 + 1) * nvec].add_to(acc);
  constexpr int kAhead = 16;
  for (int k0 = chunk + 1; k0 <= last; k0 += kAhead) {
    P buf[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (k0 + u <= last) buf[u] = part[(int64_t)(k0 + u) * 2 * nvec];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (k0 + u <= last) buf[u].add_to(acc);
  }
  write_row<G, VEC>(p, v, c, acc);
}

int chunk_of(int64_t T) {
  int chunk = 32;  // about a thousand chunks, of 32 to 256 places
  while (chunk < kMaxChunk && T > (int64_t)chunk * 1024) chunk *= 2;
  return chunk;
}

template <typename T, typename G, int VEC>
cudaError_t sums(const moe_embed_config_t& c, EmbedBwd p, cudaStream_t s) {
  const int nvec = c.H / VEC;
  const int zero_blocks = p.accumulate ? 0 : (int)ceil_div(c.V, p.zero_rows);
  const cudaError_t e = launch_after(embed_sum_kernel<T, G, VEC>,
                                     dim3((unsigned)(p.chunks + zero_blocks), (unsigned)ceil_div(nvec, 256)), 256, s, p);
  if (e != cudaSuccess || p.chunks < 2) return e;
  constexpr int JV = VEC > 4 ? 4 : VEC;  // fewer columns per lane, more partial sums in flight
  return launch_after(embed_join_kernel<G, JV>,
                      dim3((unsigned)ceil_div(p.chunks - 1, 8), (unsigned)ceil_div(c.H / JV, 32)), 256, s, p);
}

}  // namespace

EmbedScratch embed_scratch(const moe_embed_config_t& c) {
  EmbedScratch L;
  size_t o = kWsHead;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes, 256);
    return at;
  };
  const size_t T = align_up((size_t)c.T, kSortBlock);
  L.count = take(4);
  L.block_count = take(T / kSortBlock * 4);
  L.keys = take(T * 4);
  L.stoken = take(T * 4);
  L.spos = take(T * 4);
  L.mpos = take(T > (size_t)kSortBlock * run_blocks_of((int)(T / kSortBlock)) ? T * 4 : 0);
  L.part = take((size_t)ceil_div(c.T, chunk_of(c.T)) * 2 * c.H * 4);
  L.total = o;
  return L;
}

cudaError_t launch_embed(const moe_embed_config_t& c, const void* table, const int32_t* token, void* out,
                         DeviceStatus* st, cudaStream_t s) {
  if (c.T == 0) return cudaSuccess;
  const bool bf = c.act_dtype == MOE_DTYPE_BF16, wide = c.H % 8 == 0;
  const int nvec = wide ? c.H / 8 : c.H, threads = (int)std::min<int64_t>(256, ceil_div(nvec, 32) * 32);
  const dim3 grid((unsigned)c.T, (unsigned)ceil_div(nvec, threads));
  auto run = [&](auto kern, auto* t, auto* o) { kern<<<grid, threads, 0, s>>>(t, token, o, c.H, c.V, c.scale, st); };
  const auto* tb = static_cast<const __nv_bfloat16*>(table);
  const auto* tf = static_cast<const float*>(table);
  auto* ob = static_cast<__nv_bfloat16*>(out);
  auto* of = static_cast<float*>(out);
  if (bf && wide) run(embed_kernel<__nv_bfloat16, 8>, tb, ob);
  else if (bf) run(embed_kernel<__nv_bfloat16, 1>, tb, ob);
  else if (wide) run(embed_kernel<float, 8>, tf, of);
  else run(embed_kernel<float, 1>, tf, of);
  return cudaGetLastError();
}

cudaError_t launch_embed_backward(const moe_embed_config_t& c, const int32_t* token, const void* dout, void* dtable,
                                  int accumulate, void* ws, DeviceStatus* st, cudaStream_t s) {
  const bool gbf = c.grad_dtype == MOE_DTYPE_BF16, bf = c.act_dtype == MOE_DTYPE_BF16, wide = c.H % 8 == 0;
  if (c.T == 0)
    return accumulate ? cudaSuccess : cudaMemsetAsync(dtable, 0, (size_t)c.V * c.H * (gbf ? 2 : 4), s);
  const EmbedScratch L = embed_scratch(c);
  char* w = static_cast<char*>(ws);
  auto* keys = reinterpret_cast<uint32_t*>(w + L.keys);
  auto* stoken = reinterpret_cast<int32_t*>(w + L.stoken);
  auto* spos = reinterpret_cast<int32_t*>(w + L.spos);
  auto* count = reinterpret_cast<int32_t*>(w + L.count);
  auto* bcount = reinterpret_cast<int32_t*>(w + L.block_count);
  const int blocks = (int)ceil_div(c.T, kSortBlock);
  sort_blocks_kernel<<<blocks, kSortThreads, 0, s>>>(token, c.T, c.V, keys, bcount, stoken, spos, count, st);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (blocks > 1) {
    const int n = blocks * kSortBlock;
    e = launch_after(rank_kernel, n / 256, 256, s, keys, bcount, blocks, run_blocks_of(blocks), stoken, spos, count);
    // then from one pair of arrays to the other; the keys are not needed any more
    auto *token2 = reinterpret_cast<int32_t*>(keys), *pos2 = reinterpret_cast<int32_t*>(w + L.mpos);
    for (int64_t run = kSortBlock * run_blocks_of(blocks); run < n && e == cudaSuccess; run *= kMerge) {
      e = launch_after(merge_kernel, n / 256, 256, s, stoken, spos, n, (int)run, token2, pos2);
      std::swap(stoken, token2);
      std::swap(spos, pos2);
    }
    if (e != cudaSuccess) return e;
  }
  EmbedBwd p{stoken, spos, count, dout, dtable, reinterpret_cast<float*>(w + L.part)};
  p.H = c.H;
  p.V = c.V;
  p.chunk = chunk_of(c.T);
  p.chunks = (int)ceil_div(c.T, p.chunk);
  // zeros: a power of two of threads per row, and 32 rows a block or as many as give every thread
  // 16 (4096 tokens of 64 channels, 100000 rows: 54 us with a block's width per row, 21 so)
  const int words = wide ? (int)(c.H * (gbf ? 2 : 4) / 16) : c.H;
  while (p.zero_lanes_log < 8 && 1 << p.zero_lanes_log < words) ++p.zero_lanes_log;
  p.zero_rows = std::max(32, std::min(kMaxChunk, 4096 >> p.zero_lanes_log));
  p.accumulate = accumulate;
  p.scale = c.scale;
  if (wide) {
    if (bf) return gbf ? sums<__nv_bfloat16, __nv_bfloat16, 8>(c, p, s) : sums<__nv_bfloat16, float, 8>(c, p, s);
    return gbf ? sums<float, __nv_bfloat16, 8>(c, p, s) : sums<float, float, 8>(c, p, s);
  }
  if (bf) return gbf ? sums<__nv_bfloat16, __nv_bfloat16, 1>(c, p, s) : sums<__nv_bfloat16, float, 1>(c, p, s);
  return gbf ? sums<float, __nv_bfloat16, 1>(c, p, s) : sums<float, float, 1>(c, p, s);
}

}  // namespace moe
