// In front of the tensor-core attention kernels on a batch of several sequences: their tiles in the
// order of their work, the longest first (the hardware deals CTAs out in that order, so the short ones
// fill the gaps at the end), and for the backward the rows' statistics in the order its tiles read them.
//
// One block sorts: a prefix of the sequences' tiles, a histogram of their work over 64 classes, a
// scatter. Tiles of equal class come in any order; no result depends on it. Long tiles of dk and dv
// (which run over every query of a whole group of heads) are cut into pieces, so that no CTA has more
// than its part of a round left when the others are done.
#include "attn_plan.cuh"
#include "attn_tc.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kSort = 256;     // threads of a block
constexpr int kFirst = 1024;   // sequences whose prefix is kept in shared memory
constexpr int kClasses = 64;
constexpr int kLost = (int)0x80000000;  // of a sequence's entry in the prefix: its keys are not its own
constexpr int kAhead = 4;      // rows and heads whose loads a thread has in flight

// Steps (inner tiles) of a tile of queries, or of a tile of keys for all packs of heads.
__device__ __forceinline__ int tile_steps(const AttnArgs& a, const PlanJob& j, const Seq& s, int tile) {
  if (!j.keys) {
    const int last = min((tile + 1) * j.rows, s.n) - 1;
    return (max(0, visible(a, s, last)) + 127) / 128;
  }
  const int first = a.causal ? max(0, tile * 128 - (s.m - s.n)) / j.inner : 0;
  return max(0, (s.n + j.inner - 1) / j.inner - first) * j.packs;
}

__device__ void sort_tiles(const AttnArgs& a, const PlanJob& j, bool apart, bool report) {
  __shared__ int sKept[kFirst + 1];
  __shared__ int64_t sWarp[kSort / 32];
  __shared__ int sEnd[kSort / 32];
  __shared__ unsigned long long sTotal;
  __shared__ int sMost, sSlots, sClass[kClasses];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rows = j.keys ? 128 : j.rows;
  int* sFirst = a.B <= kFirst ? sKept : j.first;
  if (tid == 0) sTotal = 0, sMost = 0, sSlots = 0;
  if (tid < kClasses) sClass[tid] = 0;
  int64_t carry = 0;  // tiles of the sequences before: with rows that overlap more than 32 bits count
  int front = 0;      // where their keys end
  for (int b0 = 0; b0 < a.B; b0 += kSort) {
    const int b = b0 + tid;
    Seq s{};
    if (b < a.B) s = load_seq(a, b, report);
    bool lost = false;
    if (apart) {
      const Largest l = largest_before<kSort>(keys_end(s), sEnd);
      int end = max(front, l.before);
      lost = hold_apart(s, end);
      if (lost && report) set_status(a.status, MOE_ERR_DEVICE_BAD_INPUT, b);
      front = max(front, l.all);
    }
    const int n = ((j.keys ? s.m : s.n) + rows - 1) / rows;
    int64_t inc = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += o;
    }
    __syncthreads();
    if (lane == 31) sWarp[warp] = inc;
    __syncthreads();
    int64_t before = carry + inc - n, all = 0;
    for (int w = 0; w < kSort / 32; ++w) {
      if (w < warp) before += sWarp[w];
      all += sWarp[w];
    }
    if (b < a.B) sFirst[b] = (int)min(before, (int64_t)j.most) | (lost ? kLost : 0);
    carry += all;
  }
  __syncthreads();
  const int tiles = (int)min(carry, (int64_t)j.most);  // more only where sequences share rows, which is reported
  auto seq_of = [&](int t) {
    int lo = 0, hi = a.B - 1;  // the last sequence that begins at or before t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((sFirst[mid] & ~kLost) <= t) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  };
  struct Found {
    Seq s;
    int index, steps;
  };
  auto find = [&](int t) {
    const int b = seq_of(t), first = sFirst[b];
    Found f{load_seq(a, b, false), t - (first & ~kLost), 0};
    if (first & kLost) f.s.k0 = f.s.m = 0;
    f.steps = tile_steps(a, j, f.s, f.index);
    return f;
  };
  const Found own = tid < tiles ? find(tid) : Found{};  // the thread's first tile, for all three passes
  auto tile = [&](int t) { return t == tid ? own : find(t); };
  int64_t sum = 0;
  int most = 0;
  for (int t = tid; t < tiles; t += kSort) {
    const int n = tile(t).steps;
    sum += n;
    most = max(most, n);
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, off);
    most = max(most, __shfl_xor_sync(0xffffffffu, most, off));
  }
  if (lane == 0) {
    atomicAdd(&sTotal, (unsigned long long)sum);
    atomicMax(&sMost, most);
  }
  __syncthreads();
  // a piece is at most what a CTA has of all the work, and worth its ends
  int limit = 0x7fffffff;
  if (j.pieces > 0) limit = max(16, (int)min((unsigned long long)0x7fffffff, (sTotal * j.heads + j.pieces - 1) / j.pieces));
  const int top = max(1, min(sMost, limit));
  auto cut = [&](int n) { return n > limit ? (n + limit - 1) / limit : 1; };
  auto cls = [&](int n) { return kClasses - 1 - min(kClasses - 1, (int)((int64_t)n * (kClasses - 1) / top)); };  // 0: the longest
  for (int t = tid; t < tiles; t += kSort) {
    const int n = tile(t).steps, p = cut(n);
    atomicAdd(&sClass[cls((n + p - 1) / p)], p);
  }
  __syncthreads();
  if (warp == 0) {  // where the classes begin: two to a lane
    static_assert(kClasses == 64);
    const int x = sClass[2 * lane], y = sClass[2 * lane + 1];
    int inc = x + y;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += o;
    }
    sClass[2 * lane] = inc - x - y;
    sClass[2 * lane + 1] = inc - y;
    if (lane == 31) j.plan->count = inc;
  }
  __syncthreads();
  for (int t = tid; t < tiles; t += kSort) {
    const Found f = tile(t);
    const Seq& s = f.s;
    const int n = f.steps, p = cut(n);
    const int at = atomicAdd(&sClass[cls((n + p - 1) / p)], p), slot = p > 1 ? atomicAdd(&sSlots, p) : 0;
    for (int i = 0; i < p; ++i)
      j.plan->tile[at + i] = TileEntry{s.q0, s.n, s.k0, s.m, f.index * rows, (int)((int64_t)n * i / p),
                                       (int)((int64_t)n * (i + 1) / p), p > 1 ? (slot << 16 | i << 8 | p) : 0};
  }
}

// The backward's statistics: -lse log2(e) and -d_o . o of every row and head, the heads of a pack side
// by side, as its tiles' rows are. LANES lanes a row and head, 16 bytes of o and d_o each.
template <int LANES>
__device__ void row_stats(const AttnArgs& a, const StatsJob& j, int64_t block, int64_t blocks) {
  constexpr int kPer = kSort / LANES;
  const int lane = threadIdx.x % LANES, shift = __ffs(j.pack) - 1;
  const bool in = 8 * lane < a.D;
  // pairs (row, head) of this thread: `by` apart, from the first one on
  const int64_t first = block * kPer + threadIdx.x / LANES, by = blocks * kPer;
  const int by_rows = (int)(by / a.Hq), by_heads = (int)(by % a.Hq);
  int64_t row = first / a.Hq;
  int h = (int)(first % a.Hq);
  while (__any_sync(0xffffffffu, row < a.Tq)) {  // a warp has several rows, and its lanes stay together
    uint4 x[kAhead], y[kAhead];
    float l[kAhead];
    int64_t rows[kAhead];
    int heads[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      rows[u] = row, heads[u] = h;
      x[u] = y[u] = make_uint4(0, 0, 0, 0);
      l[u] = 0.0f;
      if (row < a.Tq) {
        if (in) {
          const int64_t at = row * a.ld_o + (int64_t)h * a.D + 8 * lane;
          x[u] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.o) + at);
          y[u] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.d_o) + at);
        }
        if (lane == 0) l[u] = a.lse[(int64_t)h * a.Tq + row];
      }
      row += by_rows, h += by_heads;
      if (h >= a.Hq) h -= a.Hq, ++row;
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const __nv_bfloat162 *xs = reinterpret_cast<const __nv_bfloat162*>(&x[u]), *ys = reinterpret_cast<const __nv_bfloat162*>(&y[u]);
      float dot = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 xf = __bfloat1622float2(xs[e]), yf = __bfloat1622float2(ys[e]);
        dot = fmaf(xf.x, yf.x, fmaf(xf.y, yf.y, dot));
      }
#pragma unroll
      for (int off = LANES / 2; off; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
      if (lane == 0 && rows[u] < a.Tq) {
        const int64_t at = (((int64_t)(heads[u] >> shift) * a.Tq + rows[u]) << shift) + (heads[u] & (j.pack - 1));
        j.neg_lse[at] = l[u] == -INFINITY ? -INFINITY : -l[u] * kLog2e;  // a row without keys: exp2(s - inf) = 0
        j.neg_delta[at] = -dot;
      }
    }
  }
}

__global__ void __launch_bounds__(kSort) plan_kernel(const AttnArgs a, const PlanJob j0, const PlanJob j1, const StatsJob st,
                                                     int jobs, int apart) {
  let_next_begin();
  if ((int)blockIdx.x < jobs) {
    if (blockIdx.x == 0) sort_tiles(a, j0, apart, true);
    else sort_tiles(a, j1, apart, j0.keys == j1.keys);
    return;
  }
  const int64_t block = blockIdx.x - jobs, blocks = gridDim.x - jobs;
  if (a.D <= 64) row_stats<8>(a, st, block, blocks);
  else row_stats<16>(a, st, block, blocks);
}

}  // namespace

cudaError_t launch_plan(const AttnArgs& a, const PlanJob& j, cudaStream_t s) {
  plan_kernel<<<1, kSort, 0, s>>>(a, j, j, StatsJob{}, 1, 0);
  return cudaGetLastError();
}

cudaError_t launch_plan_backward(const AttnArgs& a, const PlanJob& dq, const PlanJob& dkv, const StatsJob& st, cudaStream_t s) {
  const int64_t blocks = ceil_div((int64_t)a.Tq * a.Hq, (int64_t)kSort / (a.D <= 64 ? 8 : 16) * kAhead), most = 8 * (int64_t)tc::num_sms();
  plan_kernel<<<(unsigned)(2 + (blocks < most ? blocks : most)), kSort, 0, s>>>(a, dq, dkv, st, 2, 1);
  return cudaGetLastError();
}

}  // namespace attn
}  // namespace moe
