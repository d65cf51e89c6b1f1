// Attention of few query rows over many keys in fp32: 16 (query, head) rows of a key head at a time, so
// that a cache is read once for all heads of a group, and the keys of a line cut into some 300 parts in all, two
// for every SM: side by side up to 64 channels, one after the other at 128 (148 KB of shared memory a block).
//
// A block of 8 warps takes tiles of 64 keys, which come by asynchronous copies into two buffers while the
// tile before is used. Of a tile a warp has 8 keys, and its own running maximum, sum and output for all 16
// rows: a lane forms the scores of 4 rows and one key, then adds DP / 32 channels of all rows. Warps meet
// only at the copies and at the end, where their results, and later the parts', are put together in
// order. 16 requests of 4096 keys (32 query and 8 key heads of 128, 537 MB): 249 us, 2.2 TB/s. Not memory (a third of
// its rate), but what 8 warps of 170 registers on an SM can do: shared memory's pipe is at 58 %, issue at 51 %,
// FMA at 34 %, and the warps wait for shared memory most of all (counted); 384 blocks are 2.5 rounds.
#include "attn.cuh"
#include "tc_common.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int R = 16;   // rows
constexpr int K = 64;   // keys of a tile
constexpr int kMine = K / kWarps;  // keys of a warp

struct FewParams {
  AttnArgs a;
  int lines;   // tiles of 16 rows of a sequence and key head, at most
  int splits;  // parts of a line's keys
  float2* stat;  // [line][split][R]: maximum and sum
  float* part;   // [line][split][R][D]: the output times the sum
};

__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// Line -> sequence, key head, first row. Lines of a sequence and head that has fewer rows are empty.
struct Line {
  int b, hk, r0;
};
__device__ __forceinline__ Line line_of(const AttnArgs& a, int i, int row_tiles) {
  const int t = i % row_tiles, x = i / row_tiles;
  return Line{x / a.Hkv, x % a.Hkv, t * R};
}

template <int DP, bool WIDE>
__global__ void __launch_bounds__(kThreads) few_kernel(const FewParams p, int row_tiles) {
  constexpr int LD = DP + 4, kN = DP / 32;  // kN: channels of a lane
  extern __shared__ float4 smem4[];
  float* sQ = reinterpret_cast<float*>(smem4);      // [R][LD]
  float* sK = sQ + R * LD;                          // [2][K][LD]
  float* sV = sK + 2 * K * LD;                      // [2][K][LD]
  float* sP = sV + 2 * K * LD;                      // [warp][key][R]
  const AttnArgs& a = p.a;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const Line line = line_of(a, blockIdx.x, row_tiles);
  const Seq s = load_seq(a, line.b, line.hk == 0 && line.r0 == 0 && blockIdx.y == 0 && threadIdx.x == 0);
  const int rows = min(R, s.n * a.group - line.r0);
  if (rows <= 0) return;
  // row r: query (r0 + r) / group of the sequence, head (r0 + r) % group of the key head's
  auto query = [&](int r) { return (line.r0 + r) / a.group; };
  auto q_head = [&](int r) { return line.hk * a.group + (line.r0 + r) % a.group; };
  for (int i = threadIdx.x; i < R * DP; i += kThreads) {
    const int r = i / DP, d = i % DP;
    float v = 0.0f;
    if (r < rows && d < a.D)
      v = a.scale * static_cast<const float*>(a.q)[(int64_t)(s.q0 + query(r)) * a.ld_q + (int64_t)q_head(r) * a.D + d];
    sQ[r * LD + d] = v;
  }
  const int tiles = (max(0, visible(a, s, query(rows - 1))) + K - 1) / K;
  const int lo = (int)((int64_t)tiles * blockIdx.y / p.splits), hi = (int)((int64_t)tiles * (blockIdx.y + 1) / p.splits);
  auto fetch = [&](int tile, int buffer) {  // K and V rows of a tile, zeros past the last row and channel
    const float* k = static_cast<const float*>(a.k) + (int64_t)(s.k0 + tile * K) * a.ld_k + (int64_t)line.hk * a.D;
    const float* v = static_cast<const float*>(a.v) + (int64_t)(s.k0 + tile * K) * a.ld_v + (int64_t)line.hk * a.D;
    const uint32_t dk = tc::smem_addr(sK + buffer * K * LD), dv = tc::smem_addr(sV + buffer * K * LD);
    const int live = min(K, s.m - tile * K);
    constexpr int kUnit = WIDE ? 4 : 1;
    for (int i = threadIdx.x; i < K * (DP / kUnit); i += kThreads) {
      const int j = i / (DP / kUnit), d = i % (DP / kUnit) * kUnit;
      const bool there = j < live && d < a.D;
      const int64_t jk = there ? j * a.ld_k + d : 0, jv = there ? j * a.ld_v + d : 0;
      if constexpr (WIDE) {
        copy16(dk + (j * LD + d) * 4, k + jk, there);
        copy16(dv + (j * LD + d) * 4, v + jv, there);
      } else {
        copy4(dk + (j * LD + d) * 4, k + jk, there);
        copy4(dv + (j * LD + d) * 4, v + jv, there);
      }
    }
    tc::cp_async_commit();
  };
  // scores: this lane's key of the warp's, and rows g, g + 4, g + 8, g + 12
  const int key = warp * kMine + lane % kMine, g = lane / kMine;
  int end[4];  // keys that they see
#pragma unroll
  for (int i = 0; i < 4; ++i) end[i] = g + 4 * i < rows ? visible(a, s, query(g + 4 * i)) : 0;
  float top[4], sum[4], acc[R][kN] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) top[i] = -INFINITY, sum[i] = 0.0f;
  float* my_p = sP + warp * kMine * R;

  if (lo < hi) fetch(lo, 0);
  for (int t = lo; t < hi; ++t) {
    const int buffer = (t - lo) & 1;
    if (t + 1 < hi) {
      fetch(t + 1, buffer ^ 1);
      tc::cp_async_wait<1>();
    } else {
      tc::cp_async_wait<0>();
    }
    __syncthreads();
    const float* k = sK + (buffer * K + key) * LD;
    float c[4] = {};
#pragma unroll 8
    for (int d = 0; d < DP; d += 4) {
      const float4 kv = *reinterpret_cast<const float4*>(k + d);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 qv = *reinterpret_cast<const float4*>(sQ + (g + 4 * i) * LD + d);
        c[i] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, fmaf(qv.z, kv.z, fmaf(qv.w, kv.w, c[i]))));
      }
    }
    float keep[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (t * K + key >= end[i]) c[i] = -INFINITY;
      float m = c[i];
#pragma unroll
      for (int off = kMine / 2; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
      m = fmaxf(m, top[i]);
      const float base = m == -INFINITY ? 0.0f : m;  // no key yet: exp(-inf - 0) = 0
      keep[i] = expf(top[i] - base);
      const float e = expf(c[i] - base);
      float part = e;
#pragma unroll
      for (int off = kMine / 2; off; off >>= 1) part += __shfl_xor_sync(0xffffffffu, part, off);
      sum[i] = sum[i] * keep[i] + part;
      top[i] = m;
      my_p[(lane % kMine) * R + 4 * g + i] = e;  // in the order of (group, i): row g + 4 i
    }
    __syncwarp();
    // row g + 4 i of all lanes: its factor comes from a lane of group g
#pragma unroll
    for (int x = 0; x < R; ++x) {
      const float f = __shfl_sync(0xffffffffu, keep[x % 4], x / 4 * kMine);
#pragma unroll
      for (int n = 0; n < kN; ++n) acc[x][n] *= f;
    }
    // the tile's sums apart, so that a long line's do not lose more with every tile
    float fresh[R][kN] = {};
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      float v[kN];
#pragma unroll
      for (int n = 0; n < kN; ++n) v[n] = sV[(buffer * K + warp * kMine + j) * LD + 32 * n + lane];
#pragma unroll
      for (int x = 0; x < R; x += 4) {
        const float4 w = *reinterpret_cast<const float4*>(my_p + j * R + x);
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          fresh[x][n] = fmaf(w.x, v[n], fresh[x][n]);
          fresh[x + 1][n] = fmaf(w.y, v[n], fresh[x + 1][n]);
          fresh[x + 2][n] = fmaf(w.z, v[n], fresh[x + 2][n]);
          fresh[x + 3][n] = fmaf(w.w, v[n], fresh[x + 3][n]);
        }
      }
    }
#pragma unroll
    for (int x = 0; x < R; ++x)
#pragma unroll
      for (int n = 0; n < kN; ++n) acc[x][n] += fresh[x][n];
    __syncthreads();  // the buffer may be filled again
  }

  // the warps' results, in shared memory: x = 4 g + i is row g + 4 i
  float* sO = sK;                                          // [warp][R][DP]
  float2* sStat = reinterpret_cast<float2*>(sP);           // [warp][R]
  __syncthreads();
#pragma unroll
  for (int x = 0; x < R; ++x)
#pragma unroll
    for (int n = 0; n < kN; ++n) sO[(warp * R + x) * DP + 32 * n + lane] = acc[x][n];
  if (lane % kMine == 0)
#pragma unroll
    for (int i = 0; i < 4; ++i) sStat[warp * R + 4 * g + i] = make_float2(top[i], sum[i]);
  __syncthreads();
  for (int e = threadIdx.x; e < R * DP; e += kThreads) {
    const int x = e / DP, d = e % DP, r = x / 4 + 4 * (x % 4);
    if (r >= rows) continue;
    float most = -INFINITY, total = 0.0f, o = 0.0f;
    for (int w = 0; w < kWarps; ++w) most = fmaxf(most, sStat[w * R + x].x);
    for (int w = 0; w < kWarps; ++w) {
      // left out without a visible key only: where all scores are NaN the maximum is -inf, the sum NaN
      const float f = sStat[w * R + x].y == 0.0f ? 0.0f : expf(sStat[w * R + x].x - most);
      total = fmaf(f, sStat[w * R + x].y, total);
      o = fmaf(f, sO[(w * R + x) * DP + d], o);
    }
    if (p.splits > 1) {
      const int64_t at = ((int64_t)blockIdx.x * p.splits + blockIdx.y) * R + r;
      if (d < a.D) p.part[at * a.D + d] = o;
      if (d == 0) p.stat[at] = make_float2(most, total);
    } else {
      const int64_t row = s.q0 + query(r);
      if (d < a.D) static_cast<float*>(a.o)[row * a.ld_o + (int64_t)q_head(r) * a.D + d] = total == 0.0f ? 0.0f : o / total;
      if (d == 0) a.lse[(int64_t)q_head(r) * a.Tq + row] = total == 0.0f ? -INFINITY : most + logf(total);
    }
  }
}

// The parts of a line, in their order: their weights first, then a thread for every row and channel.
__global__ void __launch_bounds__(kThreads) few_join_kernel(const FewParams p, int row_tiles) {
  __shared__ float2 sStat[R][kMostSplits];  // maximum and sum; then the weight
  __shared__ float2 sRow[R];                // of the line: maximum and sum
  after_previous();
  const AttnArgs& a = p.a;
  const Line line = line_of(a, blockIdx.x, row_tiles);
  const Seq s = load_seq(a, line.b, false);
  const int rows = min(R, s.n * a.group - line.r0);
  const int64_t at = (int64_t)blockIdx.x * p.splits * R;
  for (int e = threadIdx.x; e < p.splits * R; e += kThreads) sStat[e % R][e / R] = e % R < rows ? p.stat[at + e] : float2{};
  __syncthreads();
  if ((int)threadIdx.x < rows) {
    const int r = threadIdx.x;
    float most = -INFINITY, total = 0.0f;
    for (int i = 0; i < p.splits; ++i) most = fmaxf(most, sStat[r][i].x);
    for (int i = 0; i < p.splits; ++i) {
      const float f = sStat[r][i].y == 0.0f ? 0.0f : expf(sStat[r][i].x - most);
      total = fmaf(f, sStat[r][i].y, total);
      sStat[r][i].x = f;
    }
    sRow[r] = make_float2(most, total);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < rows * a.D; e += kThreads) {
    const int r = e / a.D, d = e - r * a.D;
    const float* part = p.part + (at + r) * a.D + d;
    float o = 0.0f;
#pragma unroll 8
    for (int i = 0; i < p.splits; ++i) o = fmaf(sStat[r][i].x, part[(int64_t)i * R * a.D], o);
    const float2 st = sRow[r];
    const int64_t row = s.q0 + (line.r0 + r) / a.group;
    const int h = line.hk * a.group + (line.r0 + r) % a.group;
    static_cast<float*>(a.o)[row * a.ld_o + (int64_t)h * a.D + d] = st.y == 0.0f ? 0.0f : o / st.y;
    if (d == 0) a.lse[(int64_t)h * a.Tq + row] = st.y == 0.0f ? -INFINITY : st.x + logf(st.y);
  }
}

template <int DP, bool WIDE>
cudaError_t few(const FewParams& p, int row_tiles, cudaStream_t s) {
  constexpr size_t smem = ((R + 4 * K) * (DP + 4) + kWarps * kMine * R) * sizeof(float);
  static Once once;
  const cudaError_t e = allow_smem(once, few_kernel<DP, WIDE>, smem);
  if (e != cudaSuccess) return e;
  few_kernel<DP, WIDE><<<dim3((unsigned)p.lines, (unsigned)p.splits), kThreads, smem, s>>>(p, row_tiles);
  return cudaGetLastError();
}

}  // namespace

// Rows of a sequence and key head that are taken 16 at a time, the keys read once for each 16; beyond them attn_simt.cu's
// tiles of a head's rows, which suit prompts. The edge is for these: single tokens of a group beyond 48 lose
// by it (one query of 64 heads over 4096 keys, a key head of 128: 543 us, of 32 heads 77).
bool few_rule(const AttnArgs& a) {
  return (int64_t)a.max_q * a.group <= 3 * R && (int64_t)a.B * a.Hkv * 3 < (1ll << 31);
}

static int few_row_tiles(const AttnArgs& a) { return (int)ceil_div((int64_t)a.max_q * a.group, R); }

static int few_splits(const AttnArgs& a) {
  const int64_t lines = (int64_t)a.B * a.Hkv * few_row_tiles(a);
  const int64_t n = lines > 0 ? ceil_div(kFewParts, lines) : 1;
  return (int)(n < 1 ? 1 : n > kMostSplits ? kMostSplits : n);
}

cudaError_t launch_few(const AttnArgs& a, float2* stat, float* part, cudaStream_t s) {
  const int row_tiles = few_row_tiles(a);
  const FewParams p{a, a.B * a.Hkv * row_tiles, few_splits(a), stat, part};
  const uint64_t at = (uint64_t)a.k | (uint64_t)a.v | (uint64_t)(4 * a.D) | (uint64_t)(4 * a.ld_k) | (uint64_t)(4 * a.ld_v);
  const bool wide = at % 16 == 0;
  cudaError_t e;
  if (a.D <= 32) e = wide ? few<32, true>(p, row_tiles, s) : few<32, false>(p, row_tiles, s);
  else if (a.D <= 64) e = wide ? few<64, true>(p, row_tiles, s) : few<64, false>(p, row_tiles, s);
  else e = wide ? few<128, true>(p, row_tiles, s) : few<128, false>(p, row_tiles, s);
  if (e != cudaSuccess || p.splits == 1) return e;
  return launch_after(few_join_kernel, (unsigned)p.lines, kThreads, s, p, row_tiles);
}

}  // namespace attn
}  // namespace moe
