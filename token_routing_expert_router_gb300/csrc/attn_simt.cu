// Attention and its backward on the FMA units, in fp32 throughout: fp32 tensors, and bf16 ones whose
// rows the tensor-core kernels cannot load (channels or strides that are no multiples of 16 bytes).
//
//   s_ij = scale q_i . k_j;  lse_i = log sum_j exp s_ij;  o_i = sum_j exp(s_ij - lse_i) v_j
//   delta_i = do_i . o_i;  ds_ij = p_ij (do_i . v_j - delta_i) scale
//   dv_j = sum_i p_ij do_i;  dk_j = sum_i ds_ij q_i;  dq_i = sum_j ds_ij k_j
//
// A block of 256 threads owns 64 query rows (dk, dv: 64 key rows), or 16 of a small batch, and goes over the
// other side in tiles of 64, with the running maximum and sum of the softmax; scores are never stored. Every
// thread forms 4 x 4 (1 x 4) scores, and 4 rows (1) x DP / 16 columns of the results in registers. Two 64 x 64 x D products a
// tile forward; backward three for dq and four for dk and dv (both kernels form the scores and do . v; in return no
// result is added to by two blocks, so the bits never change). What bounds it: operands from shared memory, read at 68 to
// 75 % of that pipe's rate beside FMA units busy 50 to 55 % of the time, with one block of 8 warps an SM to hide the
// latencies of both (counted at 4096 tokens of 8 / 2 heads of 128). 16384 such tokens, causal: forward 14.8 ms,
// 37 TFLOP/s, backward 50.0 ms, 38 TFLOP/s of its seven products. From bf16 tensors delta carries the rounding of o:
// their dq forms the mean key too and puts both right, as in attn_tc_bwd.cu.
#include "attn.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int R = 64;       // rows of a tile
constexpr int PS = R + 4;   // row length of the scores in shared memory

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float* d, float v) { *d = v; }
__device__ __forceinline__ void from_f(__nv_bfloat16* d, float v) { *d = __float2bfloat16_rn(v); }

// Rows [row0, row0 + live) of one head (base points at its first channel of row 0) as fp32, times f,
// zeros past the last row and channel.
template <typename T, int DP, int ROWS>
__device__ __forceinline__ void load_tile(float* dst, const void* base, int64_t ld, int64_t row0, int live, int D, float f) {
  const T* src = static_cast<const T*>(base) + row0 * ld;
  if constexpr (sizeof(T) == 4) {
    if ((((uint64_t)src | (uint64_t)(4 * ld) | (uint64_t)(4 * D)) & 15) == 0) {
#pragma unroll 8
      for (int i = threadIdx.x; i < ROWS * (DP / 4); i += kThreads) {
        const int r = i / (DP / 4), d = i % (DP / 4) * 4;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (r < live && d < D) v = *reinterpret_cast<const float4*>(src + (int64_t)r * ld + d);
        *reinterpret_cast<float4*>(dst + r * (DP + 4) + d) = make_float4(f * v.x, f * v.y, f * v.z, f * v.w);
      }
      return;
    }
  }
#pragma unroll 8
  for (int i = threadIdx.x; i < ROWS * DP; i += kThreads) {
    const int r = i / DP, d = i % DP;
    dst[r * (DP + 4) + d] = r < live && d < D ? f * to_f(src[(int64_t)r * ld + d]) : 0.0f;
  }
}

__device__ __forceinline__ float dot4(float4 a, float4 b, float c) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}

// c[r][j] += x row (N ty + r) . y row (tx + 16 j)
template <int DP, int N>
__device__ __forceinline__ void scores(float (&c)[N][4], const float* x, const float* y, int ty, int tx) {
  constexpr int LD = DP + 4;
#pragma unroll(N == 1 ? 8 : 4)
  for (int d = 0; d < DP; d += 4) {
    float4 a[N], b[4];
#pragma unroll
    for (int r = 0; r < N; ++r) a[r] = *reinterpret_cast<const float4*>(x + (N * ty + r) * LD + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(y + (tx + 16 * j) * LD + d);
#pragma unroll
    for (int r = 0; r < N; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) c[r][j] = dot4(a[r], b[j], c[r][j]);
  }
}

// acc[r][c] += sum_j w[N ty + r][j] y[j][column c of this thread]: kV neighbouring columns, from
// kV tx on, of every 16 kV.
template <int DP>
struct Cols {
  static constexpr int kN = DP / 16;                    // columns of a thread
  static constexpr int kV = kN < 4 ? kN : 4;            // neighbouring ones
};
template <int DP, int N>
__device__ __forceinline__ void accumulate(float (&acc)[N][DP / 16], const float* w, const float* y, int ty, int tx) {
  constexpr int LD = DP + 4, kN = Cols<DP>::kN, kV = Cols<DP>::kV;
#pragma unroll(N == 1 ? 8 : 2)  // a row a thread is little work between loads
  for (int j0 = 0; j0 < R; j0 += 4) {
    float p[N][4];  // [row][j]
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float4 t = *reinterpret_cast<const float4*>(w + (N * ty + i) * PS + j0);
      p[i][0] = t.x, p[i][1] = t.y, p[i][2] = t.z, p[i][3] = t.w;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int c = 0; c < kN; c += kV) {
        float v[kV];
        const float* src = y + (j0 + j) * LD + kV * tx + 16 * c;
        if constexpr (kV == 4) {
          const float4 t = *reinterpret_cast<const float4*>(src);
          v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
        } else {
          static_assert(kV == 2);
          const float2 t = *reinterpret_cast<const float2*>(src);
          v[0] = t.x, v[1] = t.y;
        }
#pragma unroll
        for (int r = 0; r < N; ++r)
#pragma unroll
          for (int l = 0; l < kV; ++l) acc[r][c + l] = fmaf(p[r][j], v[l], acc[r][c + l]);
      }
  }
}

// The same with the tile's sums formed apart: a chain of 64 terms and one of the tiles, where rows over many tiles
// would otherwise lose with every term (32768 equal terms: up to 4e-4 of the sum).
template <int DP, int N>
__device__ __forceinline__ void add_tile(float (&acc)[N][DP / 16], const float* w, const float* y, int ty, int tx) {
  float fresh[N][DP / 16] = {};
  accumulate<DP, N>(fresh, w, y, ty, tx);
#pragma unroll
  for (int r = 0; r < N; ++r)
#pragma unroll
    for (int d = 0; d < DP / 16; ++d) acc[r][d] += fresh[r][d];
}

template <typename T, int DP, int N>
__device__ __forceinline__ void store_rows(void* base, int64_t ld, int64_t row0, int live, int D, const float (&acc)[N][DP / 16],
                                           const float (&f)[N], int ty, int tx) {
  constexpr int kN = Cols<DP>::kN, kV = Cols<DP>::kV;
#pragma unroll
  for (int r = 0; r < N; ++r) {
    if (N * ty + r >= live) continue;
    T* dst = static_cast<T*>(base) + (row0 + N * ty + r) * ld;
#pragma unroll
    for (int c = 0; c < kN; c += kV)
#pragma unroll
      for (int l = 0; l < kV; ++l) {
        const int d = kV * tx + 16 * c + l;
        if (d < D) from_f(dst + d, acc[r][c + l] * f[r]);
      }
  }
}

template <typename T>
__device__ __forceinline__ const T* head(const void* p, int h, int D) {
  return static_cast<const T*>(p) + (int64_t)h * D;
}
template <typename T>
__device__ __forceinline__ T* head(void* p, int h, int D) {
  return static_cast<T*>(p) + (int64_t)h * D;
}

template <int DP>
__host__ __device__ constexpr size_t tile_floats(int rows) {
  return (size_t)rows * (DP + 4);
}

template <typename T, int DP, int N>
__global__ void __launch_bounds__(kThreads) simt_forward_kernel(const AttnArgs a) {
  constexpr int O = 16 * N;  // rows of the block
  extern __shared__ float4 smem4[];
  float* sQ = reinterpret_cast<float*>(smem4);
  float* sK = sQ + tile_floats<DP>(O);
  float* sV = sK + tile_floats<DP>(R);
  float* sP = sV + tile_floats<DP>(R);
  const int h = blockIdx.y, hk = h / a.group, ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  __shared__ alignas(8) int sFind[kFindWords<kThreads>];
  const Tile t = find_tile<kThreads, false, false>(a, blockIdx.x, O, blockIdx.x == 0 && h == 0, sFind);
  if (t.b < 0) return;
  const Seq s = t.s;
  const int i0 = (t.count - 1 - t.index) * O, rows = min(O, s.n - i0);  // the longest first
  load_tile<T, DP, O>(sQ, head<T>(a.q, h, a.D), a.ld_q, s.q0 + i0, rows, a.D, a.scale);

  float acc[N][DP / 16] = {}, top[N], sum[N];
#pragma unroll
  for (int r = 0; r < N; ++r) top[r] = -INFINITY, sum[r] = 0.0f;
  const int keys = visible(a, s, i0 + rows - 1);
  for (int j0 = 0; j0 < keys; j0 += R) {
    __syncthreads();
    const int live = min(R, s.m - j0);
    load_tile<T, DP, R>(sK, head<T>(a.k, hk, a.D), a.ld_k, s.k0 + j0, live, a.D, 1.0f);
    load_tile<T, DP, R>(sV, head<T>(a.v, hk, a.D), a.ld_v, s.k0 + j0, live, a.D, 1.0f);
    __syncthreads();
    float c[N][4] = {};
    scores<DP, N>(c, sQ, sK, ty, tx);
#pragma unroll
    for (int r = 0; r < N; ++r) {
      const int end = visible(a, s, i0 + N * ty + r) - j0;
      float m = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (tx + 16 * j >= end) c[r][j] = -INFINITY;
        m = fmaxf(m, c[r][j]);
      }
#pragma unroll
      for (int off = 8; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
      m = fmaxf(m, top[r]);
      const float base = m == -INFINITY ? 0.0f : m;  // no key yet: exp(-inf - 0) = 0
      const float keep = expf(top[r] - base);
      float part = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = expf(c[r][j] - base);
        sP[(N * ty + r) * PS + tx + 16 * j] = p;
        part += p;
      }
#pragma unroll
      for (int off = 8; off; off >>= 1) part += __shfl_xor_sync(0xffffffffu, part, off);
      sum[r] = sum[r] * keep + part;
      top[r] = m;
#pragma unroll
      for (int d = 0; d < DP / 16; ++d) acc[r][d] *= keep;
    }
    __syncwarp();  // a row's scores come from the 16 threads that use them
    add_tile<DP, N>(acc, sP, sV, ty, tx);
  }
  float f[N];
#pragma unroll
  for (int r = 0; r < N; ++r) {
    f[r] = sum[r] == 0.0f ? 0.0f : 1.0f / sum[r];  // no visible key: a row of zeros
    if (tx == 0 && N * ty + r < rows)
      a.lse[(int64_t)h * a.Tq + s.q0 + i0 + N * ty + r] = sum[r] == 0.0f ? -INFINITY : top[r] + logf(sum[r]);
  }
  store_rows<T, DP, N>(head<T>(a.o, h, a.D), a.ld_o, s.q0 + i0, rows, a.D, acc, f, ty, tx);
}

struct RowStat {
  float lse, delta;
};

// dq of 16 N query rows of a head.
template <typename T, int DP, int N>
__device__ __forceinline__ void dq_rows(const AttnArgs& a, int block, int h) {
  constexpr int O = 16 * N;  // rows of the block
  extern __shared__ float4 smem4[];
  float* sQ = reinterpret_cast<float*>(smem4);
  float* sO = sQ + tile_floats<DP>(O);
  float* sK = sO + tile_floats<DP>(O);
  float* sV = sK + tile_floats<DP>(R);
  float* sP = sV + tile_floats<DP>(R);
  float* sM = sP + O * PS;  // kRounded: P, for the mean key
  constexpr bool kRounded = sizeof(T) == 2;
  const int hk = h / a.group, ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  __shared__ alignas(8) int sFind[kFindWords<kThreads>];
  const Tile t = find_tile<kThreads, false, true>(a, block, O, block == 0 && h == 0, sFind);
  if (t.b < 0) return;
  const Seq s = t.s;
  const int i0 = (t.count - 1 - t.index) * O, rows = min(O, s.n - i0);
  load_tile<T, DP, O>(sQ, head<T>(a.q, h, a.D), a.ld_q, s.q0 + i0, rows, a.D, a.scale);
  load_tile<T, DP, O>(sO, head<T>(a.d_o, h, a.D), a.ld_o, s.q0 + i0, rows, a.D, 1.0f);
  RowStat st[N];
#pragma unroll
  for (int r = 0; r < N; ++r) {
    const int64_t at = (int64_t)h * a.Tq + s.q0 + i0 + N * ty + r;
    const bool live = N * ty + r < rows;
    st[r] = RowStat{live ? a.lse[at] : 0.0f, live ? a.delta[at] : 0.0f};
  }
  float acc[N][DP / 16] = {}, mean[kRounded ? N : 1][DP / 16] = {}, lack[N] = {};
  const int keys = visible(a, s, i0 + rows - 1);
  for (int j0 = 0; j0 < keys; j0 += R) {
    __syncthreads();
    const int live = min(R, s.m - j0);
    load_tile<T, DP, R>(sK, head<T>(a.k, hk, a.D), a.ld_k, s.k0 + j0, live, a.D, 1.0f);
    load_tile<T, DP, R>(sV, head<T>(a.v, hk, a.D), a.ld_v, s.k0 + j0, live, a.D, 1.0f);
    __syncthreads();
    float c[N][4] = {}, dp[N][4] = {};
    scores<DP, N>(c, sQ, sK, ty, tx);
    scores<DP, N>(dp, sO, sV, ty, tx);
#pragma unroll
    for (int r = 0; r < N; ++r) {
      const int end = min(N * ty + r < rows ? visible(a, s, i0 + N * ty + r) : 0, s.m) - j0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = tx + 16 * j < end ? expf(c[r][j] - st[r].lse) : 0.0f;
        const float ds = p == 0.0f ? 0.0f : p * (dp[r][j] - st[r].delta);
        sP[(N * ty + r) * PS + tx + 16 * j] = ds;
        if constexpr (kRounded) sM[(N * ty + r) * PS + tx + 16 * j] = p;
        lack[r] += ds;
      }
    }
    __syncwarp();
    add_tile<DP, N>(acc, sP, sK, ty, tx);
    if constexpr (kRounded) add_tile<DP, N>(mean, sM, sK, ty, tx);
  }
  if constexpr (kRounded) {
#pragma unroll
    for (int r = 0; r < N; ++r) {
#pragma unroll
      for (int off = 8; off; off >>= 1) lack[r] += __shfl_xor_sync(0xffffffffu, lack[r], off);
#pragma unroll
      for (int d = 0; d < DP / 16; ++d) acc[r][d] = fmaf(-lack[r], mean[r][d], acc[r][d]);
      if (tx == 0 && N * ty + r < rows) a.delta[(int64_t)h * a.Tq + s.q0 + i0 + N * ty + r] = st[r].delta + lack[r];
    }
  }
  float f[N];
#pragma unroll
  for (int r = 0; r < N; ++r) f[r] = a.scale;
  store_rows<T, DP, N>(head<T>(a.dq, h, a.D), a.ld_q, s.q0 + i0, rows, a.D, acc, f, ty, tx);
}

// dk and dv of 16 N key rows of a key head: over the query rows that see them, of every query head of
// its group. Scores are transposed: key rows by query rows.
template <typename T, int DP, int N>
__device__ __forceinline__ void dkv_rows(const AttnArgs& a, int block, int hk) {
  constexpr int O = 16 * N;  // rows of the block
  extern __shared__ float4 smem4[];
  float* sK = reinterpret_cast<float*>(smem4);
  float* sV = sK + tile_floats<DP>(O);
  float* sQ = sV + tile_floats<DP>(O);
  float* sO = sQ + tile_floats<DP>(R);
  float* sP = sO + tile_floats<DP>(R);
  float* sS = sP + O * PS;
  __shared__ RowStat sStat[R];
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  __shared__ alignas(8) int sFind[kFindWords<kThreads>];
  const Tile t = find_tile<kThreads, true, true>(a, block, O, block == 0 && hk == 0, sFind);
  if (t.b < 0) return;
  const Seq s = t.s;
  const int j0 = t.index * O, rows = min(O, s.m - j0);
  load_tile<T, DP, O>(sK, head<T>(a.k, hk, a.D), a.ld_k, s.k0 + j0, rows, a.D, 1.0f);
  load_tile<T, DP, O>(sV, head<T>(a.v, hk, a.D), a.ld_v, s.k0 + j0, rows, a.D, 1.0f);
  float dk[N][DP / 16] = {}, dv[N][DP / 16] = {};
  // the first query row that sees key j0
  const int first = a.causal ? max(0, j0 - (s.m - s.n)) : 0;
  for (int h = hk * a.group; h < (hk + 1) * a.group; ++h)
    for (int i0 = first / R * R; i0 < s.n; i0 += R) {
      __syncthreads();
      const int live = min(R, s.n - i0);
      load_tile<T, DP, R>(sQ, head<T>(a.q, h, a.D), a.ld_q, s.q0 + i0, live, a.D, a.scale);
      load_tile<T, DP, R>(sO, head<T>(a.d_o, h, a.D), a.ld_o, s.q0 + i0, live, a.D, 1.0f);
      if (threadIdx.x < R) {
        const int64_t at = (int64_t)h * a.Tq + s.q0 + i0 + threadIdx.x;
        const bool in = (int)threadIdx.x < live;
        sStat[threadIdx.x] = RowStat{in ? a.lse[at] : 0.0f, in ? a.delta[at] : 0.0f};
      }
      __syncthreads();
      float c[N][4] = {}, dp[N][4] = {};
      scores<DP, N>(c, sK, sQ, ty, tx);
      scores<DP, N>(dp, sV, sO, ty, tx);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = tx + 16 * j;  // the query row of the thread's column
        const RowStat st = sStat[i];
        const int end = i < live ? min(visible(a, s, i0 + i), s.m) - j0 : 0;
#pragma unroll
        for (int r = 0; r < N; ++r) {
          const float p = N * ty + r < end ? expf(c[r][j] - st.lse) : 0.0f;
          sP[(N * ty + r) * PS + i] = p;
          sS[(N * ty + r) * PS + i] = p == 0.0f ? 0.0f : p * (dp[r][j] - st.delta);
        }
      }
      __syncwarp();
      add_tile<DP, N>(dv, sP, sO, ty, tx);
      add_tile<DP, N>(dk, sS, sQ, ty, tx);  // q holds the scale
    }
  float one[N];
#pragma unroll
  for (int r = 0; r < N; ++r) one[r] = 1.0f;
  store_rows<T, DP, N>(head<T>(a.dk, hk, a.D), a.ld_k, s.k0 + j0, rows, a.D, dk, one, ty, tx);
  store_rows<T, DP, N>(head<T>(a.dv, hk, a.D), a.ld_v, s.k0 + j0, rows, a.D, dv, one, ty, tx);
}

template <typename T, int DP, int N>
__global__ void __launch_bounds__(kThreads) simt_dq_kernel(const AttnArgs a) {
  dq_rows<T, DP, N>(a, blockIdx.x, blockIdx.y);
}
template <typename T, int DP, int N>
__global__ void __launch_bounds__(kThreads) simt_dkv_kernel(const AttnArgs a) {
  dkv_rows<T, DP, N>(a, blockIdx.x, blockIdx.y);
}
// Both of a small batch, the key tiles first (they take longer): with fp32 tensors dq leaves delta alone. Set up
// beside delta, and one launch less: 30 -> 22 us (256 tokens). Larger ones are launched one after the other: blocks
// that are set up early crowd the SMs that are free first (1024 tokens of 8 heads: 187 -> 263 us).
template <int DP>
__global__ void __launch_bounds__(kThreads) simt_both_kernel(const AttnArgs a, int key_tiles, int query_tiles) {
  after_previous();
  const int i = blockIdx.x - key_tiles * a.Hkv;
  if (i < 0) dkv_rows<float, DP, 1>(a, blockIdx.x % key_tiles, blockIdx.x / key_tiles);
  else dq_rows<float, DP, 1>(a, i % query_tiles, i / query_tiles);
}

// delta: a warp for every query row and head. Rows in no sequence are formed too (nothing reads them).
template <typename T>
__global__ void __launch_bounds__(kThreads) delta_kernel(const AttnArgs a) {
  let_next_begin();
  const int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  if (i >= (int64_t)a.Tq * a.Hq) return;
  const int64_t row = i / a.Hq;
  const int h = (int)(i - row * a.Hq);
  const T* o = head<T>((const void*)a.o, h, a.D) + row * a.ld_o;
  const T* d = head<T>(a.d_o, h, a.D) + row * a.ld_o;
  float sum = 0.0f;
  for (int c = lane; c < a.D; c += 32) sum = fmaf(to_f(o[c]), to_f(d[c]), sum);
#pragma unroll
  for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (lane == 0) a.delta[(int64_t)h * a.Tq + row] = sum;
}

cudaError_t launch_tiles(Once& once, void (*kern)(AttnArgs), dim3 grid, size_t smem, const AttnArgs& a, cudaStream_t s) {
  const cudaError_t e = allow_smem(once, kern, smem);
  if (e != cudaSuccess) return e;
  kern<<<grid, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

// Blocks of `rows` rows of the batch's tiles and heads, at most.
int64_t blocks_of(int total, int B, int heads, int rows) { return ((int64_t)total / rows + B) * heads; }
// Tiles of 16 rows where those of 64 would leave most SMs without one. Forward and backward together with tiles
// of 64 and of 16, causal, by the forward's blocks of 64: 24 (256 tokens, heads of 32) 53 and 37 us, 40 (512,
// heads of 64) 148 and 103, 72 (1024, heads of 128) 302 and 364, 136 (1024, heads of 32) 250 and 296.
bool small(int total, int B, int heads) { return blocks_of(total, B, heads, R) <= tc::num_sms() * 2 / 5; }

template <typename T, int DP, int N>
cudaError_t forward_n(const AttnArgs& a, cudaStream_t s) {
  constexpr int O = 16 * N;
  constexpr size_t smem = (tile_floats<DP>(O) + 2 * tile_floats<DP>(R) + O * PS) * sizeof(float);
  static Once once;
  return launch_tiles(once, simt_forward_kernel<T, DP, N>, dim3((unsigned)(a.Tq / O + a.B), a.Hq), smem, a, s);
}
template <typename T, int DP, int N>
cudaError_t dq_n(const AttnArgs& a, cudaStream_t s) {
  constexpr int O = 16 * N;
  constexpr size_t smem = (2 * tile_floats<DP>(O) + 2 * tile_floats<DP>(R) + (sizeof(T) == 2 ? 2 : 1) * O * PS) * sizeof(float);
  static Once once;
  return launch_tiles(once, simt_dq_kernel<T, DP, N>, dim3((unsigned)(a.Tq / O + a.B), a.Hq), smem, a, s);
}
template <int DP>
constexpr size_t dkv_bytes(int O) {
  return (2 * tile_floats<DP>(O) + 2 * tile_floats<DP>(R) + 2 * O * PS) * sizeof(float);
}
template <typename T, int DP, int N>
cudaError_t dkv_n(const AttnArgs& a, cudaStream_t s) {
  constexpr int O = 16 * N;
  static Once once;
  return launch_tiles(once, simt_dkv_kernel<T, DP, N>, dim3((unsigned)(a.Tk / O + a.B), a.Hkv), dkv_bytes<DP>(O), a, s);
}
template <int DP>
cudaError_t both(const AttnArgs& a, cudaStream_t s) {
  static Once once;
  const cudaError_t e = allow_smem(once, simt_both_kernel<DP>, dkv_bytes<DP>(16));  // more than dq's
  if (e != cudaSuccess) return e;
  const int key_tiles = a.Tk / 16 + a.B, query_tiles = a.Tq / 16 + a.B;
  return launch_after_smem(simt_both_kernel<DP>, dim3((unsigned)(key_tiles * a.Hkv + query_tiles * a.Hq)), kThreads, dkv_bytes<DP>(16),
                           s, a, key_tiles, query_tiles);
}

template <typename T, int DP>
cudaError_t forward(const AttnArgs& a, cudaStream_t s) {
  return small(a.Tq, a.B, a.Hq) ? forward_n<T, DP, 1>(a, s) : forward_n<T, DP, 4>(a, s);
}
template <typename T, int DP>
cudaError_t backward(const AttnArgs& a, cudaStream_t s) {
  const bool few_queries = small(a.Tq, a.B, a.Hq), few_keys = small(a.Tk, a.B, a.Hkv);
  // an SM for each: 204 blocks (512 tokens) took 87 us in one launch and 84 in two
  const bool together = blocks_of(a.Tq, a.B, a.Hq, 16) + blocks_of(a.Tk, a.B, a.Hkv, 16) <= tc::num_sms();
  if (sizeof(T) == 4 && together && few_queries && few_keys && a.Tq > 0 && a.Tk > 0) return both<DP>(a, s);
  cudaError_t e = cudaSuccess;
  if (a.Tq > 0) e = few_queries ? dq_n<T, DP, 1>(a, s) : dq_n<T, DP, 4>(a, s);
  if (e != cudaSuccess || a.Tk == 0) return e;
  return few_keys ? dkv_n<T, DP, 1>(a, s) : dkv_n<T, DP, 4>(a, s);
}

}  // namespace

cudaError_t launch_delta(const AttnArgs& a, bool bf16, cudaStream_t s) {
  const int64_t blocks = ceil_div((int64_t)a.Tq * a.Hq, kThreads / 32);
  if (blocks == 0) return cudaSuccess;
  if (bf16) delta_kernel<__nv_bfloat16><<<(unsigned)blocks, kThreads, 0, s>>>(a);
  else delta_kernel<float><<<(unsigned)blocks, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_simt(const AttnArgs& a, bool bf16, cudaStream_t s) {
  if (a.D <= 32) return bf16 ? forward<__nv_bfloat16, 32>(a, s) : forward<float, 32>(a, s);
  if (a.D <= 64) return bf16 ? forward<__nv_bfloat16, 64>(a, s) : forward<float, 64>(a, s);
  return bf16 ? forward<__nv_bfloat16, 128>(a, s) : forward<float, 128>(a, s);
}

cudaError_t launch_simt_backward(const AttnArgs& a, bool bf16, cudaStream_t s) {
  const cudaError_t e = launch_delta(a, bf16, s);
  if (e != cudaSuccess) return e;
  if (a.D <= 32) return bf16 ? backward<__nv_bfloat16, 32>(a, s) : backward<float, 32>(a, s);
  if (a.D <= 64) return bf16 ? backward<__nv_bfloat16, 64>(a, s) : backward<float, 64>(a, s);
  return bf16 ? backward<__nv_bfloat16, 128>(a, s) : backward<float, 128>(a, s);
}

}  // namespace attn
}  // namespace moe
