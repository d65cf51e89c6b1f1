// The norms and the residual around a block (attention or the MoE layer), and their backward:
//   u = y rho(y) w_post            (u = y without w_post)
//   r = res_scale x + g_t G_c u    (token gate g, channel gate G; 1 where absent)
//   n = r rho(r) w_next
// with rho(v) = 1 / sqrt(mean_c v_c^2 + eps). x and y are read once, r and n written once.
//
// What bounds it: DRAM, once the row sums are out of the way. A row group of TPR threads owns a
// row at a time and every thread the same channels of each row, so the per-channel weights stay
// in registers over the rows of a persistent CTA (w_post G is one product; read per row they
// would be more L2 traffic than the row itself). Rows arrive through a ring of cp.async stages
// in shared memory: a thread reads back only the 16-byte pieces it asked for itself, so the
// ring needs no barrier. The row sums do need one each, and a CTA that does nothing else
// meanwhile is bound by them; so the forward takes two rows through its two sums together, and
// the backward adds up one row while it finishes the row before. Products go two at a time
// (fma.f32x2): with the weights and conversions a row is otherwise near the issue limit.
// Widths that are not a multiple of 16 bytes move in pieces of 4 bytes, through the ring up to 2048
// (bf16) or 1024 (fp32) channels; odd bf16 widths in plain 2-byte loads.
#include <algorithm>
#include <atomic>

#include "step.cuh"

namespace moe {

namespace {

// Values in pairs where a piece holds more than one.
__device__ __forceinline__ float2 mul(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float fold(float2 a) { return a.x + a.y; }
__device__ __forceinline__ float fold(float a) { return a; }
__device__ __forceinline__ void splat(float v, float2* o) { *o = make_float2(v, v); }
__device__ __forceinline__ void splat(float v, float* o) { *o = v; }

template <typename T, int VEC>
struct Piece;  // VEC consecutive elements of a row, as loaded; N values of type E in fp32
template <>
struct Piece<float, 4> {
  using E = float2;
  static constexpr int N = 2;
  uint4 v;
  __device__ __forceinline__ void to(E (&f)[N]) const {
    f[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  __device__ __forceinline__ static Piece of(const E (&f)[N]) {
    return {make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y))};
  }
};
template <>
struct Piece<__nv_bfloat16, 8> {
  using E = float2;
  static constexpr int N = 4;
  uint4 v;
  __device__ __forceinline__ void to(E (&f)[N]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  __device__ __forceinline__ static Piece of(const E (&f)[N]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(f[i].x, f[i].y);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return {make_uint4(w[0], w[1], w[2], w[3])};
  }
};
template <>
struct Piece<__nv_bfloat16, 2> {
  using E = float2;
  static constexpr int N = 1;
  uint32_t v;
  __device__ __forceinline__ void to(E (&f)[N]) const {
    f[0] = make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
  __device__ __forceinline__ static Piece of(const E (&f)[N]) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(f[0].x, f[0].y);
    return {*reinterpret_cast<const uint32_t*>(&p)};
  }
};
template <>
struct Piece<float, 1> {
  using E = float;
  static constexpr int N = 1;
  float v;
  __device__ __forceinline__ void to(E (&f)[N]) const { f[0] = v; }
  __device__ __forceinline__ static Piece of(const E (&f)[N]) { return {f[0]}; }
};
template <>
struct Piece<__nv_bfloat16, 1> {
  using E = float;
  static constexpr int N = 1;
  __nv_bfloat16 v;
  __device__ __forceinline__ void to(E (&f)[N]) const { f[0] = __bfloat162float(v); }
  __device__ __forceinline__ static Piece of(const E (&f)[N]) { return {__float2bfloat16_rn(f[0])}; }
};

// One piece (16 or 4 bytes) from global to shared memory, asynchronously.
template <typename P>
__device__ __forceinline__ void cp_piece(P* dst, const P* src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  if constexpr (sizeof(P) == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Row sums of NV values over the TPR threads of a row group (blockDim = (TPR, groups), TPR a
// multiple of 32), in a fixed order, in two halves so that a barrier of the caller's stands
// between them. Both work on kP values at once (NV rounded up to a power of two): a lane ends
// up with the value lane / (32 / kP), which takes 9 shuffles for 8 values instead of 40.
// With CL > 1 a row's channels are spread over a cluster of CL CTAs, and every warp's sums are
// written to all of them (read from there, 28 loads of 250 cycles each came one after another).
constexpr int kMaxWarps = 32;
constexpr int kNormMaxSms = 152;  // bounds the grid, and so the backward's column partial sums
template <int NV, int CL>
struct RowSums {
  static constexpr int kP = NV <= 1 ? 1 : NV <= 2 ? 2 : NV <= 4 ? 4 : 8;
  static constexpr int kLanes = 32 / kP;
  float buf[2][kP * kMaxWarps * CL];  // [parity][group][value][CTA][warp]

  __device__ __forceinline__ void publish(const float (&in)[NV], int parity) {
    float v[kP];
#pragma unroll
    for (int i = 0; i < kP; ++i) v[i] = i < NV ? in[i < NV ? i : 0] : 0.0f;
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
    for (int n = kP / 2, off = 16; off; off >>= 1, n >>= 1) {
      if (n >= 1) {
        const bool upper = lane & off;
#pragma unroll
        for (int i = 0; i < kP / 2; ++i) {
          if (i < n) {
            const float send = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
          }
        }
      } else {
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
      }
    }
    if (lane % kLanes == 0) {
      const int rank = CL > 1 ? blockIdx.x % CL : 0;
      float* mine = buf[parity] + ((threadIdx.y * kP + lane / kLanes) * CL + rank) * warps + (threadIdx.x >> 5);
      if constexpr (CL == 1) {
        *mine = v[0];
      } else {
        const uint32_t here = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
#pragma unroll
        for (int r = 0; r < CL; ++r) {
          uint32_t at;
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(here), "r"(r));
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v[0]) : "memory");
        }
      }
    }
  }
  // The sums that were published with this parity, in every thread.
  __device__ __forceinline__ void total(float (&out)[NV], int parity) const {
    const int lane = threadIdx.x & 31, warps = (blockDim.x >> 5) * CL;
    const float* b = buf[parity] + (threadIdx.y * kP + lane / kLanes) * warps;
    float t = 0.0f;
    for (int w = lane % kLanes; w < warps; w += kLanes) t += b[w];
#pragma unroll
    for (int off = kLanes / 2; off; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
#pragma unroll
    for (int i = 0; i < NV; ++i) out[i] = __shfl_sync(0xffffffffu, t, i * kLanes);
  }
};

template <int CL>
__device__ __forceinline__ void row_barrier() {
  if constexpr (CL > 1)
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  else if (blockDim.x == 32) __syncwarp();  // a warp per row needs no barrier of the block
  else __syncthreads();
}

// A thread's pieces c = threadIdx.x + j TPR of a row's A arrays (of this CTA's share of the row,
// which begins at piece c0), from a ring of stages in shared
// memory (MAXT threads wide, so that a piece's place is a constant away from the stage's), or,
// with STAGES = 0, from global memory whenever they are asked for. An array that is not there
// (src NULL) and pieces past the row read as zeros: their places in the ring are zeroed once.
template <typename P, int A, int VPT, int MAXT, int STAGES>
struct Rows {
  static constexpr int kStage = A * VPT * MAXT;
  P* ring;
  const P* src[A];
  int T, nvec, c0;

  __device__ __forceinline__ int piece(int j) const { return c0 + threadIdx.x + j * blockDim.x; }
  __device__ __forceinline__ bool on(int j) const { return piece(j) < nvec; }
  __device__ __forceinline__ void zero_ring() const {
    P z{};
#pragma unroll
    for (int s = 0; s < STAGES; ++s)
#pragma unroll
      for (int a = 0; a < A; ++a)
#pragma unroll
        for (int j = 0; j < VPT; ++j)
          if (!src[a] || !on(j)) ring[s * kStage + (a * VPT + j) * MAXT] = z;
  }
  __device__ __forceinline__ void fetch(int64_t row, int stage) const {
    if (row >= T) return;
    const int64_t at = row * nvec + piece(0);
#pragma unroll
    for (int a = 0; a < A; ++a)
      if (src[a])
#pragma unroll
        for (int j = 0; j < VPT; ++j)
          if (on(j)) cp_piece(ring + stage * kStage + (a * VPT + j) * MAXT, src[a] + at + j * blockDim.x);
  }
  __device__ __forceinline__ void get(int64_t row, int stage, int a, int j, typename P::E (&f)[P::N]) const {
    if constexpr (STAGES > 0) {
      ring[stage * kStage + (a * VPT + j) * MAXT].to(f);
    } else {
      if (src[a] && row < T && on(j)) {
        src[a][row * nvec + piece(j)].to(f);
      } else {
#pragma unroll
        for (int e = 0; e < P::N; ++e) splat(0.0f, &f[e]);
      }
    }
  }
};

// Per-channel weights of a thread's piece c: a = w_post G, b = w_next (0 past the row and where
// there is no next norm).
template <typename P, int VEC>
__device__ __forceinline__ void channel_weights(const float* w_post, const float* gate, const float* w_next, int c, int nvec,
                                                typename P::E (&a)[P::N], typename P::E (&b)[P::N]) {
  float* fa = reinterpret_cast<float*>(a);
  float* fb = reinterpret_cast<float*>(b);
  if constexpr (VEC >= 4) {
#pragma unroll
    for (int e = 0; e < VEC; e += 4) {
      float4 u = make_float4(0, 0, 0, 0), n = u;
      if (c < nvec) {
        const int64_t at = ((int64_t)c * VEC + e) / 4;
        u = w_post ? __ldg(reinterpret_cast<const float4*>(w_post) + at) : make_float4(1, 1, 1, 1);
        if (gate) {
          const float4 g = __ldg(reinterpret_cast<const float4*>(gate) + at);
          u.x *= g.x, u.y *= g.y, u.z *= g.z, u.w *= g.w;
        }
        if (w_next) n = __ldg(reinterpret_cast<const float4*>(w_next) + at);
      }
      fa[e] = u.x, fa[e + 1] = u.y, fa[e + 2] = u.z, fa[e + 3] = u.w;
      fb[e] = n.x, fb[e + 1] = n.y, fb[e + 2] = n.z, fb[e + 3] = n.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const bool in = c < nvec;
      float v = !in ? 0.0f : w_post ? __ldg(w_post + c * VEC + e) : 1.0f;
      if (in && gate) v *= __ldg(gate + c * VEC + e);
      fa[e] = v;
      fb[e] = in && w_next ? __ldg(w_next + c * VEC + e) : 0.0f;
    }
  }
}

__device__ __forceinline__ float inv_rms(float sum, float inv_h, float eps) { return rsqrtf(fmaf(sum, inv_h, eps)); }

// ROWS rows per iteration: i ROWS + k is row (first + (i ROWS + k) step) of the group.
template <typename T, int VEC, int VPT, bool CACHE_W, int MAXT, int STAGES, int CL, int ROWS>
__global__ void __launch_bounds__(MAXT, MAXT <= 128 ? 4 : MAXT <= 256 || (MAXT <= 512 && STAGES == 0) ? 2 : 1)
    block_norm_kernel(NormIn in, void* r_out, void* n_out, int T_, int H, float eps, float res_scale) {
  using P = Piece<T, VEC>;
  using E = typename P::E;
  constexpr int N = P::N;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ RowSums<ROWS, CL> sums;
  const int groups = blockDim.y, nvec = H / VEC;
  const float inv_h = 1.0f / (float)H;
  const int cta = blockIdx.x / CL;  // of the row groups' walkers
  // this CTA's share of a row's pieces: VPT per thread
  const int share0 = CL > 1 ? (int)(blockIdx.x % CL * blockDim.x) * VPT : 0;
  using R = Rows<P, 2, VPT, MAXT, STAGES * ROWS>;
  const R rows{reinterpret_cast<P*>(smem) + threadIdx.y * blockDim.x + threadIdx.x,
               {static_cast<const P*>(in.x), static_cast<const P*>(in.y)}, T_, nvec, share0};
  const int64_t step = (int64_t)gridDim.x / CL * groups;
  int64_t row0 = (int64_t)cta * groups + threadIdx.y;
  // the same for every group of the CTA: the rows of its first one
  const int iters = (int)ceil_div(ceil_div(T_ - (int64_t)cta * groups, step), ROWS);
  rows.zero_ring();
  if constexpr (CL > 1) row_barrier<CL>();  // the whole cluster runs before its shared memory is written
  auto fetch = [&](int64_t row, int stage) {
    if constexpr (STAGES > 0) {
#pragma unroll
      for (int k = 0; k < ROWS; ++k) rows.fetch(row + k * step, stage * ROWS + k);
      cp_commit();
    }
  };
#pragma unroll
  for (int i = 0; i < STAGES; ++i) fetch(row0 + i * ROWS * step, i);

  E wu[CACHE_W ? VPT : 1][N], wn[CACHE_W ? VPT : 1][N];
  auto weights = [&](int j) {
    channel_weights<P, VEC>(in.w_post, in.gate, n_out ? in.w_next : nullptr, rows.piece(j), nvec, wu[CACHE_W ? j : 0], wn[CACHE_W ? j : 0]);
  };
  if constexpr (CACHE_W) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) weights(j);
  }
  E scale;
  splat(res_scale, &scale);

  int stage = 0;
  for (int it = 0; it < iters; ++it, row0 += ROWS * step) {
    if constexpr (STAGES > 0) cp_wait<(STAGES > 0 ? STAGES - 1 : 0)>();
    float su[ROWS], s[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) su[k] = 1.0f;
    if (in.w_post) {
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        E t;
        splat(0.0f, &t);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
          E y[N];
          rows.get(row0 + k * step, stage * ROWS + k, 1, j, y);
#pragma unroll
          for (int e = 0; e < N; ++e) t = fma(y[e], y[e], t);
        }
        s[k] = fold(t);
      }
      sums.publish(s, 0);
      row_barrier<CL>();
      sums.total(s, 0);
#pragma unroll
      for (int k = 0; k < ROWS; ++k) su[k] = inv_rms(s[k], inv_h, eps);
    }
    E v[ROWS][VPT][N];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const int64_t row = row0 + k * step;
      if (in.token_gate && row < T_) su[k] *= __ldg(in.token_gate + row);
      E f, t;
      splat(su[k], &f);
      splat(0.0f, &t);
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        E y[N];
        rows.get(row, stage * ROWS + k, 0, j, v[k][j]);
        rows.get(row, stage * ROWS + k, 1, j, y);
        if constexpr (!CACHE_W) weights(j);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          v[k][j][e] = fma(mul(y[e], f), wu[CACHE_W ? j : 0][e], mul(v[k][j][e], scale));
          t = fma(v[k][j][e], v[k][j][e], t);
        }
        if (r_out && row < T_ && rows.on(j))
          static_cast<P*>(r_out)[row * nvec + rows.piece(j)] = P::of(v[k][j]);
      }
      s[k] = fold(t);
    }
    // the stage has been read; its next rows are asked for
    fetch(row0 + STAGES * ROWS * step, stage);
    if (STAGES > 0 && ++stage == STAGES) stage = 0;
    if (n_out) {
      sums.publish(s, 1);
      row_barrier<CL>();
      sums.total(s, 1);
      // n is formed from r before its rounding to the activation type
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        const int64_t row = row0 + k * step;
        E f;
        splat(inv_rms(s[k], inv_h, eps), &f);
        if (row < T_) {
#pragma unroll
          for (int j = 0; j < VPT; ++j) {
            if constexpr (!CACHE_W) weights(j);
            if (!rows.on(j)) continue;
#pragma unroll
            for (int e = 0; e < N; ++e) v[k][j][e] = mul(mul(v[k][j][e], f), wn[CACHE_W ? j : 0][e]);
            static_cast<P*>(n_out)[row * nvec + rows.piece(j)] = P::of(v[k][j]);
          }
        }
      }
    }
    // with one sum in use, its buffer is free again only after a second barrier
    if ((in.w_post != nullptr) != (n_out != nullptr)) row_barrier<CL>();
  }
}

// Backward, per row, from the stored residual r and block output y (both statistics are
// formed again from them, so nothing else is kept from the forward):
//   a = dn w_next;  dr' = dr + rho_r a - k r,  k = rho_r^3 (sum_c a r) / H;   dx = res_scale dr'
//   w = G w_post;  q = sum_c w dr' y;  dy = g (rho_y w dr' - rho_y^3 y q / H)
//   dtoken_gate = rho_y q
//   column sums over the rows: N = sum dn r rho_r = dw_next, S = sum g dr' y rho_y, from which
//   dw_post = G S and dgate = w_post S (without w_post: rho_y = 1, dy = g w dr', dgate = S).
// q is linear in dr', so q = sum w dr y + rho_r sum w a y - k sum w r y, and all six sums of a
// row are formed in one go; row i's sums are added while row i - 1 is finished. Each term of q
// is rounded relative to its own size, as the terms of dr' would be.
// Each CTA keeps the column sums of its rows in registers and writes them once; colsum_kernel
// adds the CTAs' sums in a fixed order.
template <typename T, int VEC, int VPT, bool CACHE_W, int MAXT, int STAGES, int CL>
__global__ void __launch_bounds__(MAXT, MAXT <= 128 ? 4 : MAXT <= 256 || (MAXT <= 512 && STAGES == 0) ? 2 : 1)
    block_norm_bwd_kernel(NormBwd b, float* part, int T_, int H, float eps, float res_scale) {
  let_next_begin();
  using P = Piece<T, VEC>;
  using E = typename P::E;
  constexpr int N = P::N;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ RowSums<6, CL> sums;
  const int groups = blockDim.y, nvec = H / VEC;
  const float inv_h = 1.0f / (float)H;
  const int cta = blockIdx.x / CL;  // of the row groups' walkers
  // this CTA's share of a row's pieces: VPT per thread
  const int share0 = CL > 1 ? (int)(blockIdx.x % CL * blockDim.x) * VPT : 0;
  const bool need_s = b.dgate || b.dw_post;
  enum { R = 0, Y = 1, DR = 2, DN = 3 };
  using Ring = Rows<P, 4, VPT, MAXT, STAGES>;
  const Ring rows{reinterpret_cast<P*>(smem) + threadIdx.y * blockDim.x + threadIdx.x,
                  {b.w_next ? static_cast<const P*>(b.r) : nullptr, static_cast<const P*>(b.y),
                   static_cast<const P*>(b.dr), static_cast<const P*>(b.dn)},
                  T_, nvec, share0};
  const int64_t step = (int64_t)gridDim.x / CL * groups;
  int64_t row = (int64_t)cta * groups + threadIdx.y - step;  // the row that is finished, one behind the sums
  const int iters = (int)ceil_div(T_ - (int64_t)cta * groups, step);
  rows.zero_ring();
  if constexpr (CL > 1) row_barrier<CL>();  // the whole cluster runs before its shared memory is written
  if constexpr (STAGES > 0) {
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) {
      rows.fetch(row + (i + 1) * step, i);
      cp_commit();
    }
  }

  E wu[CACHE_W ? VPT : 1][N], wn[CACHE_W ? VPT : 1][N], colS[VPT][N], colN[VPT][N];
  auto weights = [&](int j) {
    channel_weights<P, VEC>(b.w_post, b.gate, b.w_next, rows.piece(j), nvec, wu[CACHE_W ? j : 0], wn[CACHE_W ? j : 0]);
  };
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    if constexpr (CACHE_W) weights(j);
#pragma unroll
    for (int e = 0; e < N; ++e) splat(0.0f, &colS[j][e]), splat(0.0f, &colN[j][e]);
  }

  int stage = 0, prev = STAGES > 0 ? STAGES - 1 : 0;  // of row + step, whose sums are formed, and of row
  for (int it = 0; it <= iters; ++it, row += step) {
    const int parity = it & 1;
    if constexpr (STAGES > 0) cp_wait<(STAGES > 2 ? STAGES - 2 : 0)>();
    float tot[6] = {0, 0, 0, 0, 0, 0};
    if (it > 0) sums.total(tot, parity ^ 1);
    if (it < iters) {
      E s[6];
#pragma unroll
      for (int i = 0; i < 6; ++i) splat(0.0f, &s[i]);
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        E r[N], y[N], dr[N], dn[N];
        rows.get(row + step, stage, R, j, r);
        rows.get(row + step, stage, Y, j, y);
        rows.get(row + step, stage, DR, j, dr);
        rows.get(row + step, stage, DN, j, dn);
        if constexpr (!CACHE_W) weights(j);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const E a = mul(dn[e], wn[CACHE_W ? j : 0][e]), wy = mul(y[e], wu[CACHE_W ? j : 0][e]);
          s[0] = fma(r[e], r[e], s[0]);
          s[1] = fma(a, r[e], s[1]);
          s[2] = fma(y[e], y[e], s[2]);
          s[3] = fma(dr[e], wy, s[3]);
          s[4] = fma(a, wy, s[4]);
          s[5] = fma(r[e], wy, s[5]);
        }
      }
      const float f[6] = {fold(s[0]), fold(s[1]), fold(s[2]), fold(s[3]), fold(s[4]), fold(s[5])};
      sums.publish(f, parity);
    }
    if (it > 0 && row < T_) {
      const float rho = b.w_next ? inv_rms(tot[0], inv_h, eps) : 0.0f;
      const float k = rho * (rho * (rho * tot[1]) * inv_h);  // rho^3 alone may overflow where the sum is 0
      const float rho_y = b.w_post ? inv_rms(tot[2], inv_h, eps) : 1.0f;
      const float g = b.token_gate ? __ldg(b.token_gate + row) : 1.0f;
      const float q = fmaf(rho, tot[4], fmaf(-k, tot[5], tot[3]));
      if (b.dtoken_gate && threadIdx.x == 0 && share0 == 0) b.dtoken_gate[row] = rho_y * q;
      E e_rho, e_k, e_g, e_ky, e_res;
      splat(rho, &e_rho);
      splat(-k, &e_k);
      splat(g * rho_y, &e_g);
      splat(b.w_post ? -g * rho_y * (rho_y * (rho_y * q) * inv_h) : 0.0f, &e_ky);
      splat(res_scale, &e_res);
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        E r[N], y[N], d[N], dn[N], o[N];
        rows.get(row, prev, R, j, r);
        rows.get(row, prev, Y, j, y);
        rows.get(row, prev, DR, j, d);
        rows.get(row, prev, DN, j, dn);
        if constexpr (!CACHE_W) weights(j);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const E p = mul(dn[e], e_rho);  // rho dn
          d[e] = fma(p, wn[CACHE_W ? j : 0][e], fma(e_k, r[e], d[e]));
          colN[j][e] = fma(p, r[e], colN[j][e]);
          const E gd = mul(e_g, d[e]);
          colS[j][e] = fma(gd, y[e], colS[j][e]);
          o[e] = fma(gd, wu[CACHE_W ? j : 0][e], mul(e_ky, y[e]));
          d[e] = mul(d[e], e_res);
        }
        if (rows.on(j)) {
          const int64_t at = row * nvec + rows.piece(j);
          if (b.dx) static_cast<P*>(b.dx)[at] = P::of(d);
          if (b.dy) static_cast<P*>(b.dy)[at] = P::of(o);
        }
      }
    }
    if constexpr (STAGES > 0) {  // row's stage has been read (in iteration 0: was never filled)
      rows.fetch(row + (int64_t)STAGES * step, prev);
      cp_commit();
      prev = stage;
      if (++stage == STAGES) stage = 0;
    }
    row_barrier<CL>();
  }
  if (need_s || b.dw_next) {  // [2][gridDim.x * groups][H]
    const int64_t p = (int64_t)cta * groups + threadIdx.y, np = (int64_t)gridDim.x / CL * groups;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = rows.piece(j);
      if (c < nvec) {
        E* ps = reinterpret_cast<E*>(part + p * H + c * VEC);
        E* pn = reinterpret_cast<E*>(part + (np + p) * H + c * VEC);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          if (need_s) ps[e] = colS[j][e];
          if (b.dw_next) pn[e] = colN[j][e];
        }
      }
    }
  }
}

// Adds the partial column sums [np][H] in a fixed order: 32 columns per block, 32 lanes of
// partials each, then the lanes. blockIdx.y: 0 the S sums, 1 the N sums.
__global__ void __launch_bounds__(1024) colsum_kernel(const float* part, int np, int H, NormBwd b) {
  __shared__ float acc[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x;
  const bool second = blockIdx.y == 1;
  after_previous();
  if (second ? !b.dw_next : !(b.dgate || b.dw_post)) return;
  const float* p = part + (second ? (int64_t)np * H : 0);
  float v = 0.0f;
  if (col < H)
    for (int i = threadIdx.y; i < np; i += 32) v += p[(int64_t)i * H + col];
  acc[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y != 0 || col >= H) return;
  v = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) v += acc[i][threadIdx.x];
  if (second) {
    b.dw_next[col] = v;
  } else {
    if (b.dgate) b.dgate[col] = b.w_post ? v * b.w_post[col] : v;
    if (b.dw_post) b.dw_post[col] = b.gate ? v * b.gate[col] : v;
  }
}

// Threads per row (of one CTA of its cluster) and rows per CTA.
struct Shape {
  int tpr, groups;
};
Shape shape_of(int nvec, int vpt, int maxt, int cl) {
  Shape s;
  s.tpr = (int)(ceil_div(ceil_div(nvec, vpt * cl), 32) * 32);
  s.groups = cl > 1 ? 1 : std::max(1, std::min(maxt, 256) / s.tpr);
  return s;
}

// Row walkers of an instantiation that are resident together, by the threads of a row, on which
// alone they depend (0: not asked for yet). The last answer by itself cost 0.9 us a call where widths
// of one instantiation come in turn (12288 and 16384 channels backward, 5.5 us a call).
using Resident = std::atomic<uint16_t>[1024 / 32 + 1];

// Persistent launch of an instantiation.
template <int CL, typename K, typename... Args>
cudaError_t launch_rows(K kern, Resident& resident, const Shape& sh, size_t smem, int64_t T, cudaStream_t s,
                        int* walkers, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(sh.tpr, sh.groups);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CL;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CL > 1 ? 1 : 0;
  const int sms = std::min(tc::num_sms(), kNormMaxSms);
  int known = resident[sh.tpr / 32].load(std::memory_order_relaxed);
  if (!known) {
    cudaError_t e = cudaSuccess;
    if (smem > 32 * 1024) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    int fit = 0;
    if constexpr (CL > 1) {
      cfg.gridDim = dim3(CL * (sms / CL));
      e = cudaOccupancyMaxActiveClusters(&fit, kern, &cfg);
    } else {
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kern, sh.tpr * sh.groups, smem);
      fit *= sms;
    }
    if (e != cudaSuccess) return e;
    known = std::max(1, std::min(fit, sms * (2048 / (sh.tpr * sh.groups)) / CL));
    resident[sh.tpr / 32].store((uint16_t)known, std::memory_order_relaxed);
  }
  *walkers = (int)std::min<int64_t>(ceil_div(T, sh.groups), known);
  cfg.gridDim = dim3((unsigned)(*walkers * CL));
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Two rows an iteration, but without the ring there are no registers for them.
template <typename T, int VEC, int VPT, bool CACHE_W, int MAXT, int STAGES, int CL, int ROWS = (STAGES > 0 ? 2 : 1)>
cudaError_t fwd(const moe_norm_config_t& c, const NormIn& in, void* r, void* n, cudaStream_t s) {
  const size_t smem = (size_t)STAGES * ROWS * 2 * VPT * MAXT * sizeof(Piece<T, VEC>);
  static Resident resident;
  int walkers = 0;
  return launch_rows<CL>(block_norm_kernel<T, VEC, VPT, CACHE_W, MAXT, STAGES, CL, ROWS>, resident, shape_of(c.H / VEC, VPT, MAXT, CL),
                         smem, c.T, s, &walkers, in, r, n, c.T, c.H, c.eps, c.res_scale);
}

template <typename T, int VEC, int VPT, bool CACHE_W, int MAXT, int STAGES, int CL>
cudaError_t bwd(const moe_norm_config_t& c, const NormBwd& b, float* part, cudaStream_t s) {
  const Shape sh = shape_of(c.H / VEC, VPT, MAXT, CL);
  const size_t smem = (size_t)STAGES * 4 * VPT * MAXT * sizeof(Piece<T, VEC>);
  static Resident resident;
  int walkers = 0;
  cudaError_t e = launch_rows<CL>(block_norm_bwd_kernel<T, VEC, VPT, CACHE_W, MAXT, STAGES, CL>, resident, sh, smem, c.T, s,
                                  &walkers, b, part, c.T, c.H, c.eps, c.res_scale);
  if (e != cudaSuccess || !(b.dgate || b.dw_post || b.dw_next)) return e;
  return launch_after(colsum_kernel, dim3((unsigned)ceil_div(c.H, 32), 2), dim3(32, 32), s, part, walkers * sh.groups, c.H, b);
}

// How a row is spread, by the number of its pieces of 16 bytes. All: the fewest stages of the ring
// that keep a row or two in flight, so that an SM holds several CTAs (backward with 4 instead of 3:
// 80 against 78 us; forward with 3 instead of 2: 50 against 47).
//
// Forward: one piece per thread up to 1024 (more threads hide its two barriers: 16384 x 2048 49
// against 51 us, 8192 x 4096 49 against 52, 8192 x 7168 77 against 79), then two, a row an iteration
// (of two there would be no shared memory for a second stage; a cluster of two CTAs instead, with
// its barriers of 1 us: 4096 x 16384 134 against 115 us, 4096 x 7168 fp32 123 against 85).
template <typename T, int VEC>
cudaError_t fwd_wide(const moe_norm_config_t& c, const NormIn& in, void* r, void* n, cudaStream_t s) {
  const int nvec = c.H / VEC;
  if (nvec <= 32) return fwd<T, VEC, 1, true, 128, 2, 1>(c, in, r, n, s);
  if (nvec <= 256) return fwd<T, VEC, 1, true, 256, 2, 1>(c, in, r, n, s);
  if (nvec <= 512) return fwd<T, VEC, 1, true, 512, 2, 1>(c, in, r, n, s);
  if (nvec <= 1024) return fwd<T, VEC, 1, true, 1024, 2, 1>(c, in, r, n, s);
  if constexpr (VEC == 4) {
    if (nvec > 2048) return fwd<T, VEC, 2, true, 1024, 3, 2, 1>(c, in, r, n, s);  // 4096 x 16384: 257 us, 266 in four of 512 threads
  }
  return fwd<T, VEC, 2, true, 1024, 3, 1, 1>(c, in, r, n, s);
}

// Backward: two pieces per thread, since its bookkeeping per row and thread is near half of its
// instructions (16384 x 2048: 80 against 88 us with one; 8192 x 7168: 141 against 203). Its columns'
// sums leave no registers for more than 512 threads in a CTA; wider rows take a cluster of four (of
// 512 threads, where one to an SM finds nothing to do during the cluster's barrier: 4096 x 16384 257
// against 232 us, 4096 x 7168 fp32 191 against 175; of eight: 281, 258).
template <typename T, int VEC>
cudaError_t bwd_wide(const moe_norm_config_t& c, const NormBwd& b, float* part, cudaStream_t s) {
  const int nvec = c.H / VEC;
  if (nvec <= 32) return bwd<T, VEC, 1, true, 128, 3, 1>(c, b, part, s);
  if (nvec <= 256) return bwd<T, VEC, 2, true, 128, 3, 1>(c, b, part, s);
  if (nvec <= 512) return bwd<T, VEC, 2, true, 256, 3, 1>(c, b, part, s);
  if (nvec <= 1024) return bwd<T, VEC, 2, true, 512, 3, 1>(c, b, part, s);
  if constexpr (VEC == 4) {
    if (nvec > 2048) return bwd<T, VEC, 2, true, 512, 3, 4>(c, b, part, s);
  }
  return bwd<T, VEC, 2, true, 256, 3, 4>(c, b, part, s);
}

}  // namespace

// Rows of H not a multiple of 16 bytes have pieces of 4 bytes (4 to 16 per thread); an odd number
// of bf16 channels leaves nothing for cp.async to copy, and takes single elements without the ring.
// STAGES: of the ring of 4-byte pieces.
#define NORM_DISPATCH(FN, STAGES, ...)                                                            \
  if (c.act_dtype == MOE_DTYPE_BF16 && c.H % 8 == 0) return FN##_wide<__nv_bfloat16, 8>(__VA_ARGS__); \
  if (c.act_dtype == MOE_DTYPE_F32 && c.H % 4 == 0) return FN##_wide<float, 4>(__VA_ARGS__);      \
  if (c.act_dtype == MOE_DTYPE_BF16 && c.H % 2 == 0) {                                            \
    if (c.H <= 2048) return FN<__nv_bfloat16, 2, 4, true, 256, STAGES, 1>(__VA_ARGS__);           \
    return FN<__nv_bfloat16, 2, 8, false, 1024, 0, 1>(__VA_ARGS__);                               \
  }                                                                                               \
  if (c.act_dtype == MOE_DTYPE_BF16) {                                                            \
    if (c.H <= 2048) return FN<__nv_bfloat16, 1, 4, true, 512, 0, 1>(__VA_ARGS__);                \
    return FN<__nv_bfloat16, 1, 16, false, 1024, 0, 1>(__VA_ARGS__);                              \
  }                                                                                               \
  if (c.H <= 1024) return FN<float, 1, 4, true, 256, STAGES, 1>(__VA_ARGS__);                     \
  if (c.H <= 2048) return FN<float, 1, 4, true, 512, 0, 1>(__VA_ARGS__);                          \
  return FN<float, 1, 16, false, 1024, 0, 1>(__VA_ARGS__);

cudaError_t launch_block_norm(const moe_norm_config_t& c, const NormIn& in, void* r, void* n, cudaStream_t s) {
  if (c.T == 0) return cudaSuccess;
  NORM_DISPATCH(fwd, 2, c, in, r, n, s)
}

cudaError_t launch_block_norm_backward(const moe_norm_config_t& c, const NormBwd& b, float* part, cudaStream_t s) {
  if (c.T == 0) {
    cudaError_t e = cudaSuccess;
    for (float* p : {b.dw_post, b.dw_next, b.dgate})
      if (p && e == cudaSuccess) e = cudaMemsetAsync(p, 0, (size_t)c.H * 4, s);
    return e;
  }
  NORM_DISPATCH(bwd, 4, c, b, part, s)
}

// Two sets of column sums for every row group of the largest grid: never more than one row
// group per row, nor than 2048 threads of them on each of 152 SMs. A row has at least H / 16
// threads.
size_t norm_part_bytes(const moe_norm_config_t& c) {
  const int64_t threads = align_up((size_t)ceil_div(c.H, 16), 32);
  const int64_t groups = std::min<int64_t>((int64_t)c.T + 8, (int64_t)kNormMaxSms * 2048 / threads);
  return (size_t)(2 * groups * c.H * 4);
}

}  // namespace moe
