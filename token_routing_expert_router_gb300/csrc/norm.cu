// The norms and the residual around a block (attention or the MoE layer), and their backward:
//   u = y rho(y) w_post            (u = y without w_post)
//   r = res_scale x + g_t G_c u    (token gate g, channel gate G; 1 where absent)
//   n = r rho(r) w_next
// with rho(v) = 1 / sqrt(mean_c v_c^2 + eps). One pass: x and y are read once, r and n
// written once; the two row sums are taken from registers.
//
// What bounds it: DRAM. A row group of TPR threads owns a row at a time and every thread the
// same channels of each row, so the per-channel weights stay in registers over the rows of a
// persistent CTA (w_post G is one product; read per row they would be more L2 traffic than
// the row itself). Rows arrive through a ring of cp.async stages in shared memory: a thread
// reads back only the 16-byte pieces it asked for itself, so the ring needs no barrier, and
// it keeps several rows in flight per CTA while the row sums of the current one are formed.
// Widths that are not a multiple of 16 bytes take plain element loads (VEC = 1).
#include <algorithm>
#include <atomic>

#include "step.cuh"

namespace moe {

namespace {

template <typename T, int VEC>
struct Piece;  // VEC consecutive elements of a row, as loaded
template <>
struct Piece<float, 4> {
  uint4 v;
  __device__ void to(float (&f)[4]) const {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
  }
  __device__ static Piece of(const float (&f)[4]) {
    return {make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]))};
  }
};
template <>
struct Piece<__nv_bfloat16, 8> {
  uint4 v;
  __device__ void to(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static Piece of(const float (&f)[8]) {
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
struct Piece<float, 1> {
  float v;
  __device__ void to(float (&f)[1]) const { f[0] = v; }
  __device__ static Piece of(const float (&f)[1]) { return {f[0]}; }
};
template <>
struct Piece<__nv_bfloat16, 1> {
  __nv_bfloat16 v;
  __device__ void to(float (&f)[1]) const { f[0] = __bfloat162float(v); }
  __device__ static Piece of(const float (&f)[1]) { return {__float2bfloat16_rn(f[0])}; }
};

__device__ __forceinline__ void cp16(void* dst, const void* src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Sums NV values over the TPR threads of each row group (blockDim = (TPR, groups), TPR a
// multiple of 32) in a fixed order; every thread gets the sums. `buf` holds NV floats per
// warp; the caller alternates two buffers, so one barrier per call is enough.
template <int NV>
__device__ __forceinline__ void row_sum(float (&v)[NV], float* buf) {
#pragma unroll
  for (int off = 16; off; off >>= 1)
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  float* b = buf + threadIdx.y * warps * NV;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < NV; ++i) b[(threadIdx.x >> 5) * NV + i] = v[i];
  __syncthreads();
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float t = lane < warps ? b[lane * NV + i] : 0.0f;
#pragma unroll
    for (int off = 16; off; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
    v[i] = t;
  }
}

constexpr int kMaxWarps = 32;
constexpr int kNormMaxSms = 152;  // bounds the grid, and so the backward's column partial sums

// The ring of row stages: A arrays per row, VPT pieces per thread and array. Slot of
// (stage, array, piece) for this thread: consecutive threads are 16 bytes apart.
template <typename P, int A, int VPT, int STAGES>
struct Ring {
  P* base;
  int threads, tid;
  __device__ P* slot(int stage, int a, int j) const {
    return base + ((stage * A + a) * VPT + j) * threads + tid;
  }
};

template <typename T, int VEC, int VPT, bool CACHE_W, int MAXT, int STAGES>
__global__ void __launch_bounds__(MAXT)
    block_norm_kernel(NormIn in, void* r_out, void* n_out, int T_, int H, float eps, float res_scale) {
  using P = Piece<T, VEC>;
  constexpr bool kAsync = STAGES > 0;
  constexpr int kStages = kAsync ? STAGES : 1;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float sums[2][kMaxWarps];
  int flip = 0;
  const int tpr = blockDim.x, groups = blockDim.y;
  const Ring<P, 2, VPT, kStages> ring{reinterpret_cast<P*>(smem), tpr * groups, (int)(threadIdx.y * tpr + threadIdx.x)};
  const int nvec = H / VEC;
  const P* x = static_cast<const P*>(in.x);
  const P* y = static_cast<const P*>(in.y);
  const float inv_h = 1.0f / (float)H;

  float wu[CACHE_W ? VPT : 1][VEC], wn[CACHE_W ? VPT : 1][VEC];
  auto channel_weights = [&](int c, float (&a)[VEC], float (&b)[VEC]) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int h = c * VEC + e;
      float v = in.w_post ? __ldg(in.w_post + h) : 1.0f;
      if (in.gate) v *= __ldg(in.gate + h);
      a[e] = v;
      b[e] = n_out ? __ldg(in.w_next + h) : 0.0f;
    }
  };
  if constexpr (CACHE_W) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = threadIdx.x + j * tpr;
      if (c < nvec) channel_weights(c, wu[j], wn[j]);
    }
  }

  const int64_t step = (int64_t)gridDim.x * groups;
  int64_t row = (int64_t)blockIdx.x * groups + threadIdx.y;
  const int64_t iters = ceil_div(T_ - (int64_t)blockIdx.x * groups, step);  // the same for every group of the CTA
  auto fetch = [&](int64_t rw, int stage) {
    if constexpr (kAsync) {
      if (rw < T_) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
          const int c = threadIdx.x + j * tpr;
          if (c < nvec) {
            cp16(ring.slot(stage, 0, j), x + rw * nvec + c);
            if (y) cp16(ring.slot(stage, 1, j), y + rw * nvec + c);
          }
        }
      }
      cp_commit();
    }
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(row + i * step, i);
  int stage = 0;
  for (int64_t it = 0; it < iters; ++it, row += step) {
    if constexpr (kAsync) {
      // the stage asked for now was read one iteration ago, by this thread alone
      fetch(row + (kStages - 1) * step, (stage + kStages - 1) % kStages);
      cp_wait<kStages - 1>();
    }
    const bool live = row < T_;
    float v[VPT][VEC], s1[1] = {0.0f};
    float yv[VPT][VEC];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = threadIdx.x + j * tpr;
      const bool on = live && c < nvec;
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[j][e] = yv[j][e] = 0.0f;
      if (on) {
        if constexpr (kAsync) {
          ring.slot(stage, 0, j)->to(v[j]);
          if (y) ring.slot(stage, 1, j)->to(yv[j]);
        } else {
          x[row * nvec + c].to(v[j]);
          if (y) y[row * nvec + c].to(yv[j]);
        }
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) s1[0] = fmaf(yv[j][e], yv[j][e], s1[0]);
    }
    float su = 1.0f;
    if (in.w_post) {
      row_sum(s1, sums[flip ^= 1]);
      su = 1.0f / sqrtf(fmaf(s1[0], inv_h, eps));
    }
    if (in.token_gate && live) su *= __ldg(in.token_gate + row);
    float s2[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = threadIdx.x + j * tpr;
      float a[VEC], b[VEC];
      if constexpr (!CACHE_W)
        if (c < nvec) channel_weights(c, a, b);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        v[j][e] *= res_scale;
        if (y && c < nvec) v[j][e] = fmaf(yv[j][e] * su, CACHE_W ? wu[CACHE_W ? j : 0][e] : a[e], v[j][e]);
        s2[0] = fmaf(v[j][e], v[j][e], s2[0]);
      }
      if (r_out && live && c < nvec) static_cast<P*>(r_out)[row * nvec + c] = P::of(v[j]);
    }
    if (n_out) {
      row_sum(s2, sums[flip ^= 1]);
      // n is formed from r before its rounding to the activation type
      const float rho = 1.0f / sqrtf(fmaf(s2[0], inv_h, eps));
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int c = threadIdx.x + j * tpr;
        if (live && c < nvec) {
          float a[VEC], b[VEC], o[VEC];
          if constexpr (!CACHE_W) channel_weights(c, a, b);
#pragma unroll
          for (int e = 0; e < VEC; ++e) o[e] = v[j][e] * rho * (CACHE_W ? wn[CACHE_W ? j : 0][e] : b[e]);
          static_cast<P*>(n_out)[row * nvec + c] = P::of(o);
        }
      }
    }
    if constexpr (kAsync) stage = (stage + 1) % kStages;
  }
}

// Backward, per row, from the stored residual r and block output y (both statistics are
// formed again from them, so nothing else is kept from the forward):
//   a = dn w_next;  dr' = dr + rho_r a - rho_r^3 r (sum_c a r) / H;   dx = res_scale dr'
//   b = G w_post dr';  q = sum_c b y;  dy = g (rho_y b - rho_y^3 y q / H)
//   dtoken_gate = rho_y q
//   column sums over the rows: N = sum dn r rho_r = dw_next, S = sum g dr' y rho_y, from which
//   dw_post = G S and dgate = w_post S (without w_post: rho_y = 1, dy = g b, dgate = S).
// Each CTA keeps the column sums of its rows in registers and writes them once; colsum_kernel
// adds the CTAs' sums in a fixed order.
template <typename T, int VEC, int VPT, bool CACHE_W, int MAXT, int STAGES>
__global__ void __launch_bounds__(MAXT)
    block_norm_bwd_kernel(NormBwd b, float* part, int T_, int H, float eps, float res_scale) {
  using P = Piece<T, VEC>;
  constexpr bool kAsync = STAGES > 0;
  constexpr int kStages = kAsync ? STAGES : 1;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float sums[2][3 * kMaxWarps];
  int flip = 0;
  const int tpr = blockDim.x, groups = blockDim.y;
  const Ring<P, 4, VPT, kStages> ring{reinterpret_cast<P*>(smem), tpr * groups, (int)(threadIdx.y * tpr + threadIdx.x)};
  const int nvec = H / VEC;
  const P* src[4] = {b.w_next ? static_cast<const P*>(b.r) : nullptr, static_cast<const P*>(b.y),
                     static_cast<const P*>(b.dr), static_cast<const P*>(b.dn)};
  const float inv_h = 1.0f / (float)H;
  const bool need_s = b.dgate || b.dw_post;

  float wu[CACHE_W ? VPT : 1][VEC], wn[CACHE_W ? VPT : 1][VEC];
  float colS[VPT][VEC], colN[VPT][VEC];
  auto channel_weights = [&](int c, float (&wa)[VEC], float (&wb)[VEC]) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int h = c * VEC + e;
      float v = b.w_post ? __ldg(b.w_post + h) : 1.0f;
      if (b.gate) v *= __ldg(b.gate + h);
      wa[e] = v;
      wb[e] = b.w_next ? __ldg(b.w_next + h) : 0.0f;
    }
  };
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    if constexpr (CACHE_W) {
      const int c = threadIdx.x + j * tpr;
      if (c < nvec) channel_weights(c, wu[j], wn[j]);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) colS[j][e] = colN[j][e] = 0.0f;
  }

  const int64_t step = (int64_t)gridDim.x * groups;
  int64_t row = (int64_t)blockIdx.x * groups + threadIdx.y;
  const int64_t iters = ceil_div(T_ - (int64_t)blockIdx.x * groups, step);
  auto fetch = [&](int64_t rw, int stage) {
    if constexpr (kAsync) {
      if (rw < T_) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
          const int c = threadIdx.x + j * tpr;
          if (c < nvec) {
#pragma unroll
            for (int a = 0; a < 4; ++a)
              if (src[a]) cp16(ring.slot(stage, a, j), src[a] + rw * nvec + c);
          }
        }
      }
      cp_commit();
    }
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(row + i * step, i);
  int stage = 0;
  for (int64_t it = 0; it < iters; ++it, row += step) {
    if constexpr (kAsync) {
      fetch(row + (kStages - 1) * step, (stage + kStages - 1) % kStages);
      cp_wait<kStages - 1>();
    }
    const bool live = row < T_;
    auto piece = [&](int a, int j, float (&f)[VEC]) {  // zeros where there is nothing to read
      const int c = threadIdx.x + j * tpr;
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[e] = 0.0f;
      if (src[a] && live && c < nvec) {
        if constexpr (kAsync) ring.slot(stage, a, j)->to(f);
        else src[a][row * nvec + c].to(f);
      }
    };
    float d[VPT][VEC], yv[VPT][VEC], rv[VPT][VEC];
    float s[3] = {0.0f, 0.0f, 0.0f};  // sum r^2, sum a r, sum y^2
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = threadIdx.x + j * tpr;
      float dn[VEC], wa[VEC], wb[VEC];
      piece(0, j, rv[j]);
      piece(1, j, yv[j]);
      piece(3, j, dn);
      if constexpr (!CACHE_W)
        if (c < nvec) channel_weights(c, wa, wb);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float a = c < nvec ? dn[e] * (CACHE_W ? wn[CACHE_W ? j : 0][e] : wb[e]) : 0.0f;
        s[0] = fmaf(rv[j][e], rv[j][e], s[0]);
        s[1] = fmaf(a, rv[j][e], s[1]);
        s[2] = fmaf(yv[j][e], yv[j][e], s[2]);
      }
    }
    row_sum(s, sums[flip ^= 1]);
    const float rho = 1.0f / sqrtf(fmaf(s[0], inv_h, eps));
    const float k = b.w_next ? rho * rho * rho * s[1] * inv_h : 0.0f;
    const float rho_y = b.w_post ? 1.0f / sqrtf(fmaf(s[2], inv_h, eps)) : 1.0f;
    const float g = b.token_gate && live ? __ldg(b.token_gate + row) : 1.0f;
    float q[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = threadIdx.x + j * tpr;
      const bool on = live && c < nvec;
      float dn[VEC], wa[VEC], wb[VEC], o[VEC];
      piece(2, j, d[j]);
      piece(3, j, dn);
      if constexpr (!CACHE_W)
        if (c < nvec) channel_weights(c, wa, wb);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if (on) {
          const float w_n = CACHE_W ? wn[CACHE_W ? j : 0][e] : wb[e], w_u = CACHE_W ? wu[CACHE_W ? j : 0][e] : wa[e];
          if (b.w_next) {
            d[j][e] = fmaf(rho, dn[e] * w_n, fmaf(-k, rv[j][e], d[j][e]));
            colN[j][e] = fmaf(dn[e], rv[j][e] * rho, colN[j][e]);
          }
          if (need_s) colS[j][e] = fmaf(g * d[j][e], yv[j][e] * rho_y, colS[j][e]);
          q[0] = fmaf(w_u * d[j][e], yv[j][e], q[0]);
        }
        o[e] = res_scale * d[j][e];
      }
      if (b.dx && on) static_cast<P*>(b.dx)[row * nvec + c] = P::of(o);
    }
    if (b.y) {
      if (b.w_post || b.dtoken_gate) row_sum(q, sums[flip ^= 1]);
      const float ky = b.w_post ? g * rho_y * rho_y * rho_y * q[0] * inv_h : 0.0f;
      if (b.dtoken_gate && live && threadIdx.x == 0) b.dtoken_gate[row] = rho_y * q[0];
      if (b.dy) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
          const int c = threadIdx.x + j * tpr;
          if (live && c < nvec) {
            float wa[VEC], wb[VEC], o[VEC];
            if constexpr (!CACHE_W) channel_weights(c, wa, wb);
#pragma unroll
            for (int e = 0; e < VEC; ++e)
              o[e] = fmaf(g * rho_y * (CACHE_W ? wu[CACHE_W ? j : 0][e] : wa[e]), d[j][e], -ky * yv[j][e]);
            static_cast<P*>(b.dy)[row * nvec + c] = P::of(o);
          }
        }
      }
    }
    if constexpr (kAsync) stage = (stage + 1) % kStages;
  }
  if (need_s || b.dw_next) {  // [2][gridDim.x * groups][H]
    const int64_t p = (int64_t)blockIdx.x * groups + threadIdx.y, np = (int64_t)gridDim.x * groups;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = threadIdx.x + j * tpr;
      if (c < nvec) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          if (need_s) part[p * H + c * VEC + e] = colS[j][e];
          if (b.dw_next) part[(np + p) * H + c * VEC + e] = colN[j][e];
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

// Threads per row, rows per CTA and pieces per thread for a row of `nvec` pieces.
struct Shape {
  int vpt, tpr, groups;
};
Shape shape_of(int nvec, int vpt) {
  Shape s;
  s.vpt = vpt;
  s.tpr = (int)(ceil_div(ceil_div(nvec, vpt), 32) * 32);
  s.groups = std::max(1, 128 / s.tpr);
  return s;
}

// Persistent grid of an instantiation. What fits on an SM depends on the threads of a row only;
// the last answer is kept (one word, so that concurrent callers see a whole one).
template <typename K>
cudaError_t grid_of(K kern, std::atomic<uint32_t>& last, const Shape& sh, size_t smem, int64_t T, int* grid) {
  uint32_t known = last.load(std::memory_order_relaxed);  // tpr << 8 | blocks per SM
  if (known >> 8 != (uint32_t)sh.tpr) {
    cudaError_t e = cudaSuccess;
    if (smem > 32 * 1024) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    int per_sm = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, sh.tpr * sh.groups, smem);
    if (e != cudaSuccess) return e;
    known = (uint32_t)sh.tpr << 8 | (uint32_t)std::max(1, per_sm);
    last.store(known, std::memory_order_relaxed);
  }
  *grid = (int)std::min<int64_t>(ceil_div(T, sh.groups),
                                 (int64_t)std::min(tc::num_sms(), kNormMaxSms) * (known & 255));
  return cudaSuccess;
}

template <typename T, int VEC, int VPT, bool CACHE_W, int MAXT, int STAGES>
cudaError_t fwd(const moe_norm_config_t& c, const NormIn& in, void* r, void* n, cudaStream_t s) {
  const Shape sh = shape_of(c.H / VEC, VPT);
  const size_t smem = (size_t)STAGES * 2 * VPT * sh.tpr * sh.groups * 16;
  auto kern = block_norm_kernel<T, VEC, VPT, CACHE_W, MAXT, STAGES>;
  int grid = 0;
  static std::atomic<uint32_t> last{0};
  cudaError_t e = grid_of(kern, last, sh, smem, c.T, &grid);
  if (e != cudaSuccess) return e;
  kern<<<grid, dim3(sh.tpr, sh.groups), smem, s>>>(in, r, n, c.T, c.H, c.eps, c.res_scale);
  return cudaGetLastError();
}

template <typename T, int VEC, int VPT, bool CACHE_W, int MAXT, int STAGES>
cudaError_t bwd(const moe_norm_config_t& c, const NormBwd& b, float* part, cudaStream_t s) {
  const Shape sh = shape_of(c.H / VEC, VPT);
  const size_t smem = (size_t)STAGES * 4 * VPT * sh.tpr * sh.groups * 16;
  auto kern = block_norm_bwd_kernel<T, VEC, VPT, CACHE_W, MAXT, STAGES>;
  int grid = 0;
  static std::atomic<uint32_t> last{0};
  cudaError_t e = grid_of(kern, last, sh, smem, c.T, &grid);
  if (e != cudaSuccess) return e;
  kern<<<grid, dim3(sh.tpr, sh.groups), smem, s>>>(b, part, c.T, c.H, c.eps, c.res_scale);
  e = cudaGetLastError();
  if (e != cudaSuccess || !(b.dgate || b.dw_post || b.dw_next)) return e;
  colsum_kernel<<<dim3((unsigned)ceil_div(c.H, 32), 2), dim3(32, 32), 0, s>>>(part, grid * sh.groups, c.H, b);
  return cudaGetLastError();
}

}  // namespace

// A row's pieces are spread over at most 1024 threads: bf16 rows have up to 2048 16-byte
// pieces (H = 16384), fp32 rows up to 4096, rows of odd width up to 16384 elements. STAGES:
// rows of the cp.async ring (FS with one piece per thread, BS with two).
// Rows of more than 1024 pieces and odd widths do without the ring (0).
#define NORM_DISPATCH(FN, FS, BS, ...)                                                         \
  if (c.act_dtype == MOE_DTYPE_BF16 && c.H % 8 == 0) {                                         \
    const int nvec = c.H / 8;                                                                  \
    if (nvec <= 256) return FN<__nv_bfloat16, 8, 1, true, 256, FS>(__VA_ARGS__);               \
    if (nvec <= 1024) return FN<__nv_bfloat16, 8, 2, true, 512, BS>(__VA_ARGS__);              \
    return FN<__nv_bfloat16, 8, 4, false, 512, 0>(__VA_ARGS__);                                \
  }                                                                                            \
  if (c.act_dtype == MOE_DTYPE_F32 && c.H % 4 == 0) {                                          \
    const int nvec = c.H / 4;                                                                  \
    if (nvec <= 512) return FN<float, 4, 1, true, 512, FS>(__VA_ARGS__);                       \
    if (nvec <= 1024) return FN<float, 4, 2, true, 512, BS>(__VA_ARGS__);                      \
    if (nvec <= 2048) return FN<float, 4, 4, false, 512, 0>(__VA_ARGS__);                      \
    return FN<float, 4, 4, false, 1024, 0>(__VA_ARGS__);                                       \
  }                                                                                            \
  if (c.act_dtype == MOE_DTYPE_BF16) {                                                         \
    if (c.H <= 2048) return FN<__nv_bfloat16, 1, 8, true, 256, 0>(__VA_ARGS__);                \
    return FN<__nv_bfloat16, 1, 16, false, 1024, 0>(__VA_ARGS__);                              \
  }                                                                                            \
  if (c.H <= 2048) return FN<float, 1, 8, true, 256, 0>(__VA_ARGS__);                          \
  return FN<float, 1, 16, false, 1024, 0>(__VA_ARGS__);

cudaError_t launch_block_norm(const moe_norm_config_t& c, const NormIn& in, void* r, void* n, cudaStream_t s) {
  if (c.T == 0) return cudaSuccess;
  NORM_DISPATCH(fwd, 4, 3, c, in, r, n, s)
}

cudaError_t launch_block_norm_backward(const moe_norm_config_t& c, const NormBwd& b, float* part, cudaStream_t s) {
  if (c.T == 0) {
    cudaError_t e = cudaSuccess;
    for (float* p : {b.dw_post, b.dw_next, b.dgate})
      if (p && e == cudaSuccess) e = cudaMemsetAsync(p, 0, (size_t)c.H * 4, s);
    return e;
  }
  NORM_DISPATCH(bwd, 3, 2, c, b, part, s)
}

// Two sets of column sums for every row group of the largest grid: at most 2048 / (threads of
// a row) row groups on each of 152 SMs, and never more than one per row.
size_t norm_part_bytes(const moe_norm_config_t& c) {
  const int vec = c.act_dtype == MOE_DTYPE_BF16 ? (c.H % 8 ? 1 : 8) : (c.H % 4 ? 1 : 4);
  const int nvec = c.H / vec;
  const int vpt = vec == 1 ? (c.H <= 2048 ? 8 : 16) : nvec <= (vec == 8 ? 256 : 512) ? 1 : nvec <= 1024 ? 2 : 4;
  const Shape sh = shape_of(nvec, vpt);
  const int64_t groups = std::min<int64_t>(align_up(c.T, sh.groups), (int64_t)kNormMaxSms * (2048 / sh.tpr));
  return (size_t)(2 * groups * c.H * 4);
}

}  // namespace moe
