// The global norm of many gradients and their scaling by min(1, max_norm / norm).
//
// Two passes, both bound by DRAM: the norm reads every element once, the scaling reads and
// writes them once (in place and below the limit it still reads them: the tiles are asked for before
// the factor is known; 604 M fp32 elements 669 us, the norm alone 343). The list of tensors travels in the kernel parameters, kPerLaunch tensors a
// launch, so a call needs no device table and captures into a graph. Each tensor is cut into
// tiles of kTile 16-byte pieces between 16-byte boundaries, so a view that starts at any
// element still moves as whole pieces but for its two ends. The grids are many blocks of few
// tiles: a persistent grid of what is resident keeps its blocks in step, with the reads and the
// writes of all of them on the same DRAM pages (604 M fp32 elements: scaling 1336 us with 4
// blocks per SM, 870 with 8, 767 with 64, 759 with a block per tile, of 712 for the bytes; the
// sum 395, 407, 354). The scaling walks the tiles in the opposite order: of a list the size of
// L2, what the norm read last is still there.
//
// Squares are added in fp32 over the 8 pieces of one thread's share of a tile and in fp64
// from there on (one fp64 add per 32 or 64 elements; every element in fp64 would be bound by
// the fp64 rate). A share whose fp32 sum leaves [2^-80, 2^120] - overflow, or squares that
// could have underflowed - is added again in fp64 from the elements, so neither 1e30 nor 1e-30
// is lost. Partial sums land in fixed slots and one block adds them in a fixed order.
#include <algorithm>

#include "step.cuh"

namespace moe {
namespace {

constexpr int kPerLaunch = 120;   // 24 bytes each: the parameters stay below 4 KB
constexpr int kShare = 8;         // pieces of a tile per thread
constexpr int kMaxBlocks = 152 * 64;  // of the sum: its blocks' sums are added by one block
// Threads of a block: 256, or 128 for lists that would give an SM fewer than four tiles of 256
// (48 views, 3 M elements: sum 8.4 -> 7.7, scaling 7.6 -> 5.9 us; 604 M: scaling 759 -> 788 us).
constexpr int kThreadsLarge = 256, kThreadsSmall = 128;

struct ClipTensor {
  const void* in;
  void* out;
  int64_t n2;  // elements * 2 + (1: bf16)
};
struct ClipList {
  ClipTensor t[kPerLaunch];
  int64_t tile0[kPerLaunch + 1];  // first tile (kShare pieces per thread) of each tensor
  int count;
};
static_assert(sizeof(ClipList) <= 4096 - 64, "kernel parameters");

// Workspace after the status head: a ticket, the scale, and the blocks' sums.
struct ClipState {
  uint32_t ticket;
  float scale;
};

struct View {  // one tensor as 16-byte pieces; elements [lo, hi) of the pieces belong to it
  const uint4* base;
  int64_t lo, hi, pieces;
  int per;  // elements per piece
};
__device__ __forceinline__ View view_of(const ClipTensor& t) {
  View v;
  const bool bf = t.n2 & 1;
  const uintptr_t a = reinterpret_cast<uintptr_t>(t.in);
  v.per = bf ? 8 : 4;
  v.base = reinterpret_cast<const uint4*>(a & ~uintptr_t(15));
  v.lo = (int64_t)(a & 15) / (bf ? 2 : 4);
  v.hi = v.lo + (t.n2 >> 1);
  v.pieces = (v.hi + v.per - 1) / v.per;
  return v;
}

__device__ __forceinline__ int tensor_of(const ClipList& l, int64_t tile) {
  int lo = 0, hi = l.count - 1;  // the last tensor whose first tile is <= tile (and that has tiles)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (l.tile0[mid] <= tile) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// One piece as up to 8 values; elements outside the tensor read as 0 and are not touched.
__device__ __forceinline__ uint4 load_piece(const View& v, int64_t i, bool bf) {
  const int64_t e0 = i * v.per;
  if (e0 >= v.lo && e0 + v.per <= v.hi) return __ldg(v.base + i);
  uint4 r = make_uint4(0, 0, 0, 0);
  uint32_t w[4] = {0, 0, 0, 0};
  for (int e = 0; e < v.per; ++e) {
    if (e0 + e < v.lo || e0 + e >= v.hi) continue;
    if (bf) w[e >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(v.base)[e0 + e] << (16 * (e & 1));
    else w[e] = reinterpret_cast<const uint32_t*>(v.base)[e0 + e];
  }
  r = make_uint4(w[0], w[1], w[2], w[3]);
  return r;
}

__device__ __forceinline__ void values(const uint4& p, bool bf, float (&f)[8]) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf ? __uint_as_float(w[i] << 16) : __uint_as_float(w[i]);
    f[2 * i + 1] = bf ? __uint_as_float(w[i] & 0xffff0000u) : 0.0f;
  }
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads)
    sum_squares_kernel(const __grid_constant__ ClipList list, double* sums, int slot0, int last, float max_norm,
                       float* norm, ClipState* state, DeviceStatus* st) {
  constexpr int kTile = kThreads * kShare;
  let_next_begin();
  if (slot0 > 0) after_previous();  // an earlier launch of the same call
  const int64_t tiles = list.tile0[list.count];
  double total = 0.0;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int k = tensor_of(list, tile);
    const View v = view_of(list.t[k]);
    const bool bf = list.t[k].n2 & 1;
    const int64_t p0 = (tile - list.tile0[k]) * kTile + threadIdx.x;
    uint4 p[kShare];
#pragma unroll
    for (int j = 0; j < kShare; ++j) {
      const int64_t i = p0 + j * kThreads;
      p[j] = i < v.pieces ? load_piece(v, i, bf) : make_uint4(0, 0, 0, 0);
    }
    float s = 0.0f;
    uint32_t any = 0;
#pragma unroll
    for (int j = 0; j < kShare; ++j) {
      float f[8];
      values(p[j], bf, f);
      any |= p[j].x | p[j].y | p[j].z | p[j].w;
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(f[e], f[e], s);
    }
    if (s >= 8.2718061e-25f && s <= 1.3292280e36f) {  // [2^-80, 2^120]
      total += (double)s;
    } else if (any) {
#pragma unroll 1
      for (int j = 0; j < kShare; ++j) {
        const int64_t i = p0 + j * kThreads;
        if (i >= v.pieces) break;
        float f[8];
        values(load_piece(v, i, bf), bf, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) total = fma((double)f[e], (double)f[e], total);
      }
    }
  }
  __shared__ double warp_sum[kThreads / 32];
  __shared__ bool finish;
  auto block_sum = [&](double x) {
#pragma unroll
    for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = x;
    __syncthreads();
    double r = 0.0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) r += warp_sum[i];
    return r;
  };
  total = block_sum(total);
  if (threadIdx.x == 0) {
    sums[slot0 + blockIdx.x] = total;
    __threadfence();
    finish = last && atomicInc(&state->ticket, gridDim.x - 1) == gridDim.x - 1;  // wraps to 0
  }
  __syncthreads();
  if (!finish) return;
  __threadfence();
  double all = 0.0;
  for (int i = threadIdx.x; i < slot0 + (int)gridDim.x; i += kThreads) all += __ldcg(sums + i);
  all = block_sum(all);
  if (threadIdx.x == 0) {
    const double nrm = sqrt(all);
    const bool fine = (float)nrm < INFINITY;  // false for NaN too, and for a norm beyond fp32
    if (!fine) set_status(st, MOE_ERR_DEVICE_BAD_INPUT, -1);
    *norm = (float)nrm;
    state->scale = fine && max_norm >= 0.0f && nrm > (double)max_norm ? (float)((double)max_norm / nrm) : 1.0f;
  }
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ ClipList list, const ClipState* state) {
  constexpr int kTile = kThreads * kShare;
  const int64_t tiles = list.tile0[list.count];
  float scale = 0.0f;  // read once the norm is there; the block's tile (its only one, but for huge lists) is on its way
  for (int64_t back = blockIdx.x; back < tiles; back += gridDim.x) {
    const int64_t tile = tiles - 1 - back;
    const int k = tensor_of(list, tile);
    const ClipTensor t = list.t[k];
    const View v = view_of(t);
    const bool bf = t.n2 & 1;
    uint8_t* out0 = static_cast<uint8_t*>(t.out) - v.lo * (bf ? 2 : 4);  // the place of element 0 of piece 0
    const bool same = (reinterpret_cast<uintptr_t>(out0) & 15) == 0;
    const int64_t p0 = (tile - list.tile0[k]) * kTile + threadIdx.x;
    uint4 p[kShare];
#pragma unroll
    for (int j = 0; j < kShare; ++j) {
      const int64_t i = p0 + j * kThreads;
      if (i < v.pieces) p[j] = load_piece(v, i, bf);
    }
    if (back == blockIdx.x) {
      after_previous();
      scale = *reinterpret_cast<const volatile float*>(&state->scale);
    }
    if (scale == 1.0f) {
      if (t.in == t.out) continue;
    }
#pragma unroll
    for (int j = 0; j < kShare; ++j) {
      const int64_t i = p0 + j * kThreads;
      if (i >= v.pieces) break;
      float f[8];
      values(p[j], bf, f);
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (bf) {
          const __nv_bfloat162 q = __floats2bfloat162_rn(f[2 * e] * scale, f[2 * e + 1] * scale);
          w[e] = *reinterpret_cast<const uint32_t*>(&q);
        } else {
          w[e] = __float_as_uint(f[2 * e] * scale);
        }
      }
      const int64_t e0 = i * v.per;
      if (same && e0 >= v.lo && e0 + v.per <= v.hi) {
        reinterpret_cast<uint4*>(out0)[i] = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        for (int e = 0; e < v.per; ++e) {
          if (e0 + e < v.lo || e0 + e >= v.hi) continue;
          if (bf) reinterpret_cast<uint16_t*>(out0)[e0 + e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
          else reinterpret_cast<uint32_t*>(out0)[e0 + e] = w[e];
        }
      }
    }
  }
}

// The pieces a gradient spans, from the 16-byte boundary before it.
int64_t pieces_of(const moe_grad_t& g) {
  const bool bf = g.dtype == MOE_DTYPE_BF16;
  return ceil_div((int64_t)((uintptr_t)g.grad & 15) / (bf ? 2 : 4) + g.n, bf ? 8 : 4);
}

// The next launch's tensors, from grads[*at] on (empty ones are left out).
void fill(ClipList* l, const moe_grad_t* grads, int32_t count, int tile, int32_t* at) {
  l->count = 0;
  l->tile0[0] = 0;
  for (; *at < count && (l->count < kPerLaunch || grads[*at].n == 0); ++*at) {
    const moe_grad_t& g = grads[*at];
    if (g.n == 0) continue;
    l->t[l->count] = {g.grad, g.out ? g.out : const_cast<void*>(g.grad), g.n * 2 + (g.dtype == MOE_DTYPE_BF16 ? 1 : 0)};
    l->tile0[l->count + 1] = l->tile0[l->count] + ceil_div(pieces_of(g), tile);
    ++l->count;
  }
}

template <int kThreads>
cudaError_t clip_launches(const moe_grad_t* grads, int32_t count, float max_norm, float* norm, char* w, DeviceStatus* st,
                          cudaStream_t s) {
  ClipState* state = reinterpret_cast<ClipState*>(w + kClipState);
  double* sums = reinterpret_cast<double*>(w + kWsHead);
  ClipList l;
  int slot = 0;
  int32_t at = 0;
  do {
    fill(&l, grads, count, kThreads * kShare, &at);
    const int grid = (int)std::min<int64_t>(std::max<int64_t>(l.tile0[l.count], 1), kMaxBlocks);
    cudaError_t e;
    if (slot == 0) {
      sum_squares_kernel<kThreads><<<grid, kThreads, 0, s>>>(l, sums, slot, at >= count, max_norm, norm, state, st);
      e = cudaGetLastError();
    } else {
      e = launch_after(sum_squares_kernel<kThreads>, grid, kThreads, s, l, sums, slot, at >= count, max_norm, norm, state, st);
    }
    if (e != cudaSuccess) return e;
    slot += grid;
  } while (at < count);
  if (max_norm < 0.0f) return cudaSuccess;
  at = 0;
  while (at < count) {
    fill(&l, grads, count, kThreads * kShare, &at);
    if (l.count == 0) break;
    const unsigned grid = (unsigned)std::min<int64_t>(l.tile0[l.count], INT32_MAX);
    const cudaError_t e = launch_after(scale_kernel<kThreads>, grid, kThreads, s, l, static_cast<const ClipState*>(state));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t grad_clip_ws_bytes(int32_t count) {
  return kWsHead + (size_t)std::max<int64_t>(1, ceil_div(count, kPerLaunch)) * kMaxBlocks * 8;
}

cudaError_t launch_grad_clip(const moe_grad_t* grads, int32_t count, float max_norm, float* norm, void* ws,
                             DeviceStatus* st, cudaStream_t s) {
  int64_t pieces = 0;
  for (int32_t i = 0; i < count; ++i) pieces += grads[i].n ? pieces_of(grads[i]) : 0;
  return pieces < (int64_t)4 * 152 * kThreadsLarge * kShare
             ? clip_launches<kThreadsSmall>(grads, count, max_norm, norm, static_cast<char*>(ws), st, s)
             : clip_launches<kThreadsLarge>(grads, count, max_norm, norm, static_cast<char*>(ws), st, s);
}

}  // namespace moe
