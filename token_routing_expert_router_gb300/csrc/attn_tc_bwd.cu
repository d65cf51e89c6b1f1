// The backward of attention on the tensor cores (bf16, D <= 128): dk and dv of 128 keys of a head by one
// kernel, dq of 128 (query, head) rows by another. Both are the same loop: an outer tile stays in shared
// memory (X1, X2 = K, V or Q, dO), inner tiles of 128 rows go by (Y1, Y2 = Q, dO or K, V), and
//   S = X1 Y1^T,  dP = X2 Y2^T   (tensor memory)
//   P = exp2(c S - lse2),  dS = P (dP - delta)   (bf16, over the columns of S and dP)
//   [dV += P Y2]   dK or dQ += dS Y1
// with rows of the outer tile as lanes of tensor memory, so that P and dS are first operands where they
// are. Sums over the query heads of a group and over all queries stay in one accumulator: no atomics,
// and the bits never change. In return S and dP are formed twice: seven products instead of five.
//
// Warp 0 loads by TMA, warp 1 issues the products, warp 2 brings lse and delta of the inner rows (dk, dv),
// warpgroups 1 and 2 form P and dS, each of one half of the columns. The products of one inner tile
// take the tensor cores twice as long as P and dS take the warps, and they interleave without a second
// set of accumulators (there is no room for one: S, dP, dK and dV fill tensor memory): while dS(t) is
// formed, dV(t) and S(t+1) run, while P(t+1) is formed, dK(t) and dP(t+1).
#include "attn_tc.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int R = 128;  // rows of every tile

template <int DP>
struct Bwd {
  static constexpr int kSlabs = DP / 64;
  static constexpr int kTile = R * DP * 2;
  static constexpr int kStats = 2 * R * 2 * 4;  // two stages of -lse2 and -delta
  static constexpr size_t kUsed = 1024 + 6 * kTile + kStats + 256;
  // a CTA takes all of tensor memory: no second one on its SM
  static constexpr size_t kBytes = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
};

struct BwdParams {
  AttnArgs a;
  int pack;  // query heads in a tile
  float c;   // scale log2(e)
};

// (a, b) -> (a, b) * f + (c, d)
__device__ __forceinline__ void scale_add2(float& a, float& b, float f, float c, float d) {
  asm("{\n\t.reg .b64 x, s, t;\n\t"
      "mov.b64 x, {%0, %1};\n\t"
      "mov.b64 s, {%2, %2};\n\t"
      "mov.b64 t, {%3, %4};\n\t"
      "fma.rn.f32x2 x, x, s, t;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(f), "f"(c), "f"(d));
}
// (a, b) *= (x, y)
__device__ __forceinline__ void mul2(float& a, float& b, float x, float y) {
  asm("{\n\t.reg .b64 p, q;\n\t"
      "mov.b64 p, {%0, %1};\n\t"
      "mov.b64 q, {%2, %3};\n\t"
      "mul.rn.f32x2 p, p, q;\n\t"
      "mov.b64 {%0, %1}, p;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y));
}

template <int DP, bool DKV>
__global__ void __launch_bounds__(kThreads, 1)
    attn_backward_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                         const BwdParams p) {
  using F = Bwd<DP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sX = smem;                   // X1, X2
  uint8_t* sY1 = smem + 2 * F::kTile;   // two stages each
  uint8_t* sY2 = smem + 4 * F::kTile;
  float* sStat = reinterpret_cast<float*>(smem + 6 * F::kTile);  // [stage][-lse2, -delta][R]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + 6 * F::kTile + F::kStats);
  uint64_t* x_full = bars;
  uint64_t* y1_full = bars + 1;
  uint64_t* y2_full = bars + 3;
  uint64_t* y1_empty = bars + 5;
  uint64_t* y2_empty = bars + 7;
  uint64_t* stat_full = bars + 9;
  uint64_t* stat_empty = bars + 11;
  uint64_t* s_full = bars + 13;
  uint64_t* dp_full = bars + 14;
  uint64_t* p_ready = bars + 15;
  uint64_t* ds_ready = bars + 16;
  uint64_t* acc_full = bars + 17;
  uint64_t* drain = bars + 18;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 19);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const AttnArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = R / p.pack;  // queries of a tile
  const int hk = DKV ? (int)blockIdx.y : (int)blockIdx.y * p.pack / a.group;
  const int h0 = DKV ? hk * a.group : (int)blockIdx.y * p.pack;  // first query head
  const Tile t = find_tile<kThreads, DKV>(a, blockIdx.x, DKV ? R : per, true, blockIdx.x == 0 && blockIdx.y == 0);
  if (t.b < 0) return;
  const Seq s = load_seq(a, t.b, true, false);
  // the outer tile's first row (key, or query: the longest first), and how many inner tiles it meets
  const int o0 = DKV ? t.index * R : (t.count - 1 - t.index) * per;
  int first = 0, tiles;  // DKV: of every pack of heads
  if constexpr (DKV) {
    first = a.causal ? max(0, o0 - (s.m - s.n)) / per : 0;  // the first queries that see key o0
    tiles = max(0, (s.n + per - 1) / per - first);
  } else {
    tiles = (max(0, visible(a, s, min(o0 + per, s.n) - 1)) + R - 1) / R;
  }
  const int steps = DKV ? tiles * (a.group / p.pack) : tiles;
  // inner tile i: DKV: first query and head; else first key
  auto inner_row = [&](int i) { return DKV ? (first + i % tiles) * per : i * R; };
  auto inner_head = [&](int i) { return h0 + i / tiles * p.pack; };
  // rows of it that are the sequence's
  auto inner_live = [&](int i) { return DKV ? min(R, (s.n - inner_row(i)) * p.pack) : min(R, s.m - inner_row(i)); };

  if (threadIdx.x == 0) {
    mbar_init(x_full, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&y1_full[b], 1);
      mbar_init(&y2_full[b], 1);
      mbar_init(&y1_empty[b], 1);
      mbar_init(&y2_empty[b], 1);
      mbar_init(&stat_full[b], 32);
      mbar_init(&stat_empty[b], 8);
    }
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    mbar_init(p_ready, 8);
    mbar_init(ds_ready, 8);
    mbar_init(acc_full, 1);
    mbar_init(drain, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  const uint32_t tS = tmem, tP = tmem + 128, tA1 = tmem + 256, tA2 = tmem + 256 + DP;  // S, dP, dK or dQ, dV

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 0 && lane == 0 && steps > 0) {
      // ===================== loads
      auto load = [&](const CUtensorMap* m, uint8_t* dst, uint64_t* bar, int head, int row) {
#pragma unroll
        for (int d = 0; d < F::kSlabs; ++d) tma_load_3d(m, dst + d * 16384, bar, 64 * d, head, row);
      };
      mbar_arrive_expect_tx(x_full, 2 * F::kTile);
      load(DKV ? &tmK : &tmQ, sX, x_full, DKV ? hk : h0, DKV ? s.k0 + o0 : s.q0 + o0);
      load(DKV ? &tmV : &tmO, sX + F::kTile, x_full, DKV ? hk : h0, DKV ? s.k0 + o0 : s.q0 + o0);
      bool ok = true;
      int n1 = 0, n2 = 0;
      for (int i = 0; i < steps && ok; ++i) {
        const int b = i & 1, head = DKV ? inner_head(i) : hk, row = (DKV ? s.q0 : s.k0) + inner_row(i);
        const uint32_t parity = (i >> 1 & 1) ^ 1;
        if (!(ok = mbar_wait(&y1_empty[b], parity, abort, kTimeoutNs, a.status))) break;
        mbar_arrive_expect_tx(&y1_full[b], F::kTile);
        load(DKV ? &tmQ : &tmK, sY1 + b * F::kTile, &y1_full[b], head, row);
        ++n1;
        if (!(ok = mbar_wait(&y2_empty[b], parity, abort, kTimeoutNs, a.status))) break;
        mbar_arrive_expect_tx(&y2_full[b], F::kTile);
        load(DKV ? &tmO : &tmV, sY2 + b * F::kTile, &y2_full[b], head, row);
        ++n2;
      }
      // leave no copy in flight
      mbar_wait_drain(x_full, 0, kTimeoutNs, a.status);
      for (int i = max(0, n1 - 2); i < n1; ++i) mbar_wait_drain(&y1_full[i & 1], i >> 1 & 1, kTimeoutNs, a.status);
      for (int i = max(0, n2 - 2); i < n2; ++i) mbar_wait_drain(&y2_full[i & 1], i >> 1 & 1, kTimeoutNs, a.status);
    } else if (warp == 1 && steps > 0) {
      // ===================== products
      const uint32_t idesc_s = idesc_make(1, R, R);
      const uint32_t idesc_a = idesc_make(1, R, DP) | (1u << 16);  // the inner tile is read MN-major
      auto all = [&](bool ok) { return (bool)__all_sync(0xffffffffu, ok); };
      const bool one = lane == 0;
      // S or dP = X Y^T
      auto scores = [&](uint32_t d, const uint8_t* x, const uint8_t* y, uint64_t* bar) {
        const uint32_t xa = uniform(k_desc(smem_addr(x))), ya = uniform(k_desc(smem_addr(y)));
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          const uint32_t off = (k / 4) * (16384 / 16) + (k % 4) * 2;
          mma_ss(d, xa + off, ya + off, idesc_s, k > 0, one);
        }
        commit(bar, one);
      };
      // acc += W Y, W in tensor memory: the columns' halves each at the start of their half of the scores
      auto products = [&](uint32_t d, uint32_t w, const uint8_t* y, bool begin) {
        const uint32_t ya = uniform(mn_desc(smem_addr(y)));
#pragma unroll
        for (int k = 0; k < R / 16; ++k)
          mma_ts(d, w + (k / 4) * 64 + (k % 4) * 8, ya + (2048 / 16) * k, idesc_a, !begin || k > 0, one);
      };
      // inner tile i's Y1 (Y2) has come; rows that are not the sequence's are zeroed
      auto arrived = [&](uint64_t* bar, uint8_t* y, int i) {
        if (!all(mbar_wait(&bar[i & 1], i >> 1 & 1, abort, kTimeoutNs, a.status))) return false;
        const int live = inner_live(i);
        if (live < R) clear_rows(y + (i & 1) * F::kTile, F::kSlabs, R, live, lane);
        tc_fence_after();
        return true;
      };
      bool ok = all(mbar_wait(x_full, 0, abort, kTimeoutNs, a.status)) && arrived(y1_full, sY1, 0);
      if (ok) scores(tS, sX, sY1, s_full);
      ok = ok && arrived(y2_full, sY2, 0);
      if (ok) scores(tP, sX + F::kTile, sY2, dp_full);
      for (int i = 0; i < steps && ok; ++i) {
        const int b = i & 1;
        if (!(ok = all(mbar_wait(p_ready, b, abort, kTimeoutNs, a.status)))) break;
        tc_fence_after();
        if constexpr (DKV) products(tA2, tS, sY2 + b * F::kTile, i == 0);
        commit(&y2_empty[b], one);
        if (i + 1 < steps) {
          if (!(ok = arrived(y1_full, sY1, i + 1))) break;
          scores(tS, sX, sY1 + (b ^ 1) * F::kTile, s_full);
        }
        if (!(ok = all(mbar_wait(ds_ready, b, abort, kTimeoutNs, a.status)))) break;
        tc_fence_after();
        products(tA1, tP, sY1 + b * F::kTile, i == 0);
        commit(&y1_empty[b], one);
        if (i + 1 < steps) {
          if (!(ok = arrived(y2_full, sY2, i + 1))) break;
          scores(tP, sX + F::kTile, sY2 + (b ^ 1) * F::kTile, dp_full);
        }
      }
      __syncwarp();
      if (lane == 0) {
        if (ok) mma_commit(acc_full);
        mma_commit(drain);
        mbar_wait_drain(drain, 0, kTimeoutNs, a.status);
      }
      __syncwarp();
    } else if (DKV && warp == 2) {
      // ===================== -lse2 and -delta of the inner rows; a row that is not there, or sees no key,
      // gets p = exp2(s - inf) = 0
      for (int i = 0; i < steps; ++i) {
        const int b = i & 1, row0 = inner_row(i), head = inner_head(i), live = inner_live(i);
        float v[8];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = 32 * q + lane;
          v[q] = -INFINITY, v[4 + q] = 0.0f;
          if (r < live) {
            const int64_t at = (int64_t)(head + r % p.pack) * a.Tq + s.q0 + row0 + r / p.pack;
            const float l = __ldg(a.lse + at);
            if (l != -INFINITY) v[q] = -l * kLog2e;
            v[4 + q] = -__ldg(a.delta + at);
          }
        }
        if (!__all_sync(0xffffffffu, mbar_wait(&stat_empty[b], (i >> 1 & 1) ^ 1, abort, kTimeoutNs, a.status))) break;
#pragma unroll
        for (int q = 0; q < 8; ++q) sStat[b * 2 * R + q / 4 * R + 32 * (q % 4) + lane] = v[q];
        mbar_arrive(&stat_full[b]);
      }
    }
  } else {
    // ===================== P and dS: a lane of tensor memory a thread, one half of the columns
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int half = warp / 4 - 1, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t my_s = tS + lanes + 64 * half, my_p = tP + lanes + 64 * half;
    // DKV: the row's key is o0 + row; else its query and head
    const int i_q = DKV ? 0 : o0 + row / p.pack, h = DKV ? 0 : h0 + row % p.pack;
    float neg_lse = -INFINITY, neg_delta = 0.0f;
    int seen = 0;
    if (!DKV && i_q < s.n) {
      const int64_t at = (int64_t)h * a.Tq + s.q0 + i_q;
      const float l = __ldg(a.lse + at);
      if (l != -INFINITY) neg_lse = -l * kLog2e;
      neg_delta = -__ldg(a.delta + at);
      seen = visible(a, s, i_q);
    }
    bool ok = true;
    for (int i = 0; i < steps; ++i) {
      const int b = i & 1, row0 = inner_row(i);
      const float4* stat = reinterpret_cast<const float4*>(sStat + b * 2 * R + 64 * half);
      if (DKV && !(ok = __all_sync(0xffffffffu, mbar_wait(&stat_full[b], i >> 1 & 1, abort, kTimeoutNs, a.status)))) break;
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(s_full, b, abort, kTimeoutNs, a.status)))) break;
      tc_fence_after();
      uint32_t r[2][32];
      tmem_ld32(my_s, r[0]);
      tmem_ld32(my_s + 32, r[1]);
      tmem_ld_wait();
      if constexpr (!DKV) {  // S may be formed again
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready);
      }
      float pr[64];
#pragma unroll
      for (int l = 0; l < 64; l += 4) {
        float4 n;
        if constexpr (DKV) n = stat[l / 4];
        else n = make_float4(neg_lse, neg_lse, neg_lse, neg_lse);
#pragma unroll
        for (int e = 0; e < 4; ++e) pr[l + e] = __uint_as_float(r[(l + e) / 32][(l + e) % 32]);
        scale_add2(pr[l], pr[l + 1], p.c, n.x, n.y);
        scale_add2(pr[l + 2], pr[l + 3], p.c, n.z, n.w);
#pragma unroll
        for (int e = 0; e < 4; ++e) pr[l + e] = ex2(pr[l + e]);
      }
      if constexpr (DKV) {
        // query r / pack of the tile sees key o0 + row from row `from` on
        if (a.causal && o0 + R - 1 - (s.m - s.n) > row0) {
          const int from = (o0 + row - (s.m - s.n) - row0) * p.pack - 64 * half;
#pragma unroll
          for (int l = 0; l < 64; ++l)
            if (l < from) pr[l] = 0.0f;
        }
        uint32_t w[32];
#pragma unroll
        for (int l = 0; l < 32; ++l) w[l] = pack2(pr[2 * l], pr[2 * l + 1]);
        tmem_st32(my_s, w);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready);
      } else if ((i + 1) * R > visible(a, s, o0)) {
        const int end = seen - row0 - 64 * half;
#pragma unroll
        for (int l = 0; l < 64; ++l)
          if (l >= end) pr[l] = 0.0f;
      }
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(dp_full, b, abort, kTimeoutNs, a.status)))) break;
      tc_fence_after();
      tmem_ld32(my_p, r[0]);
      tmem_ld32(my_p + 32, r[1]);
      tmem_ld_wait();
      uint32_t w[32];
#pragma unroll
      for (int l = 0; l < 64; l += 4) {
        float4 n;
        if constexpr (DKV) n = stat[R / 4 + l / 4];
        else n = make_float4(neg_delta, neg_delta, neg_delta, neg_delta);
        float d[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] = __uint_as_float(r[(l + e) / 32][(l + e) % 32]);
        add2(d[0], d[1], n.x, n.y);
        add2(d[2], d[3], n.z, n.w);
        mul2(d[0], d[1], pr[l], pr[l + 1]);
        mul2(d[2], d[3], pr[l + 2], pr[l + 3]);
        w[l / 2] = pack2(d[0], d[1]);
        w[l / 2 + 1] = pack2(d[2], d[3]);
      }
      tmem_st32(my_p, w);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(ds_ready);
        if constexpr (DKV) mbar_arrive(&stat_empty[b]);
      }
    }
    // ===================== the accumulators, a half of the channels each
    if (steps > 0) ok = __all_sync(0xffffffffu, ok && mbar_wait(acc_full, 0, abort, kTimeoutNs, a.status));
    tc_fence_after();
    const bool live = ok && (DKV ? o0 + row < s.m : i_q < s.n);
    constexpr int kCols = DP / 2;
    auto store = [&](uint32_t from, void* base, int64_t at, float f) {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(base) + at + kCols * half;
#pragma unroll
      for (int q = 0; q < kCols / 32; ++q) {
        uint32_t o[32] = {};
        if (steps > 0) {
          tmem_ld32(from + lanes + kCols * half + 32 * q, o);
          tmem_ld_wait();
        }
#pragma unroll
        for (int l = 0; l < 32; l += 8) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(o[l + e]) * f;
          if (live && kCols * half + 32 * q + l < a.D)
            *reinterpret_cast<uint4*>(dst + 32 * q + l) =
                make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
        }
      }
    };
    if constexpr (DKV) {
      store(tA1, a.dk, (int64_t)(s.k0 + o0 + row) * a.ld_k + (int64_t)hk * a.D, a.scale);
      store(tA2, a.dv, (int64_t)(s.k0 + o0 + row) * a.ld_v + (int64_t)hk * a.D, 1.0f);
    } else {
      store(tA1, a.dq, (int64_t)(s.q0 + i_q) * a.ld_q + (int64_t)h * a.D, a.scale);
    }
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int DP, bool DKV>
cudaError_t launch(dim3 grid, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& o,
                   const BwdParams& p, cudaStream_t s) {
  static const cudaError_t e = cudaFuncSetAttribute(attn_backward_kernel<DP, DKV>,
                                                    cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Bwd<DP>::kBytes);
  if (e != cudaSuccess) return e;
  attn_backward_kernel<DP, DKV><<<grid, kThreads, Bwd<DP>::kBytes, s>>>(q, k, v, o, p);
  return cudaGetLastError();
}

template <int DP>
cudaError_t backward(const AttnArgs& a, cudaStream_t s) {
  BwdParams p{a, heads_packed(a.group), a.scale * kLog2e};
  CUtensorMap q, k, v, o;
  if (a.Tq > 0 && (!head_map(&q, a.q, a.Tq, a.Hq, a.D, a.ld_q, p.pack, R / p.pack) ||
                   !head_map(&o, a.d_o, a.Tq, a.Hq, a.D, a.ld_o, p.pack, R / p.pack)))
    return cudaErrorInvalidValue;
  if (a.Tk > 0 && (!head_map(&k, a.k, a.Tk, a.Hkv, a.D, a.ld_k, 1, R) || !head_map(&v, a.v, a.Tk, a.Hkv, a.D, a.ld_v, 1, R)))
    return cudaErrorInvalidValue;
  // without queries or keys nothing of them is loaded
  if (a.Tq == 0) q = o = k;
  if (a.Tk == 0) k = v = q;
  cudaError_t e = cudaSuccess;
  if (a.Tq > 0) e = launch<DP, false>(dim3((unsigned)(a.Tq / (R / p.pack) + a.B), a.Hq / p.pack), q, k, v, o, p, s);
  if (e != cudaSuccess || a.Tk == 0) return e;
  return launch<DP, true>(dim3((unsigned)(a.Tk / R + a.B), a.Hkv), q, k, v, o, p, s);
}

}  // namespace

cudaError_t launch_tc_backward(const AttnArgs& a, cudaStream_t s) {
  const cudaError_t e = launch_delta(a, true, s);
  if (e != cudaSuccess) return e;
  return a.D <= 64 ? backward<64>(a, s) : backward<128>(a, s);
}

}  // namespace attn
}  // namespace moe
