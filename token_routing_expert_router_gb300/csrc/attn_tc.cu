// Attention on the tensor cores (bf16, D <= 128), one pass over the keys.
//
// A CTA has two tiles of 128 rows of Q against one key head, and goes over its keys in tiles of 128:
//   S = Q K^T (tensor memory) -> P = exp2(c (S - m)), bf16, over S's columns -> O += P V (tensor memory)
// Rows of a tile are (query, head) pairs, `pack` query heads of the group side by side: a key tile is
// loaded once for 256 of them, and few queries of many heads still fill a tile.
// Warp 0 loads by TMA (K and V tiles through one ring), warp 1 issues the products, and each of the two
// warpgroups 1 and 2 is one tile's softmax, a thread a row: no exchange between threads. While one
// tile's softmax runs, the tensor cores work on the other tile's products; S is free for the next scores
// as soon as P V has been issued behind them, since one thread's products run in their order.
//
// The running maximum is only followed when it grows by more than 2^8 in the exponentials (then O is
// read, scaled and written back, by the rows' own threads); until then the old one is as good a
// reference, since all sums are fp32 and P's rounding is relative. The keys are taken from the last to
// the first, so that the tile with the mask comes first. Key rows behind the sequence's end belong to
// somebody else: their scores are replaced, and their V rows are zeroed in shared memory.
#include "attn_plan.cuh"
#include "attn_tc.cuh"

namespace moe {
namespace attn {
namespace {

struct FwdParams {
  AttnArgs a;
  int pack;     // query heads in a tile
  float c;      // scale log2(e)
  int tiles, heads, chunk;  // the grid: tiles (at most), packs of heads, packs that share the L2
  const TilePlan* plan;     // NULL: tiles in their order
};

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attn_forward_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const FwdParams p) {
  using F = Fwd<DP>;
  constexpr int kUnits = F::kUnits;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + 2 * F::kTile;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sKV + kUnits * F::kTile);
  uint64_t* full = bars;
  uint64_t* empty = bars + kUnits;
  uint64_t* q_full = bars + 2 * kUnits;
  uint64_t* s_full = q_full + 1;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* drain = o_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert((2 * 8 + 8) * 8 + 8 <= 256);

  const AttnArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Place at = place_of(blockIdx.x, p.tiles, p.heads, p.chunk);
  const int h0 = at.head * p.pack, hk = h0 / a.group;  // first query head, key head
  const int per = 128 / p.pack;                        // queries of a tile
  Seq s;
  int i0;  // the first query
  if (p.plan) {
    after_previous();
    if (at.rank >= p.plan->count) return;
    const TileEntry e = p.plan->tile[at.rank];
    s = Seq{e.q0, e.n, e.k0, e.m};
    i0 = e.start;
  } else {
    __shared__ int sFind[kThreads / 32 + 3];
    const Tile t = find_tile<kThreads, false>(a, at.rank, 2 * per, false, blockIdx.x == 0, sFind);
    if (t.b < 0) return;
    s = load_seq(a, t.b, false, false);
    i0 = (t.count - 1 - t.index) * 2 * per;  // the longest first
  }
  // key tiles of the two row tiles
  auto key_tiles = [&](int m) {
    const int first = i0 + m * per, last = min(first + per, s.n) - 1;
    return last < first ? 0 : (max(0, visible(a, s, last)) + BK - 1) / BK;
  };
  const int n0 = key_tiles(0), n1 = key_tiles(1), steps = max(n0, n1);
  auto tiles_of = [&](int m) { return m ? n1 : n0; };

  if (threadIdx.x == 0) {
    for (int u = 0; u < kUnits; ++u) {
      mbar_init(&full[u], 1);
      mbar_init(&empty[u], 1);
    }
    mbar_init(q_full, 1);
    for (int m = 0; m < 2; ++m) {
      mbar_init(&s_full[m], 1);
      mbar_init(&p_full[m], 4);
      mbar_init(&o_full[m], 1);
    }
    mbar_init(drain, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  const uint32_t tS = tmem, tO = tmem + 256;  // S and P of tile m at 128 m, O at DP m

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 0 && lane == 0 && steps > 0) {
      // ===================== loads: Q; K of the last tile; then K of the next and V of this one, in turn
      mbar_arrive_expect_tx(q_full, 2 * F::kTile);
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int d = 0; d < F::kSlabs; ++d)
          tma_load_3d(&tmQ, sQ + m * F::kTile + d * 16384, q_full, 64 * d, h0, s.q0 + i0 + m * per);
      int unit = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      auto load = [&](const CUtensorMap* map, int tile) {
        if (!ok || !(ok = mbar_wait(&empty[unit], phase ^ 1, abort, kTimeoutNs, a.status))) return;
        mbar_arrive_expect_tx(&full[unit], F::kTile);
#pragma unroll
        for (int d = 0; d < F::kSlabs; ++d)
          tma_load_3d(map, sKV + unit * F::kTile + d * 16384, &full[unit], 64 * d, hk, s.k0 + tile * BK);
        ++issued;
        if (++unit == kUnits) unit = 0, phase ^= 1;
      };
      load(&tmK, steps - 1);
      for (int j = steps - 1; j >= 0 && ok; --j) {
        if (j > 0) load(&tmK, j - 1);
        load(&tmV, j);
      }
      // leave no copy in flight
      mbar_wait_drain(q_full, 0, kTimeoutNs, a.status);
      for (int i = 0; i < min(issued, kUnits); ++i) {
        const int u = (unit - 1 - i + 2 * kUnits) % kUnits;
        mbar_wait_drain(&full[u], unit - 1 - i < 0 ? phase ^ 1 : phase, kTimeoutNs, a.status);
      }
    } else if (warp == 1 && steps > 0) {
      // ===================== products
      const uint32_t idesc_s = idesc_make(1, 128, BK);
      const uint32_t idesc_o = idesc_make(1, 128, DP) | (1u << 16);  // V is read MN-major
      int unit = 0;
      uint32_t phase = 0;
      auto wait_unit = [&] {
        const bool ok = mbar_wait(&full[unit], phase, abort, kTimeoutNs, a.status);
        return __all_sync(0xffffffffu, ok);
      };
      auto next = [&](int& u) {
        u = unit;
        if (++unit == kUnits) unit = 0, phase ^= 1;
      };
      const bool one = lane == 0;
      auto scores = [&](int m, int u) {  // S_m = Q_m K^T
        const uint32_t qa = uniform(k_desc(smem_addr(sQ + m * F::kTile))), ka = uniform(k_desc(smem_addr(sKV + u * F::kTile)));
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          const uint32_t off = (k / 4) * (16384 / 16) + (k % 4) * 2;
          mma_ss(tS + 128 * m, qa + off, ka + off, idesc_s, k > 0, one);
        }
        commit(&s_full[m], one);
      };
      bool ok = mbar_wait(q_full, 0, abort, kTimeoutNs, a.status);
      ok = __all_sync(0xffffffffu, ok) && wait_unit();
      if (ok) {
        tc_fence_after();
        int uk, uv;
        next(uk);
        for (int m = 0; m < 2; ++m)
          if (tiles_of(m) == steps) scores(m, uk);
        commit(&empty[uk], one);
        for (int j = steps - 1; j >= 0; --j) {
          if (j > 0) {
            if (!(ok = wait_unit())) break;
            next(uk);
          }
          if (!(ok = wait_unit())) break;
          next(uv);
          if ((j + 1) * BK > s.m) clear_rows(sKV + uv * F::kTile, F::kSlabs, BK, s.m - j * BK, lane);
          tc_fence_after();
          for (int m = 0; m < 2 && ok; ++m) {
            const int n = tiles_of(m);
            if (j < n) {
              ok = mbar_wait(&p_full[m], (n - 1 - j) & 1, abort, kTimeoutNs, a.status);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              tc_fence_after();
              const uint32_t va = uniform(mn_desc(smem_addr(sKV + uv * F::kTile)));
#pragma unroll
              for (int k = 0; k < BK / 16; ++k)  // O_m += P_m V
                mma_ts(tO + DP * m, tS + 128 * m + 8 * k, va + (2048 / 16) * k, idesc_o, j < n - 1 || k > 0, one);
              if (j == 0) commit(&o_full[m], one);
            }
            if (j > 0 && j - 1 < n) scores(m, uk);
          }
          if (!ok) break;
          commit(&empty[uv], one);
          if (j > 0) commit(&empty[uk], one);
        }
      }
      __syncwarp();
      if (lane == 0) {
        mma_commit(drain);
        mbar_wait_drain(drain, 0, kTimeoutNs, a.status);
      }
      __syncwarp();
    }
  } else {
    // ===================== softmax of tile m, a thread a row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int m = warp / 4 - 1, quarter = warp & 3;
    const int row = quarter * 32 + lane, i = i0 + m * per + row / p.pack, h = h0 + row % p.pack;
    const int n = tiles_of(m);
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t my_s = tS + 128 * m + lanes, my_o = tO + DP * m + lanes;
    const int seen = visible(a, s, i);                               // of this row
    const int least = visible(a, s, i0 + m * per);                   // of the tile's first row
    Running w;
    bool ok = true;
    for (int j = n - 1; j >= 0; --j) {
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&s_full[m], (n - 1 - j) & 1, abort, kTimeoutNs, a.status)))) break;
      tc_fence_after();
      softmax_step<DP>(my_s, my_o, p.c, (j + 1) * BK > least ? seen - j * BK : BK, j < n - 1, w);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[m]);
    }
    // ===================== O / sum and the log sum
    const float sum = w.sum0 + w.sum1, top = w.top;
    if (n > 0) ok = __all_sync(0xffffffffu, ok && mbar_wait(&o_full[m], 0, abort, kTimeoutNs, a.status));
    tc_fence_after();
    const bool live = ok && i < s.n;
    const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.o) + (int64_t)(s.q0 + i) * a.ld_o + (int64_t)h * a.D;
#pragma unroll
    for (int q = 0; q < DP / 32; ++q) {
      uint32_t o[32];
      if (n > 0) {
        tmem_ld32(my_o + 32 * q, o);
        tmem_ld_wait();
      }
#pragma unroll
      for (int l = 0; l < 32; l += 8) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = sum == 0.0f ? 0.0f : __uint_as_float(o[l + e]) * f;  // no key: a row of zeros
        if (live && 32 * q + l < a.D)
          *reinterpret_cast<uint4*>(dst + 32 * q + l) =
              make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
      }
    }
    if (live)
      a.lse[(int64_t)h * a.Tq + s.q0 + i] = sum == 0.0f ? -INFINITY : (top * p.c + log2f(sum)) * kLn2;
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int DP>
cudaError_t forward(const AttnArgs& a, TilePlan* plan, cudaStream_t s) {
  FwdParams p{a, heads_packed(a.group), a.scale * kLog2e};
  p.tiles = (int)forward_tiles(a);
  p.heads = a.Hq / p.pack;
  p.chunk = head_chunk((int64_t)a.Tk * a.D * 4, a.Hkv) * (a.group / p.pack);
  if ((int64_t)p.tiles * p.heads >= (1ll << 31)) return cudaErrorInvalidConfiguration;
  CUtensorMap q, k, v;
  if (!head_map(&q, a.q, a.Tq, a.Hq, a.D, a.ld_q, p.pack, 128 / p.pack)) return cudaErrorInvalidValue;
  if (a.Tk > 0) {
    if (!head_map(&k, a.k, a.Tk, a.Hkv, a.D, a.ld_k, 1, BK) || !head_map(&v, a.v, a.Tk, a.Hkv, a.D, a.ld_v, 1, BK))
      return cudaErrorInvalidValue;
  } else {
    k = v = q;  // no key is loaded
  }
  static const cudaError_t e =
      cudaFuncSetAttribute(attn_forward_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Fwd<DP>::kBytes);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)p.tiles * p.heads;
  // one sequence's tiles are in the order of their work as they are
  if (a.B > 1 && a.B <= kPlanMaxB) {
    p.plan = plan;
    const cudaError_t l = launch_plan(a, PlanJob{0, 256 / p.pack, 0, 0, p.heads, 0, p.tiles, plan}, s);
    if (l != cudaSuccess) return l;
    return launch_after_smem(attn_forward_kernel<DP>, grid, kThreads, Fwd<DP>::kBytes, s, q, k, v, p);
  }
  attn_forward_kernel<DP><<<grid, kThreads, Fwd<DP>::kBytes, s>>>(q, k, v, p);
  return cudaGetLastError();
}

}  // namespace

int64_t forward_tiles(const AttnArgs& a) { return a.Tq / (256 / heads_packed(a.group)) + a.B; }

cudaError_t launch_tc(const AttnArgs& a, TilePlan* plan, cudaStream_t s) {
  return a.D <= 64 ? forward<64>(a, plan, s) : forward<128>(a, plan, s);
}

}  // namespace attn
}  // namespace moe
