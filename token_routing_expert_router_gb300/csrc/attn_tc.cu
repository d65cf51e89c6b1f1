// Attention on the tensor cores (bf16, D <= 128), one pass over the keys.
//
// A CTA takes one item after the other, two tiles of 128 rows of Q against one key head, and goes over
// its keys in tiles of 128:
//   S = Q K^T (tensor memory) -> P = exp2(c (S - m)), bf16, over S's columns -> O += P V (tensor memory)
// Rows of a tile are (query, head) pairs, `pack` query heads of the group side by side: a key tile is
// loaded once for 256 of them, and few queries of many heads still fill a tile.
// Warps 0 and 3 load by TMA (K two tiles ahead, V three, each on its own: through one ring of five a tile of
// V had no more than a step to come), warp 1 issues the products, and each of the two
// warpgroups 1 and 2 is one tile's softmax, a thread a row: no exchange between threads. While one
// tile's softmax runs, the tensor cores work on the other tile's products; S is free for the next scores
// as soon as P V has been issued behind them, since one thread's products run in their order.
//
// The online softmax is Milakov and Gimelshein's (2018); following the maximum past a threshold only is a
// published refinement of it. The running maximum is only followed when it grows by more than 2^8 in the exponentials (then O is
// read, scaled and written back, by the rows' own threads); until then the old one is as good a
// reference, since all sums are fp32 and P's rounding is relative. The keys are taken from the last to
// the first, so that the tile with the mask comes first. Key rows behind the sequence's end belong to
// somebody else: their scores are replaced, and their V rows are zeroed in shared memory.
//
// Items come in the order of their work, the longest first, and a CTA takes the next one when its loads
// are nearly through with the last (shares fixed beforehand cost 15 % with two items a CTA: SMs are not
// equally far from memory). The loads and the first scores of an item run while the last one's O is
// written: a short sequence's tile is little more than such ends (40 prompts of 225 tokens: 51 us with a
// CTA for every item).
//
// Bound by the tensor cores and what feeds them. A step's products read shared memory in 1536 wavefronts of 128 bytes
// (counted), 1024 of them in the scores' products, which take as many cycles: all there is meanwhile, and the
// next keys are written beside. The rest of a step is the chain from scores to P. 16384 tokens, 32 query
// and 8 key heads of 128, causal: 1.66 ms, 1.32 PFLOP/s (69 % of the measured peak).
#include "attn_plan.cuh"
#include "attn_tc.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kIds = 2;  // items whose number is known at once

struct FwdParams {
  AttnArgs a;
  int pack;     // query heads in a tile
  float c;      // scale log2(e)
  int tiles, heads, chunk;  // tiles (at most), packs of heads, packs that share the L2
  const TilePlan* plan;     // NULL: one sequence
  int* queue;               // [2]: items taken beyond the CTAs' first ones, CTAs that are through; zero between calls
};

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attn_forward_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const FwdParams p) {
  using F = Fwd<DP>;
  constexpr int kNK = F::kNK, kNV = F::kNV;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = smem + 2 * F::kQ * F::kTile;
  uint8_t* sV = sK + kNK * F::kTile;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(sV + kNV * F::kTile);
  uint64_t* k_empty = k_full + kNK;
  uint64_t* v_full = k_empty + kNK;
  uint64_t* v_empty = v_full + kNV;
  uint64_t* q_full = v_empty + kNV;
  uint64_t* q_empty = q_full + F::kQ;
  uint64_t* s_full = q_empty + F::kQ;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* o_free = o_full + 2;
  uint64_t* id_full = o_free + 2;
  uint64_t* id_empty = id_full + kIds;
  uint64_t* drain = id_empty + kIds;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* ids = abort + 1;  // of the items, -1 behind the last
  static_assert((2 * 8 + 13 + 2 * kIds) * 8 + 8 + 4 * kIds <= 512);

  const AttnArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = 128 / p.pack;  // queries of a tile

  if (threadIdx.x == 0) {
    for (int u = 0; u < kNK; ++u) {
      mbar_init(&k_full[u], 1);
      mbar_init(&k_empty[u], 1);
    }
    for (int u = 0; u < kNV; ++u) {
      mbar_init(&v_full[u], 1);
      mbar_init(&v_empty[u], 1);
    }
    for (int b = 0; b < F::kQ; ++b) {
      mbar_init(&q_full[b], 1);
      mbar_init(&q_empty[b], 1);
    }
    for (int m = 0; m < 2; ++m) {
      mbar_init(&s_full[m], 1);
      mbar_init(&p_full[m], 4);
      mbar_init(&o_full[m], 1);
      mbar_init(&o_free[m], 4);
    }
    for (int i = 0; i < kIds; ++i) {
      mbar_init(&id_full[i], 1);
      mbar_init(&id_empty[i], 10);  // the warp that loads V, the issuing warp, the softmax warps
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

  after_previous();
  Seq only{};
  if (!p.plan) only = load_seq(a, 0, blockIdx.x == 0 && threadIdx.x == 0);
  const int tiles = p.plan ? p.plan->count : (only.n + 2 * per - 1) / (2 * per), items = tiles * p.heads;
  struct Item {
    Seq s;
    int i0, h0;     // first query, first query head
    int n0, n1;     // key tiles of the two row tiles
    __device__ int steps() const { return max(n0, n1); }
    __device__ int of(int m) const { return m ? n1 : n0; }
  };
  auto item = [&](int id, Item& it) {
    const Place at = place_of(id, tiles, p.heads, p.chunk);
    it.h0 = at.head * p.pack;
    if (p.plan) {
      const TileEntry* e = p.plan->tile + at.rank;
      it.s = Seq{e->q0, e->n, e->k0, e->m};
      it.i0 = e->start;
    } else {
      it.s = only;
      it.i0 = (tiles - 1 - at.rank) * 2 * per;
    }
    auto key_tiles = [&](int first) {
      const int last = min(first + per, it.s.n) - 1;
      return last < first ? 0 : (max(0, visible(a, it.s, last)) + BK - 1) / BK;
    };
    it.n0 = key_tiles(it.i0), it.n1 = key_tiles(it.i0 + per);
  };
  // a warp's view of the CTA's k-th item; false: there is none (or given up)
  auto taken = [&](int k, Item& it) {
    const bool come = mbar_wait(&id_full[k % kIds], k / kIds & 1, abort, kTimeoutNs, a.status);
    if (!__all_sync(0xffffffffu, come)) return false;
    const int id = ids[k % kIds];
    __syncwarp();
    if (lane == 0) mbar_arrive(&id_empty[k % kIds]);
    if (id < 0) return false;
    item(id, it);
    return true;
  };

  auto load_tile = [&](const CUtensorMap* map, uint8_t* dst, uint64_t* bar, int head, int row) {
    mbar_arrive_expect_tx(bar, F::kTile);
#pragma unroll
    for (int d = 0; d < F::kSlabs; ++d) tma_load_3d(map, dst + d * 16384, bar, 64 * d, head, row);
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 0 && lane == 0) {
      // ===================== loads of Q and K, from the last tile on, and the queue
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      int unit = 0, issued = 0, queries = 0;
      uint32_t phase = 0;
      bool ok = true;
      auto take = [&] { return (int)gridDim.x + atomicAdd(p.queue, 1); };
      Item it;
      for (int k = 0, id = blockIdx.x; ok; ++k) {
        if (!(ok = mbar_wait(&id_empty[k % kIds], (k / kIds & 1) ^ 1, abort, kTimeoutNs, a.status))) break;
        ids[k % kIds] = id < items ? id : -1;
        mbar_arrive(&id_full[k % kIds]);
        if (id >= items) break;
        item(id, it);
        const int steps = it.steps(), hk = it.h0 / a.group;
        if (steps == 0) {
          id = take();
          continue;
        }
        const int b = queries % F::kQ;
        if (!(ok = mbar_wait(&q_empty[b], (queries / F::kQ & 1) ^ 1, abort, kTimeoutNs, a.status))) break;
        ++queries;
        mbar_arrive_expect_tx(&q_full[b], 2 * F::kTile);
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int d = 0; d < F::kSlabs; ++d)
            tma_load_3d(&tmQ, sQ + (2 * b + m) * F::kTile + d * 16384, &q_full[b], 64 * d, it.h0, it.s.q0 + it.i0 + m * per);
        for (int j = steps - 1; j >= 0; --j) {
          if (j == min(steps - 1, 2)) id = take();
          if (!(ok = mbar_wait(&k_empty[unit], phase ^ 1, abort, kTimeoutNs, a.status))) break;
          load_tile(&tmK, sK + unit * F::kTile, &k_full[unit], hk, it.s.k0 + j * BK);
          ++issued;
          if (++unit == kNK) unit = 0, phase ^= 1;
        }
      }
      // the last CTA leaves the queue as it was
      __threadfence();
      if (ok && atomicAdd(p.queue + 1, 1) == (int)gridDim.x - 1) p.queue[0] = p.queue[1] = 0;
      // leave no copy in flight
      for (int i = max(0, queries - F::kQ); i < queries; ++i)
        mbar_wait_drain(&q_full[i % F::kQ], i / F::kQ & 1, kTimeoutNs, a.status);
      for (int i = max(0, issued - kNK); i < issued; ++i) mbar_wait_drain(&k_full[i % kNK], i / kNK & 1, kTimeoutNs, a.status);
    } else if (warp == 3) {
      // ===================== loads of V
      if (lane == 0) tma_prefetch_desc(&tmV);
      int unit = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      Item it;
      for (int k = 0; ok && taken(k, it); ++k) {
        const int hk = it.h0 / a.group;
        for (int j = it.steps() - 1; j >= 0; --j) {
          ok = mbar_wait(&v_empty[unit], phase ^ 1, abort, kTimeoutNs, a.status);
          if (!(ok = __all_sync(0xffffffffu, ok))) break;
          if (lane == 0) load_tile(&tmV, sV + unit * F::kTile, &v_full[unit], hk, it.s.k0 + j * BK);
          __syncwarp();
          ++issued;
          if (++unit == kNV) unit = 0, phase ^= 1;
        }
      }
      for (int i = max(0, issued - kNV); i < issued; ++i) mbar_wait_drain(&v_full[i % kNV], i / kNV & 1, kTimeoutNs, a.status);
    } else if (warp == 1) {
      // ===================== products
      const uint32_t idesc_s = idesc_make(1, 128, BK);
      const uint32_t idesc_o = idesc_make(1, 128, DP) | (1u << 16);  // V is read MN-major
      int uk = 0, uv = 0;  // tiles of K and V that are next
      uint32_t k_phase = 0, v_phase = 0, p_phase = 0, o_phase = 0;  // the latter two a bit for each row tile
      int queries = 0;
      const bool one = lane == 0;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool ok = mbar_wait(bar, parity, abort, kTimeoutNs, a.status);
        return (bool)__all_sync(0xffffffffu, ok);
      };
      auto scores = [&](int m, uint32_t q_desc, uint32_t ka) {  // S_m = Q_m K^T
        const uint32_t qa = q_desc + m * (F::kTile / 16);
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          const uint32_t off = (k / 4) * (16384 / 16) + (k % 4) * 2;
          mma_ss(tS + 128 * m, qa + off, ka + off, idesc_s, k > 0, one);
        }
        commit(&s_full[m], one);
      };
      bool ok = true;
      Item it;
      for (int k = 0; ok && taken(k, it); ++k) {
        const int steps = it.steps(), keys = it.s.m;
        if (steps == 0) continue;
        const int b = queries % F::kQ;
        if (!(ok = wait(&q_full[b], queries / F::kQ & 1) && wait(&k_full[uk], k_phase))) break;
        ++queries;
        const uint32_t q_desc = uniform(k_desc(smem_addr(sQ + 2 * b * F::kTile)));
        tc_fence_after();
        auto next_k = [&] {
          if (++uk == kNK) uk = 0, k_phase ^= 1;
        };
        for (int m = 0; m < 2; ++m)
          if (it.of(m) == steps) scores(m, q_desc, uniform(k_desc(smem_addr(sK + uk * F::kTile))));
        commit(&k_empty[uk], one);
        next_k();
        if (steps == 1) commit(&q_empty[b], one);
        for (int j = steps - 1; j >= 0; --j) {
          if (j > 0 && !(ok = wait(&k_full[uk], k_phase))) break;
          if (!(ok = wait(&v_full[uv], v_phase))) break;
          if ((j + 1) * BK > keys) clear_rows(sV + uv * F::kTile, F::kSlabs, BK, keys - j * BK, lane);
          tc_fence_after();
          // all that the products need is at hand before their P is waited for
          const uint32_t va = uniform(mn_desc(smem_addr(sV + uv * F::kTile))), ka = uniform(k_desc(smem_addr(sK + uk * F::kTile)));
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            if (!ok) break;
            const int n = it.of(m);
            if (j < n) {
              if (!(ok = wait(&p_full[m], p_phase >> m & 1))) break;
              p_phase ^= 1u << m;
              if (j == n - 1) {  // O of the item before has been read
                if (!(ok = wait(&o_free[m], (o_phase >> m & 1) ^ 1))) break;
                o_phase ^= 1u << m;
              }
              tc_fence_after();
#pragma unroll
              for (int q = 0; q < BK / 16; ++q)  // O_m += P_m V
                mma_ts(tO + DP * m, tS + 128 * m + 8 * q, va + (2048 / 16) * q, idesc_o, j < n - 1 || q > 0, one);
              if (j == 0) commit(&o_full[m], one);
            }
            if (m == 1) commit(&v_empty[uv], one);  // ahead of the last scores
            if (j > 0 && j - 1 < n) scores(m, q_desc, ka);
          }
          if (!ok) break;
          if (++uv == kNV) uv = 0, v_phase ^= 1;
          if (j > 0) {
            commit(&k_empty[uk], one);
            next_k();
          }
          if (j == 1) commit(&q_empty[b], one);
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
    // ===================== softmax of row tile m, a thread a row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int m = warp / 4 - 1, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t my_s = tS + 128 * m + lanes, my_o = tO + DP * m + lanes;
    uint32_t s_phase = 0, o_phase = 0;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      const bool ok = mbar_wait(bar, parity, abort, kTimeoutNs, a.status);
      return (bool)__all_sync(0xffffffffu, ok);
    };
#pragma unroll 1
    for (int k = 0;; ++k) {
      int n, seen, least, q_row, h;  // key tiles; keys that this row and that the tile's first row see; the row (-1: none)
      {
        Item it;
        if (!taken(k, it)) break;
        const int i = it.i0 + m * per + row / p.pack;
        n = it.of(m);
        seen = visible(a, it.s, i);
        least = visible(a, it.s, it.i0 + m * per);
        q_row = i < it.s.n ? it.s.q0 + i : -1;
        h = it.h0 + row % p.pack;
      }
      Running w;
      bool ok = true;
#pragma unroll 1
      for (int j = n - 1; j >= 0; --j) {
        if (!(ok = wait(&s_full[m], s_phase))) break;
        s_phase ^= 1;
        tc_fence_after();
        softmax_step<DP>(my_s, my_o, p.c, (j + 1) * BK > least ? seen - j * BK : BK, j < n - 1, w);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[m]);
      }
      // ===================== O / sum and the log sum
      const float sum = w.sum0 + w.sum1, top = w.top;
      if (n > 0) {
        if (!ok || !wait(&o_full[m], o_phase)) break;
        o_phase ^= 1;
        tc_fence_after();
      }
      const bool live = q_row >= 0;
      const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.o) + (int64_t)q_row * a.ld_o + (int64_t)h * a.D;
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
      if (n > 0) {  // O may be written again
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_free[m]);
      }
      if (live)
        a.lse[(int64_t)h * a.Tq + q_row] = sum == 0.0f ? -INFINITY : (top * p.c + log2f(sum)) * kLn2;
    }
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int DP>
cudaError_t forward(const AttnArgs& a, TilePlan* plan, int* first, int* queue, cudaStream_t s) {
  FwdParams p{a, heads_packed(a.group), a.scale * kLog2e};
  p.queue = queue;
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
  static Once once;
  const cudaError_t e = allow_smem(once, attn_forward_kernel<DP>, Fwd<DP>::kBytes);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)min((int64_t)tc::num_sms(), (int64_t)p.tiles * p.heads);
  // one sequence's tiles are in the order of their work as they are
  if (a.B > 1) {
    p.plan = plan;
    const cudaError_t l = launch_plan(a, PlanJob{0, 256 / p.pack, 0, 0, p.heads, 0, p.tiles, plan, first}, s);
    if (l != cudaSuccess) return l;
    return launch_after_smem(attn_forward_kernel<DP>, grid, kThreads, Fwd<DP>::kBytes, s, q, k, v, p);
  }
  attn_forward_kernel<DP><<<grid, kThreads, Fwd<DP>::kBytes, s>>>(q, k, v, p);
  return cudaGetLastError();
}

}  // namespace

int64_t forward_tiles(const AttnArgs& a) { return a.Tq / (256 / heads_packed(a.group)) + a.B; }

cudaError_t launch_tc(const AttnArgs& a, TilePlan* plan, int* first, int* queue, cudaStream_t s) {
  return a.D <= 64 ? forward<64>(a, plan, first, queue, s) : forward<128>(a, plan, first, queue, s);
}

}  // namespace attn
}  // namespace moe
