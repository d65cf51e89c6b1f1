// The backward of attention on the tensor cores (bf16, D <= 128): dk and dv of 128 keys of a head by one
// kernel, dq of 128 (query, head) rows by another. Both are the same loop: an outer tile stays in shared
// memory (X1, X2 = K, V or Q, dO), inner tiles of 128 rows go by (Y1, Y2 = Q, dO or K, V), and
//   S = X1 Y1^T,  dP = X2 Y2^T   (tensor memory)
//   P = exp2(c S - lse2),  dS = P (dP - delta)   (bf16, over the columns of S and dP)
//   dV += P Y2, dK += dS Y1;   M += P Y1, dQ += dS Y1
// with rows of the outer tile as lanes of tensor memory, so that P and dS are first operands where they
// are. Sums over the query heads of a group and over all queries stay in one accumulator: no atomics,
// and the bits never change. In return S and dP are formed twice.
//
// P and dS are rounded to bf16 (2^-8 of each at most): the tensor cores take both operands of a product in one
// type. The sums of dS are of the unrounded ones. By norm gradients are off by 0.24 %, where their own rounding
// alone makes 0.17.
//
// M serves delta. It is the sum over the keys of P dP, and formed as d_o . o it carries the rounding of o
// to bf16 and of P in the forward: where a row looks at few keys, dP - delta is small against both, and
// gradients were off by up to 0.4 % for that alone (their own rounding: 0.17 %). The sum e of a row's dS
// is what delta lacks, as the sum of P is 1: dq takes e M back, M the mean key, and leaves delta + e for dk.
//
// A tile of keys that meets very many queries is cut into pieces (attn_plan.cu): each leaves its sums in
// the workspace, and the CTA that comes last (a ticket; it waits for nobody) adds them in their order.
//
// Warp 0 loads by TMA, warp 1 issues the products, warp 2 brings lse and delta of the inner rows (dk, dv),
// warpgroups 1 and 2 form P and dS, each of one half of the columns. The products of one inner tile
// take the tensor cores twice as long as P and dS take the warps, and they interleave without a second
// set of accumulators (there is no room for one: S, dP, dK and dV fill tensor memory): while dS(t) is
// formed, dV(t) and S(t+1) run, while P(t+1) is formed, dK(t) and dP(t+1).
//
// Bound by the tensor cores and their shared-memory operands: 8192 tokens, 32 query and 8 key heads of 128,
// causal: dq 755 us, dk and dv 760 us, 1.45 PFLOP/s of products each.
#include "attn_plan.cuh"
#include "attn_tc.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int R = 128;  // rows of every tile

template <int DP>
struct Bwd {
  static constexpr int kSlabs = DP / 64;
  static constexpr int kTile = R * DP * 2;
  // Stages of Y1, which is read from S to the end of a step, and of Y2. A load takes about a step.
  static constexpr int kN1 = DP == 64 ? 4 : 3, kN2 = DP == 64 ? 4 : 2;
  static constexpr int kStats = 2 * R * 2 * 4;  // two stages of -lse2 and -delta
  static constexpr int kTiles = 2 + kN1 + kN2;
  // All of it is dynamic, and begins on a boundary of 1024 bytes. A CTA takes all of tensor memory: the
  // size leaves no second one on its SM.
  static constexpr size_t kBytes = kTiles * kTile + kStats + 256;
  static_assert(kBytes > 116 * 1024 && kBytes <= 227 * 1024);
};

struct BwdParams {
  AttnArgs a;
  int pack;   // query heads in a tile
  float c;    // scale log2(e)
  int tiles, heads, chunk;  // the grid: tiles (at most), packs of heads or key heads, those that share the L2
  const TilePlan* plan;
  const float* neg_lse;
  float* neg_delta;   // dq leaves it exact for dk
  float* part;
  uint32_t* tickets;
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
  constexpr int kN1 = F::kN1, kN2 = F::kN2;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sX = smem;                   // X1, X2
  uint8_t* sY1 = smem + 2 * F::kTile;
  uint8_t* sY2 = sY1 + kN1 * F::kTile;
  float* sStat = reinterpret_cast<float*>(smem + F::kTiles * F::kTile);  // [stage][-lse2, -delta][R]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + F::kTiles * F::kTile + F::kStats);
  uint64_t* x_full = bars;
  uint64_t* y1_full = x_full + 1;
  uint64_t* y1_empty = y1_full + kN1;
  uint64_t* y2_full = y1_empty + kN1;
  uint64_t* y2_empty = y2_full + kN2;
  uint64_t* stat_full = y2_empty + kN2;
  uint64_t* stat_empty = stat_full + 2;
  uint64_t* s_full = stat_empty + 2;
  uint64_t* dp_full = s_full + 1;
  uint64_t* p_ready = s_full + 2;
  uint64_t* ds_ready = s_full + 3;
  uint64_t* acc_full = s_full + 4;
  uint64_t* both = s_full + 5;
  uint64_t* drain = s_full + 6;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* last_one = abort + 1;
  static_assert((1 + 2 * kN1 + 2 * kN2 + 4 + 7) * 8 + 12 <= 256);

  const AttnArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (smem_addr(smem) & 1023) {  // the tiles' swizzle counts on it; a launch without static shared memory has it so
    if (threadIdx.x == 0) set_status(a.status, MOE_ERR_CUDA, -1);
    return;
  }
  const int per = R / p.pack;  // queries of a tile
  const Place at = place_of(blockIdx.x, p.tiles, p.heads, p.chunk);
  const int hk = DKV ? at.head : at.head * p.pack / a.group;
  const int h0 = DKV ? hk * a.group : at.head * p.pack;  // first query head
  let_next_begin();
  after_previous();
  if (at.rank >= p.plan->count) return;
  const TileEntry e = p.plan->tile[at.rank];
  const Seq s{e.q0, e.n, e.k0, e.m};
  const int o0 = e.start;  // the outer tile's first key or query
  // inner tiles: of queries, from the first one that sees key o0, for one pack of heads after the other;
  // or of keys
  const int first = DKV && a.causal ? max(0, o0 - (s.m - s.n)) / per : 0;
  const int tiles = max(0, (s.n + per - 1) / per - first);
  const int from = e.lo, steps = e.hi - e.lo;
  struct Inner {  // walks over them
    int tile, head;
  };
  auto begin = [&] { return DKV && steps > 0 ? Inner{from % tiles, h0 + from / tiles * p.pack} : Inner{from, h0}; };
  auto advance = [&](Inner& i) {
    ++i.tile;
    if (DKV && i.tile == tiles) i.tile = 0, i.head += p.pack;
  };
  auto row_of = [&](const Inner& i) { return DKV ? (first + i.tile) * per : i.tile * R; };  // in the sequence
  // rows of it that are the sequence's
  auto live_of = [&](const Inner& i) { return DKV ? min(per, s.n - row_of(i)) * p.pack : min(R, s.m - row_of(i)); };

  if (threadIdx.x == 0) {
    mbar_init(x_full, 1);
    for (int b = 0; b < kN1; ++b) {
      mbar_init(&y1_full[b], 1);
      mbar_init(&y1_empty[b], 1);
    }
    for (int b = 0; b < kN2; ++b) {
      mbar_init(&y2_full[b], 1);
      mbar_init(&y2_empty[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&stat_full[b], 32);
      mbar_init(&stat_empty[b], 8);
    }
    mbar_init(both, 8);
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
      int u1 = 0, u2 = 0, n1 = 0, n2 = 0;  // stages, loads
      uint32_t ph1 = 0, ph2 = 0;
      Inner in = begin();
      for (int i = 0; i < steps && ok; ++i, advance(in)) {
        const int head = DKV ? in.head : hk, row = (DKV ? s.q0 : s.k0) + row_of(in);
        if (!(ok = mbar_wait(&y1_empty[u1], ph1 ^ 1, abort, kTimeoutNs, a.status))) break;
        mbar_arrive_expect_tx(&y1_full[u1], F::kTile);
        load(DKV ? &tmQ : &tmK, sY1 + u1 * F::kTile, &y1_full[u1], head, row);
        ++n1;
        if (++u1 == kN1) u1 = 0, ph1 ^= 1;
        if (!(ok = mbar_wait(&y2_empty[u2], ph2 ^ 1, abort, kTimeoutNs, a.status))) break;
        mbar_arrive_expect_tx(&y2_full[u2], F::kTile);
        load(DKV ? &tmO : &tmV, sY2 + u2 * F::kTile, &y2_full[u2], head, row);
        ++n2;
        if (++u2 == kN2) u2 = 0, ph2 ^= 1;
      }
      // leave no copy in flight
      mbar_wait_drain(x_full, 0, kTimeoutNs, a.status);
      for (int i = max(0, n1 - kN1); i < n1; ++i) mbar_wait_drain(&y1_full[i % kN1], i / kN1 & 1, kTimeoutNs, a.status);
      for (int i = max(0, n2 - kN2); i < n2; ++i) mbar_wait_drain(&y2_full[i % kN2], i / kN2 & 1, kTimeoutNs, a.status);
    } else if (warp == 1 && steps > 0) {
      // ===================== products
      const uint32_t idesc_s = idesc_make(1, R, R);
      const uint32_t idesc_a = idesc_make(1, R, DP) | (1u << 16);  // the inner tile is read MN-major
      auto all = [&](bool ok) { return (bool)__all_sync(0xffffffffu, ok); };
      const bool one = lane == 0;
      // S or dP = X Y^T
      auto scores = [&](uint32_t d, uint32_t xa, uint32_t ya, uint64_t* bar) {
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          const uint32_t off = (k / 4) * (16384 / 16) + (k % 4) * 2;
          mma_ss(d, xa + off, ya + off, idesc_s, k > 0, one);
        }
        commit(bar, one);
      };
      // acc += W Y, W in tensor memory: the columns' halves each at the start of their half of the scores
      auto products = [&](uint32_t d, uint32_t w, uint32_t ya, bool begin) {
#pragma unroll
        for (int k = 0; k < R / 16; ++k)
          mma_ts(d, w + (k / 4) * 64 + (k % 4) * 8, ya + (2048 / 16) * k, idesc_a, !begin || k > 0, one);
      };
      // the next inner tile's Y1 (Y2) has come; rows that are not the sequence's are zeroed
      auto arrived = [&](uint64_t* bar, uint32_t parity, uint8_t* y, const Inner& in) {
        if (!all(mbar_wait(bar, parity, abort, kTimeoutNs, a.status))) return false;
        const int live = live_of(in);
        if (live < R) clear_rows(y, F::kSlabs, R, live, lane);
        tc_fence_after();
        return true;
      };
      const uint32_t x1 = uniform(k_desc(smem_addr(sX))), x2 = uniform(k_desc(smem_addr(sX + F::kTile)));
      int u1 = 0, u2 = 0;  // stages of the step
      uint32_t ph1 = 0, ph2 = 0;
      Inner in = begin();
      bool ok = all(mbar_wait(x_full, 0, abort, kTimeoutNs, a.status)) && arrived(y1_full, 0, sY1, in);
      if (ok) scores(tS, x1, uniform(k_desc(smem_addr(sY1))), s_full);
      ok = ok && arrived(y2_full, 0, sY2, in);
      if (ok) scores(tP, x2, uniform(k_desc(smem_addr(sY2))), dp_full);
      for (int i = 0; i < steps && ok; ++i) {
        const uint32_t parity = i & 1;
        const int v1 = u1 + 1 == kN1 ? 0 : u1 + 1, v2 = u2 + 1 == kN2 ? 0 : u2 + 1;  // of the next step
        if (v1 == 0) ph1 ^= 1;
        if (v2 == 0) ph2 ^= 1;
        advance(in);
        // all that the products need is at hand before what they wait for
        const uint32_t y1 = uniform(mn_desc(smem_addr(sY1 + u1 * F::kTile))), y2 = uniform(mn_desc(smem_addr(sY2 + u2 * F::kTile)));
        const uint32_t z1 = uniform(k_desc(smem_addr(sY1 + v1 * F::kTile))), z2 = uniform(k_desc(smem_addr(sY2 + v2 * F::kTile)));
        if (!(ok = all(mbar_wait(p_ready, parity, abort, kTimeoutNs, a.status)))) break;
        tc_fence_after();
        products(tA2, tS, DKV ? y2 : y1, i == 0);
        commit(&y2_empty[u2], one);
        if (i + 1 < steps) {
          if (!(ok = arrived(&y1_full[v1], ph1, sY1 + v1 * F::kTile, in))) break;
          scores(tS, x1, z1, s_full);
        }
        if (!(ok = all(mbar_wait(ds_ready, parity, abort, kTimeoutNs, a.status)))) break;
        tc_fence_after();
        products(tA1, tP, y1, i == 0);
        commit(&y1_empty[u1], one);
        if (i + 1 < steps) {
          if (!(ok = arrived(&y2_full[v2], ph2, sY2 + v2 * F::kTile, in))) break;
          scores(tP, x2, z2, dp_full);
        }
        u1 = v1, u2 = v2;
      }
      __syncwarp();
      if (lane == 0) {
        if (ok) mma_commit(acc_full);
        mma_commit(drain);
        mbar_wait_drain(drain, 0, kTimeoutNs, a.status);
      }
      __syncwarp();
    } else if (DKV && warp == 2) {
      // ===================== -lse2 and -delta of the inner rows, a step ahead of their use; a row that is
      // not there gets p = exp2(s - inf) = 0
      Inner in = begin();
      float v[8];
      auto fetch = [&] {  // from L2: dq, whose CTAs may have been on this SM until now, has written delta
        const int64_t base = (int64_t)(in.head / p.pack) * a.Tq * p.pack + (int64_t)(s.q0 + row_of(in)) * p.pack;
        const int live = live_of(in);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = 32 * q + lane;
          v[q] = r < live ? __ldcg(p.neg_lse + base + r) : -INFINITY;
          v[4 + q] = r < live ? __ldcg(p.neg_delta + base + r) : 0.0f;
        }
      };
      if (steps > 0) fetch();
      for (int i = 0; i < steps; ++i) {
        const int b = i & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(&stat_empty[b], (i >> 1 & 1) ^ 1, abort, kTimeoutNs, a.status))) break;
#pragma unroll
        for (int q = 0; q < 8; ++q) sStat[b * 2 * R + q / 4 * R + 32 * (q % 4) + lane] = v[q];
        mbar_arrive(&stat_full[b]);
        advance(in);
        if (i + 1 < steps) fetch();
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
    float neg_lse = -INFINITY, neg_delta = 0.0f, lack0 = 0.0f, lack1 = 0.0f;  // lack: what delta lacks, of this half
    int seen = 0;
    const int64_t stat_at = ((int64_t)at.head * a.Tq + s.q0 + i_q) * p.pack + row % p.pack;
    if (!DKV && i_q < s.n) {
      neg_lse = p.neg_lse[stat_at];
      neg_delta = p.neg_delta[stat_at];
      seen = visible(a, s, i_q);
    }
    Inner in = begin();
    bool ok = true;
    for (int i = 0; i < steps; ++i, advance(in)) {
      const int b = i & 1, row0 = row_of(in);
      const float4* stat = reinterpret_cast<const float4*>(sStat + b * 2 * R + 64 * half);
      if (DKV && !(ok = __all_sync(0xffffffffu, mbar_wait(&stat_full[b], i >> 1 & 1, abort, kTimeoutNs, a.status)))) break;
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(s_full, b, abort, kTimeoutNs, a.status)))) break;
      tc_fence_after();
      uint32_t r[2][32];
      tmem_ld32(my_s, r[0]);
      tmem_ld32(my_s + 32, r[1]);
      tmem_ld_wait();
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
      } else if (row0 + R > visible(a, s, o0)) {
        const int end = seen - row0 - 64 * half;
#pragma unroll
        for (int l = 0; l < 64; ++l)
          if (l >= end) pr[l] = 0.0f;
      }
      {
        uint32_t w[32];
#pragma unroll
        for (int l = 0; l < 32; ++l) w[l] = pack2(pr[2 * l], pr[2 * l + 1]);
        tmem_st32(my_s, w);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_ready);
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
        if constexpr (!DKV) {
          add2(lack0, lack1, d[0], d[1]);
          add2(lack0, lack1, d[2], d[3]);
        }
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
    uint32_t turn = 0;
    auto both_sync = [&] {  // of both warpgroups; false: given up
      __syncwarp();
      if (lane == 0) mbar_arrive(both);
      const bool come = __all_sync(0xffffffffu, mbar_wait(both, turn, abort, kTimeoutNs, a.status));
      turn ^= 1;
      return come;
    };
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
    if (DKV && e.cut) {
      // a piece: its sums into the workspace, added up by whoever comes last
      const int slot = e.cut >> 16, number = e.cut >> 8 & 255, pieces = e.cut & 255;
      auto place = [&](int i) { return (int64_t)((slot + i) * p.heads + hk) * 2 * R * DP; };
      float* mine = p.part + place(number) + row * DP + kCols * half;
#pragma unroll 1
      for (int q = 0; q < 2 * kCols; q += 16) {
        const int which = q >= kCols, col = q - which * kCols;
        uint32_t o[16] = {};
        if (steps > 0) {
          tmem_ld16((which ? tA2 : tA1) + lanes + kCols * half + col, o);
          tmem_ld_wait();
        }
        if (live)
#pragma unroll
          for (int l = 0; l < 16; l += 4)
            *reinterpret_cast<uint4*>(mine + which * R * DP + col + l) = make_uint4(o[l], o[l + 1], o[l + 2], o[l + 3]);
      }
      __threadfence();
      if (ok && both_sync()) {
        uint32_t* ticket = p.tickets + slot * p.heads + hk;
        if (half == 0 && row == 0) {
          const bool last = atomicAdd(ticket, 1u) == (uint32_t)pieces - 1;
          if (last) *ticket = 0;
          *last_one = last;
        }
        if (both_sync() && *last_one) {
          __threadfence();
          const int rows = min(R, s.m - o0);
          for (int x = half * 128 + row; x < 2 * rows * (DP / 4); x += 256) {
            const int which = x >= rows * (DP / 4), y = x - which * rows * (DP / 4), r = y / (DP / 4), d = y % (DP / 4) * 4;
            float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int i = 0; i < pieces; ++i) {
              const float4 v = __ldcg(reinterpret_cast<const float4*>(p.part + place(i) + which * R * DP + r * DP + d));
              sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
            }
            const float f = which ? 1.0f : a.scale;
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(which ? a.dv : a.dk) +
                                 (int64_t)(s.k0 + o0 + r) * (which ? a.ld_v : a.ld_k) + (int64_t)hk * a.D + d;
            if (d < a.D) *reinterpret_cast<uint2*>(dst) = make_uint2(pack2(sum.x * f, sum.y * f), pack2(sum.z * f, sum.w * f));
          }
        }
      }
    } else if constexpr (DKV) {
      store(tA1, a.dk, (int64_t)(s.k0 + o0 + row) * a.ld_k + (int64_t)hk * a.D, a.scale);
      store(tA2, a.dv, (int64_t)(s.k0 + o0 + row) * a.ld_v + (int64_t)hk * a.D, 1.0f);
    } else {
      sStat[half * R + row] = lack0 + lack1;
      ok = ok && both_sync();
      const float lack = sStat[row] + sStat[R + row];
      if (ok && half == 0 && i_q < s.n) p.neg_delta[stat_at] = neg_delta - lack;
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.dq) + (int64_t)(s.q0 + i_q) * a.ld_q + (int64_t)h * a.D;
#pragma unroll 1
      for (int col = kCols * half; col < kCols * (half + 1); col += 16) {
        uint32_t x[16] = {}, y[16] = {};
        if (steps > 0) {
          tmem_ld16(tA1 + lanes + col, x);
          tmem_ld16(tA2 + lanes + col, y);
          tmem_ld_wait();
        }
        float v[16];
#pragma unroll
        for (int l = 0; l < 16; ++l) v[l] = a.scale * fmaf(-lack, __uint_as_float(y[l]), __uint_as_float(x[l]));
#pragma unroll
        for (int l = 0; l < 16; l += 8)
          if (live && ok && col + l < a.D)
            *reinterpret_cast<uint4*>(dst + col + l) =
                make_uint4(pack2(v[l], v[l + 1]), pack2(v[l + 2], v[l + 3]), pack2(v[l + 4], v[l + 5]), pack2(v[l + 6], v[l + 7]));
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int DP, bool DKV>
cudaError_t launch(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const CUtensorMap& o, const BwdParams& p,
                   cudaStream_t s) {
  static Once once;
  const cudaError_t e = allow_smem(once, attn_backward_kernel<DP, DKV>, Bwd<DP>::kBytes);
  if (e != cudaSuccess) return e;
  if ((int64_t)p.tiles * p.heads >= (1ll << 31)) return cudaErrorInvalidConfiguration;
  return launch_after_smem(attn_backward_kernel<DP, DKV>, (unsigned)p.tiles * p.heads, kThreads, Bwd<DP>::kBytes, s, q, k, v, o, p);
}

template <int DP>
cudaError_t backward(const AttnArgs& a, const BackwardSpace& w, cudaStream_t s) {
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
  const int packs = a.group / p.pack, per = R / p.pack;
  const PlanJob dq{0, per, 0, 0, a.Hq / p.pack, 0, (int)dq_tiles(a), w.dq_plan, w.first};
  const PlanJob dkv{1, 0, per, packs, a.Hkv, kPieces, (int)(a.Tk / R + a.B), w.dkv_plan, w.first + a.B + 1};
  cudaError_t e = launch_plan_backward(a, dq, dkv, StatsJob{p.pack, w.neg_lse, w.neg_delta}, s);
  if (e != cudaSuccess) return e;
  p.neg_lse = w.neg_lse, p.neg_delta = w.neg_delta, p.part = w.part, p.tickets = w.tickets;
  if (a.Tq > 0) {
    p.tiles = (int)dq_tiles(a);
    p.heads = a.Hq / p.pack;
    p.chunk = head_chunk((int64_t)a.Tk * a.D * 4, a.Hkv) * packs;
    p.plan = w.dq_plan;
    if ((e = launch<DP, false>(q, k, v, o, p, s)) != cudaSuccess) return e;
  }
  if (a.Tk == 0) return cudaSuccess;
  p.tiles = (int)dkv_tiles(a);
  p.heads = a.Hkv;
  p.chunk = head_chunk((int64_t)a.Tq * a.group * a.D * 4, a.Hkv);
  p.plan = w.dkv_plan;
  return launch<DP, true>(q, k, v, o, p, s);
}

}  // namespace

int64_t dq_tiles(const AttnArgs& a) { return a.Tq / (R / heads_packed(a.group)) + a.B; }
int64_t dkv_tiles(const AttnArgs& a) { return a.Tk / R + a.B + kMostPieces / a.Hkv; }

cudaError_t launch_tc_backward(const AttnArgs& a, const BackwardSpace& w, cudaStream_t s) {
  return a.D <= 64 ? backward<64>(a, w, s) : backward<128>(a, w, s);
}

}  // namespace attn
}  // namespace moe
