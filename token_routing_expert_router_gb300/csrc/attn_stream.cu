// Attention of few query rows over many keys, on the tensor cores: single tokens over a cache, and
// batches whose tiles would not fill the SMs. The products and the softmax are those of attn_tc.cu; here
// one tile of 128 (query, head) rows at a time, and the work is cut at fixed shares of the key tiles:
//
// Every (sequence, tile of queries, pack of heads) is a line of key tiles, and all lines lie one behind
// the other. CTA c of N takes the c-th of N equal shares: parts of lines, at most its first and its last
// not whole. Reading the keys is all the time there is, so equal bytes are equal times, whatever the
// lengths. A line that is cut leaves its parts' maxima, sums and O (fp32) in the workspace; the CTA that
// comes last (a ticket; it waits for nobody) puts them together, in the parts' order: the same bits on
// every run.
//
// Warp 2 walks over the share and posts its parts; warp 0 loads (Q into two buffers in turn, K and V
// through a ring that runs on over the parts), warp 1 issues products, warpgroups 1 and 2 take the key
// tiles in turn, with a maximum, sum and O of their own: scores -> P -> O of one tile is a chain of some
// 3500 cycles, longer than its keys take from memory, and two of them overlap. At a part's end both
// put the two together, a half of the channels each.
//
// Bound by reading the keys: 64 requests of 1200 to 10700 of them (32 query and 8 key heads of 128, 1.75 GB):
// 276 us, 6.3 TB/s, 93 % of the measured copy rate. One request over 8192: 18 us, most of it latencies.
#include "attn_tc.cuh"

namespace moe {
namespace attn {
namespace {

constexpr int kItems = 4;  // parts posted ahead

template <int DP>
struct Ring {
  static constexpr int kUnits = DP == 128 ? 4 : 8;  // tiles of K and V: 128 KB, three times what the memory's latency asks for
  static constexpr size_t kBytes = 1024 + (2 + kUnits) * Fwd<DP>::kTile + 512;
};

struct Item {
  int kind;            // 0: the end; 1: a whole line; 2: a part of one
  int q, i0, n, m;     // first query's row of q, its place in the sequence, the sequence's queries and keys
  int k0;              // the sequence's first row of k
  int lo, hi;          // key tiles [lo, hi)
  int h0;              // first query head
  int c0, c1;          // a part: the first and the last CTA of its line
  int slot;            // a part: its place in the workspace
};

struct StreamParams {
  AttnArgs a;
  int pack, packs;     // query heads in a tile, tiles of heads
  float c;             // scale log2(e)
  double inv_ctas;     // 1 / CTAs
  uint32_t* tickets;   // [CTAs], zero between calls
  float2* stat;        // [2 CTAs][128]: maximum (of the scores as they are) and sum of every row of a part
  float* part;         // [2 CTAs][128][DP]: its O
};

// What find_share leaves: the block's share [u, end) of all tiles, and the line that u lies in.
struct Share {
  int64_t u, end;
  int64_t each;        // tiles of a share (the last one may have fewer)
  int64_t line;        // first tile of the line, of all
  int b, tile, pack;   // its sequence, tile of queries, pack of heads
};

__device__ __forceinline__ int line_tiles(const AttnArgs& a, const Seq& s, int tile, int per) {
  const int last = min((tile + 1) * per, s.n) - 1;
  return (max(0, visible(a, s, last)) + BK - 1) / BK;
}

// A line without keys still takes a turn: its rows are zeros. longest: raised to the longest line's tiles.
__device__ __forceinline__ int64_t seq_turns(const AttnArgs& a, const Seq& s, int per, int packs, int& longest) {
  int64_t n = 0;
  for (int t = 0; t * per < s.n; ++t) {
    const int len = max(1, line_tiles(a, s, t, per));
    n += len;
    longest = max(longest, len);
  }
  return n * packs;
}

__device__ void find_share(const StreamParams& p, int per, Share* out) {
  __shared__ int64_t sWarp[kThreads / 32];
  __shared__ int sLongest[kThreads / 32];
  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int each = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(a.B, tid * each), b1 = min(a.B, b0 + each);
  int64_t mine = 0;
  int longest = 0;
  for (int b = b0; b < b1; ++b) mine += seq_turns(a, load_seq(a, b, blockIdx.x == 0), per, p.packs, longest);
  int64_t inc = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += o;
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, off));
  if (lane == 31) sWarp[warp] = inc, sLongest[warp] = longest;
  __syncthreads();
  int64_t all = 0, before = inc - mine;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sWarp[w];
    all += sWarp[w];
    longest = max(longest, sLongest[w]);
  }
  int64_t share = (int64_t)(all * p.inv_ctas);
  while (share * gridDim.x < all) ++share;
  // What a CTA takes at least: lines of up to 6 tiles whole (1 query over 300 keys: 10.9 us, 14.6 with a tile
  // a CTA; over 700 14.1 and 16.8), longer ones two tiles (4 tiles: 1 query over 2048 keys 18.2 us, 14.8 with
  // two; 64 queries over 2048 40 and 29).
  share = max(share, (int64_t)(longest <= 6 ? longest : 2));
  const int64_t u = min(all, share * blockIdx.x);
  if (tid == 0) {
    out->each = share;
    out->u = u;
    out->end = min(all, u + share);
  }
  if (u >= before && u < before + mine) {
    int64_t at = before;
    for (int b = b0; b < b1; ++b) {
      const Seq s = load_seq(a, b, false);
      const int64_t turns = seq_turns(a, s, per, p.packs, longest);
      if (u < at + turns) {
        int t = 0;
        int64_t len;
        while (u >= at + (len = max(1, line_tiles(a, s, t, per))) * p.packs) at += len * p.packs, ++t;
        out->b = b;
        out->tile = t;
        out->pack = (int)((u - at) / len);
        out->line = at + out->pack * len;
        break;
      }
      at += turns;
    }
  }
  __syncthreads();
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attn_stream_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const StreamParams p) {
  using F = Fwd<DP>;
  constexpr int kUnits = Ring<DP>::kUnits;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Share share;
  __shared__ Item items[kItems];
  __shared__ float2 sStat[2][2][128];  // [part's turn][warpgroup][row]: maximum and sum
  __shared__ int last_one;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + 2 * F::kTile;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sKV + kUnits * F::kTile);
  uint64_t* full = bars;
  uint64_t* empty = bars + kUnits;
  uint64_t* q_full = bars + 2 * kUnits;
  uint64_t* q_empty = q_full + 2;
  uint64_t* s_full = q_full + 4;
  uint64_t* p_full = q_full + 6;
  uint64_t* o_full = q_full + 8;
  uint64_t* o_free = q_full + 9;
  uint64_t* it_full = q_full + 10;
  uint64_t* it_empty = it_full + kItems;
  uint64_t* both = it_empty + kItems;
  uint64_t* drain = both + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert((2 * 8 + 10 + 2 * kItems + 2) * 8 + 8 <= 512);

  const AttnArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = 128 / p.pack;  // queries of a tile
  find_share(p, per, &share);
  if (share.u >= share.end) return;

  if (threadIdx.x == 0) {
    for (int u = 0; u < kUnits; ++u) {
      mbar_init(&full[u], 1);
      mbar_init(&empty[u], 1);
    }
    for (int m = 0; m < 2; ++m) {
      mbar_init(&q_full[m], 1);
      mbar_init(&q_empty[m], 1);
      mbar_init(&s_full[m], 1);
      mbar_init(&p_full[m], 4);
    }
    mbar_init(o_full, 1);
    mbar_init(o_free, 8);
    mbar_init(both, 8);
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&it_full[i], 1);
      mbar_init(&it_empty[i], 10);  // the loading thread, the issuing warp, both warpgroups
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
  const uint32_t tS = tmem, tO = tmem + 256;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 2 && lane == 0) {
      // ===================== the share's parts
      int b = share.b, tile = share.tile, pack = share.pack;
      int64_t u = share.u, line = share.line;
      Seq s = load_seq(a, b, false);
      bool ok = true;
      for (int k = 0, end = 0; ok && !end; ++k) {
        Item it{};
        if (u < share.end) {
          const int tiles = line_tiles(a, s, tile, per), len = max(1, tiles);
          const int from = (int)(u - line), count = (int)min((int64_t)(len - from), share.end - u);
          it.kind = count == len ? 1 : 2;
          it.q = s.q0 + tile * per, it.i0 = tile * per, it.n = s.n, it.m = s.m, it.k0 = s.k0;
          it.lo = from, it.hi = tiles ? from + count : from;
          it.h0 = pack * p.pack;
          if (it.kind == 2) {
            it.c0 = it.c1 = blockIdx.x;
            for (int64_t at = share.u; at > line; at -= share.each) --it.c0;
            for (int64_t at = share.u + share.each; at < line + len; at += share.each) ++it.c1;
            it.slot = 2 * blockIdx.x + (from > 0 ? 0 : 1);
          }
          u += count;
          if (from + count == len) {  // the next line
            line += len;
            if (++pack == p.packs) {
              pack = 0;
              if (++tile * per >= s.n && u < share.end) {
                tile = 0;
                do s = load_seq(a, ++b, false);
                while (s.n == 0);
              }
            }
          }
        } else {
          end = 1;
        }
        if (!(ok = mbar_wait(&it_empty[k % kItems], (k / kItems & 1) ^ 1, abort, kTimeoutNs, a.status))) break;
        items[k % kItems] = it;
        mbar_arrive(&it_full[k % kItems]);
      }
    } else if (warp == 0 && lane == 0) {
      // ===================== loads
      int unit = 0, issued = 0;
      uint32_t phase = 0, q_phase = 0, q_used = 0;  // of the two buffers of Q, a bit each
      bool ok = true;
      auto load = [&](const CUtensorMap* map, int head, int row) {
        if (!ok || !(ok = mbar_wait(&empty[unit], phase ^ 1, abort, kTimeoutNs, a.status))) return;
        mbar_arrive_expect_tx(&full[unit], F::kTile);
#pragma unroll
        for (int d = 0; d < F::kSlabs; ++d) tma_load_3d(map, sKV + unit * F::kTile + d * 16384, &full[unit], 64 * d, head, row);
        ++issued;
        if (++unit == kUnits) unit = 0, phase ^= 1;
      };
      for (int k = 0, filled = 0; ok; ++k) {
        if (!(ok = mbar_wait(&it_full[k % kItems], k / kItems & 1, abort, kTimeoutNs, a.status))) break;
        const Item& it = items[k % kItems];
        const int kind = it.kind, lo = it.lo, hi = it.hi, q = it.q, k0 = it.k0, h0 = it.h0;
        mbar_arrive(&it_empty[k % kItems]);
        if (kind == 0) break;
        if (lo == hi) continue;
        const int m = filled++ & 1, hk = h0 / a.group;
        if (!(ok = mbar_wait(&q_empty[m], (q_phase >> m & 1) ^ 1, abort, kTimeoutNs, a.status))) break;
        q_phase ^= 1u << m, q_used |= 1u << m;
        mbar_arrive_expect_tx(&q_full[m], F::kTile);
#pragma unroll
        for (int d = 0; d < F::kSlabs; ++d) tma_load_3d(&tmQ, sQ + m * F::kTile + d * 16384, &q_full[m], 64 * d, h0, q);
        load(&tmK, hk, k0 + (hi - 1) * BK);
        for (int j = hi - 1; j >= lo; --j) {
          if (j > lo) load(&tmK, hk, k0 + (j - 1) * BK);
          load(&tmV, hk, k0 + j * BK);
        }
      }
      // leave no copy in flight
      for (int m = 0; m < 2; ++m)
        if (q_used >> m & 1) mbar_wait_drain(&q_full[m], (q_phase >> m & 1) ^ 1, kTimeoutNs, a.status);
      for (int i = 0; i < min(issued, kUnits); ++i) {
        const int u = (unit - 1 - i + 2 * kUnits) % kUnits;
        mbar_wait_drain(&full[u], unit - 1 - i < 0 ? phase ^ 1 : phase, kTimeoutNs, a.status);
      }
    } else if (warp == 1) {
      // ===================== products
      const uint32_t idesc_s = idesc_make(1, 128, BK);
      const uint32_t idesc_o = idesc_make(1, 128, DP) | (1u << 16);  // V is read MN-major
      int unit = 0;
      const bool one = lane == 0;
      uint32_t phase = 0, tile_phase = 0, turn = 0;  // tile_phase: a bit for each warpgroup; turn: whose tile is next
      auto all = [&](bool ok) { return (bool)__all_sync(0xffffffffu, ok); };
      auto wait = [&](uint64_t* bar, uint32_t parity) { return all(mbar_wait(bar, parity, abort, kTimeoutNs, a.status)); };
      auto next = [&](int& u) {
        if (!wait(&full[unit], phase)) return false;
        u = unit;
        if (++unit == kUnits) unit = 0, phase ^= 1;
        return true;
      };
      // S_m = Q K^T of the unit; the last scores of a part give its Q back
      auto scores = [&](int m, int q, int u, bool final) {
        tc_fence_after();
        const uint32_t qa = uniform(k_desc(smem_addr(sQ + q * F::kTile))), ka = uniform(k_desc(smem_addr(sKV + u * F::kTile)));
        const uint32_t d = uniform(tS + 128 * m);
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          const uint32_t off = (k / 4) * (16384 / 16) + (k % 4) * 2;
          mma_ss(d, qa + off, ka + off, idesc_s, k > 0, one);
        }
        commit(&s_full[m], one);
        commit(&empty[u], one);
        if (final) commit(&q_empty[q], one);
      };
      uint32_t q_phase = 0, free_phase = 1;  // q_phase: of the two buffers of Q, a bit each
      int filled = 0;        // parts with keys so far: their Q lies in buffer filled & 1
      // the first scores of a part, for the warpgroup m
      auto begin = [&](int m, int tiles) {
        const int q = filled & 1;
        int u;
        if (!wait(&q_full[q], q_phase >> q & 1) || !next(u)) return false;
        q_phase ^= 1u << q;
        ++filled;
        scores(m, q, u, tiles == 1);
        return true;
      };
      bool ok = true, begun = false;  // begun: the part's first scores were issued ahead of the last part's sums
      for (int k = 0; ok; ++k) {
        if (!(ok = wait(&it_full[k % kItems], k / kItems & 1))) break;
        const int kind = items[k % kItems].kind, lo = items[k % kItems].lo, hi = items[k % kItems].hi, keys = items[k % kItems].m;
        __syncwarp();
        if (lane == 0) mbar_arrive(&it_empty[k % kItems]);
        if (kind == 0) break;
        if (lo == hi) continue;
        if (!begun && !(ok = begin(turn, hi - lo))) break;
        begun = false;
        const int q = (filled - 1) & 1;
        for (int j = hi - 1; j >= lo && ok; --j) {
          const uint32_t m = turn;
          turn ^= 1;
          int uv;
          if (j > lo) {  // the other warpgroup's scores go ahead of this one's sums
            int uk;
            if (!(ok = next(uk))) break;
            scores(m ^ 1, q, uk, j - 1 == lo);
          }
          if (!(ok = next(uv))) break;
          if ((j + 1) * BK > keys) clear_rows(sKV + uv * F::kTile, F::kSlabs, BK, keys - j * BK, lane);
          if (j == lo && all(mbar_try_wait(&it_full[(k + 1) % kItems], (k + 1) / kItems & 1))) {
            // so do the next part's, where its keys are here already
            const Item& ahead = items[(k + 1) % kItems];
            if (ahead.kind && ahead.lo < ahead.hi && all(mbar_try_wait(&full[unit], phase))) {
              if (!(ok = begin(m ^ 1, ahead.hi - ahead.lo))) break;
              begun = true;
            }
          }
          if (!(ok = wait(&p_full[m], tile_phase >> m & 1))) break;
          tile_phase ^= 1u << m;
          // O of the part before has been read
          if (j == hi - 1) {
            if (!(ok = wait(o_free, free_phase))) break;
            free_phase ^= 1;
          }
          tc_fence_after();
          const uint32_t va = uniform(mn_desc(smem_addr(sKV + uv * F::kTile))), d = uniform(tO + DP * m), w = uniform(tS + 128 * m);
#pragma unroll
          for (int i = 0; i < BK / 16; ++i)  // O_m += P_m V
            mma_ts(d, w + 8 * i, va + (2048 / 16) * i, idesc_o, j < hi - 2 || i > 0, one);
          commit(&empty[uv], one);
          if (j == lo) commit(o_full, one);
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
    // ===================== softmax of every second tile, a thread a row; output, a thread half a row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const uint32_t m = warp / 4 - 1, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lanes = quarter * 32 << 16;
    const uint32_t my_s = tS + 128 * m + lanes;
    auto all = [&](bool ok) { return (bool)__all_sync(0xffffffffu, ok); };
    uint32_t tile_phase = 0, part_phase = 0, both_phase = 0, turn = 0;
    auto both_sync = [&] {  // of both warpgroups; false: given up
      __syncwarp();
      if (lane == 0) mbar_arrive(both);
      const bool ok = all(mbar_wait(both, both_phase, abort, kTimeoutNs, a.status));
      both_phase ^= 1;
      return ok;
    };
#pragma unroll 1
    for (int k = 0;; ++k) {
      if (!all(mbar_wait(&it_full[k % kItems], k / kItems & 1, abort, kTimeoutNs, a.status))) break;
      const Item& it = items[k % kItems];
      if (it.kind == 0) break;
      const int lo = it.lo, hi = it.hi;
      Running w;
      bool ok = true;
      {
        const Seq s{it.q - it.i0, it.n, it.k0, it.m};
        const int seen = visible(a, s, it.i0 + row / p.pack), least = visible(a, s, it.i0);
#pragma unroll 1
        for (int j = hi - 1 - (turn ^ m); j >= lo; j -= 2) {
          if (!(ok = all(mbar_wait(&s_full[m], tile_phase, abort, kTimeoutNs, a.status)))) break;
          tile_phase ^= 1;
          tc_fence_after();
          softmax_step<DP>(my_s, tO + DP * m + lanes, p.c, (j + 1) * BK > least ? seen - j * BK : BK, j < hi - 2, w);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[m]);
        }
      }
      if (!all(ok)) break;
      turn ^= (hi - lo) & 1;
      sStat[k & 1][m][row] = make_float2(w.top, w.sum0 + w.sum1);
      if (!both_sync()) break;
      const float2 s0 = sStat[k & 1][0][row], s1 = sStat[k & 1][1][row];
      const float top = fmaxf(s0.x, s1.x);
      // a warpgroup without a tile, or without a visible key, has the weight 0, and its O is not looked at
      const float w0 = s0.y == 0.0f ? 0.0f : ex2((s0.x - top) * p.c), w1 = s1.y == 0.0f ? 0.0f : ex2((s1.x - top) * p.c);
      const float sum = w0 * s0.y + w1 * s1.y;
      if (lo < hi) {
        if (!all(mbar_wait(o_full, part_phase, abort, kTimeoutNs, a.status))) break;
        part_phase ^= 1;
        tc_fence_after();
      }
      const int i = it.i0 + row / p.pack, h = it.h0 + row % p.pack, q0 = it.q - it.i0;
      const bool live = i < it.n, cut = it.kind == 2;
      const float f = cut ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.o) + (int64_t)(q0 + i) * a.ld_o + (int64_t)h * a.D;
      float* part = p.part + ((int64_t)it.slot * 128 + row) * DP;
#pragma unroll 1
      for (int col = m * (DP / 2); col < (m + 1) * (DP / 2); col += 16) {
        uint32_t x[16], y[16];
        if (lo < hi) {
          tmem_ld16(tO + lanes + col, x);
          tmem_ld16(tO + DP + lanes + col, y);
          tmem_ld_wait();
        }
        float o[16];
#pragma unroll
        for (int l = 0; l < 16; ++l)
          o[l] = f * ((s0.y == 0.0f ? 0.0f : w0 * __uint_as_float(x[l])) + (s1.y == 0.0f ? 0.0f : w1 * __uint_as_float(y[l])));
        if (live && cut) {
#pragma unroll
          for (int l = 0; l < 16; l += 4) *reinterpret_cast<float4*>(part + col + l) = make_float4(o[l], o[l + 1], o[l + 2], o[l + 3]);
        } else if (live) {
#pragma unroll
          for (int l = 0; l < 16; l += 8)
            if (col + l < a.D)
              *reinterpret_cast<uint4*>(dst + col + l) = make_uint4(pack2(o[l], o[l + 1]), pack2(o[l + 2], o[l + 3]),
                                                                    pack2(o[l + 4], o[l + 5]), pack2(o[l + 6], o[l + 7]));
        }
      }
      if (lo < hi) {  // O may be written again
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_free);
      }
      if (live && m == 0) {
        if (cut) p.stat[(int64_t)it.slot * 128 + row] = make_float2(top, sum);
        else a.lse[(int64_t)h * a.Tq + q0 + i] = sum == 0.0f ? -INFINITY : (top * p.c + log2f(sum)) * kLn2;
      }
      if (cut) {
        // whoever comes last puts the parts of the line together
        const int c0 = it.c0, parts = it.c1 - it.c0 + 1;
        __threadfence();
        if (!both_sync()) break;
        if (m == 0 && row == 0) {
          const bool last = atomicAdd(p.tickets + c0, 1u) == (uint32_t)parts - 1;
          if (last) p.tickets[c0] = 0;
          last_one = last;
        }
        if (!both_sync()) break;
        if (last_one) {
          __threadfence();
          // the line's first part is its CTA's last (place 1), the others are their CTAs' first (place 0)
          auto place = [&](int g) { return (int64_t)(2 * (c0 + g) + (g == 0)) * 128; };
          const int rows = min(per, it.n - it.i0) * p.pack, h_first = it.h0, i_first = it.i0;
          float2* sRow = sStat[k & 1][0];  // maximum and 1 / sum of every row; its last readers are past two meetings
          if (m == 0 && (int)row < rows) {
            float most = -INFINITY, total = 0.0f;
#pragma unroll 8
            for (int g = 0; g < parts; ++g) most = fmaxf(most, __ldcg(&p.stat[place(g) + row].x));
#pragma unroll 8
            for (int g = 0; g < parts; ++g) {
              const float2 st = __ldcg(&p.stat[place(g) + row]);
              if (st.y != 0.0f) total = fmaf(ex2((st.x - most) * p.c), st.y, total);
            }
            sRow[row] = make_float2(most, total == 0.0f ? 0.0f : 1.0f / total);
            a.lse[(int64_t)(h_first + row % p.pack) * a.Tq + q0 + i_first + row / p.pack] =
                total == 0.0f ? -INFINITY : (most * p.c + log2f(total)) * kLn2;
          }
          if (!both_sync()) break;
          for (int e = m * 128 + row; e < rows * (DP / 4); e += 256) {
            const int r = e / (DP / 4), d = e % (DP / 4) * 4;
            const float2 whole = sRow[r];
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (whole.y != 0.0f)
#pragma unroll 8
              for (int g = 0; g < parts; ++g) {
                const float x = __ldcg(&p.stat[place(g) + r].x);
                const float4 o = __ldcg(reinterpret_cast<const float4*>(p.part + (place(g) + r) * DP + d));
                const float weight = ex2((x - whole.x) * p.c);
                acc.x = fmaf(weight, o.x, acc.x);
                acc.y = fmaf(weight, o.y, acc.y);
                acc.z = fmaf(weight, o.z, acc.z);
                acc.w = fmaf(weight, o.w, acc.w);
              }
            if (d < a.D)
              *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + (int64_t)(q0 + i_first + r / p.pack) * a.ld_o +
                                        (int64_t)(h_first + r % p.pack) * a.D + d) =
                  make_uint2(pack2(acc.x * whole.y, acc.y * whole.y), pack2(acc.z * whole.y, acc.w * whole.y));
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&it_empty[k % kItems]);
    }
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int DP>
cudaError_t forward(const AttnArgs& a, const StreamSpace& w, cudaStream_t s) {
  const int pack = heads_packed(a.group);
  const StreamParams p{a, pack, a.Hq / pack, a.scale * kLog2e, 1.0 / stream_ctas(), w.tickets, w.stat, w.part};
  CUtensorMap q, k, v;
  if (!head_map(&q, a.q, a.Tq, a.Hq, a.D, a.ld_q, pack, 128 / pack)) return cudaErrorInvalidValue;
  if (a.Tk > 0) {
    if (!head_map(&k, a.k, a.Tk, a.Hkv, a.D, a.ld_k, 1, BK) || !head_map(&v, a.v, a.Tk, a.Hkv, a.D, a.ld_v, 1, BK))
      return cudaErrorInvalidValue;
  } else {
    k = v = q;  // no key is loaded
  }
  static Once once;
  const cudaError_t e = allow_smem(once, attn_stream_kernel<DP>, Ring<DP>::kBytes);
  if (e != cudaSuccess) return e;
  attn_stream_kernel<DP><<<stream_ctas(), kThreads, Ring<DP>::kBytes, s>>>(q, k, v, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_stream(const AttnArgs& a, const StreamSpace& w, cudaStream_t s) {
  return a.D <= 64 ? forward<64>(a, w, s) : forward<128>(a, w, s);
}

}  // namespace attn
}  // namespace moe
