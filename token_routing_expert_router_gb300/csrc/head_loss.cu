// The vocabulary head: softmax cross entropy of tokens x [T, H] against w [V, H], and its
// gradients, without ever holding the logits z = x w^T [T, V]:
//   lse_t = log sum_v exp z_tv;  loss_t = lse_t - z_{t,target}
//   dz_tv = (exp(z_tv - lse_t) - [v = target_t]) dloss_t;  dx = dz w;  dw = dz^T x
// Forward: one GEMM whose epilogue keeps, per token and half tile of columns, the running
// maximum and the sum of exponentials against it, and the target's logit; join_kernel puts the
// halves together. Backward: piece after piece of the vocabulary, the GEMM is run again and its
// epilogue turns the logits into dz (bf16, the operand of the next products), then
// dx += dz w_piece and dw_piece = dz^T x. Memory beside the inputs and outputs: one piece of dz
// and 16 bytes per token and tile.
//
// bf16 with H a multiple of 8 runs on the tensor cores (tcgen05): warp 0 feeds a ring of
// shared-memory stages by TMA, warp 1 issues the MMAs into two TMEM accumulators, warps 2-9
// are the epilogue of one accumulator while the other fills. Tiles are 256 x 256 on a CTA pair,
// or 128 x 128 on one CTA for up to 128 tokens, where reading w is all the time there is and
// smaller tiles spread it more evenly over the SMs. Edges need no special case in the operands:
// the TMA fills zeros past the last row and column. fp32, and widths of other multiples, take
// exact fp32 FMA tiles (simt_kernel), with dz kept in fp32.
#include <cudaTypedefs.h>

#include <algorithm>

#include "step.cuh"
#include "tc_common.cuh"

namespace moe {
namespace tc {

bool make_tmap(CUtensorMap* m, const void* base, CUtensorMapDataType dt, int esize, uint64_t rows, uint64_t cols,
               uint32_t box_rows, uint32_t box_cols);

namespace {

constexpr int BM = 128, BK = 64;  // rows of A per CTA; bf16 elements of a K stage (128 bytes)
constexpr int kThreads = 320;
constexpr int kEpiWarps = 8;
constexpr int kABytes = BM * BK * 2;
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kRun = 16;  // K stages (1024 elements) added by the tensor core in one go

enum Mode { STATS = 0, DLOGITS = 1, DX = 2, DW = 3 };

struct HeadParams {
  int M, N;            // rows and columns of the product that exist
  int m_tiles, n_tiles, kblocks;
  int direct;          // DX: the first `direct` tiles are whole; the K of each further one is
  int splits;          //   split over `splits` units, which write fp32 tiles to `slices`
  float* slices;       //   [tile - direct][split][TM][BN]
  int b_row0;          // first vocabulary row of the piece (STATS: 0)
  int V;
  const int32_t* target;
  // STATS: (max, sum) per token and half tile [2 n_tiles][T], and the target's logit [T]
  float2* part;
  float* target_logit;
  // DLOGITS
  const float *lse, *dloss;
  // outputs of the other modes, and their row length in elements
  void* out;
  int64_t ldo;
  int out_f32;         // DX, DW: fp32 output (else bf16)
  int add;             // DX: added to what out holds (a later piece of the vocabulary)
  const float* factor; // DX, DW: every value is multiplied by it (the mean's 1 / count), or NULL
  DeviceStatus* status;
  uint64_t timeout_ns;
};

template <int CG, int BN>
struct HeadSmem {
  static constexpr int kBBytes = (BN / CG) * BK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = 6;
  static constexpr size_t kBytes = 1024 + (size_t)kStages * kStageBytes + 256 + kEpiWarps * 2048;
};

// MN-major operand: 64-element MN blocks of the stage's 64 K rows (8 KB each, 128-byte swizzle).
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(8192u >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// 2^x (the PTX instruction, relative error 2^-22).
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// A row's next 64 bytes into the staging buffer: 32 columns as bf16, or 16 as fp32.
__device__ __forceinline__ void stage_bf16(uint8_t* stage, int lane, const float* v) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    stage_piece(stage, lane, q, make_uint4(pack2(v[8 * q], v[8 * q + 1]), pack2(v[8 * q + 2], v[8 * q + 3]),
                                           pack2(v[8 * q + 4], v[8 * q + 5]), pack2(v[8 * q + 6], v[8 * q + 7])));
}
__device__ __forceinline__ void stage_f32(uint8_t* stage, int lane, const float* v) {
#pragma unroll
  for (int q = 0; q < 4; ++q)
    stage_piece(stage, lane, q, make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]),
                                           __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3])));
}

// flush_rows_64B with a column bound: the 16-byte pieces c >= pieces are left out.
__device__ __forceinline__ void flush_edge(uint8_t* stage, int lane, uint8_t* base, int64_t stride, int live, int pieces,
                                           bool add) {
  __syncwarp();
  const int c = lane & 3;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int row = 8 * j + (lane >> 2);
    uint4 v = *reinterpret_cast<const uint4*>(stage + row * 64 + 16 * (c ^ ((row >> 1) & 3)));
    if (row < live && c < pieces) {
      uint4* dst = reinterpret_cast<uint4*>(base + row * stride + 16 * c);
      if (add) {
        const uint4 o = *dst;
        v = make_uint4(__float_as_uint(__uint_as_float(v.x) + __uint_as_float(o.x)),
                       __float_as_uint(__uint_as_float(v.y) + __uint_as_float(o.y)),
                       __float_as_uint(__uint_as_float(v.z) + __uint_as_float(o.z)),
                       __float_as_uint(__uint_as_float(v.w) + __uint_as_float(o.w)));
      }
      *dst = v;
    }
  }
  __syncwarp();
}

struct HeadTile {
  int mb, nb, slice, kb0, kb1;  // slice: -1, or the tile's place in `slices`
};

// Which tiles run side by side, and so share operands through L2. Logits and dx: the m tiles
// (a tile of w is read once, x or a K slice of dz stays in L2). dw: the n tiles (the columns of
// dz are read once, x stays in L2; with the m tiles first, dz came from DRAM once per n tile,
// 4.2 GB for 4096 x 4096 x 32000, and the product took 700 us).
template <int MODE>
__device__ __forceinline__ HeadTile head_tile(int unit_index, const HeadParams& p) {
  HeadTile t;
  int tile = unit_index;
  t.slice = -1;
  t.kb0 = 0;
  t.kb1 = p.kblocks;
  if (MODE == DX && unit_index >= p.direct) {
    t.slice = unit_index - p.direct;
    const int split = t.slice % p.splits;
    tile = p.direct + t.slice / p.splits;
    t.kb0 = (int)((int64_t)p.kblocks * split / p.splits);
    t.kb1 = (int)((int64_t)p.kblocks * (split + 1) / p.splits);
  }
  if (MODE == DW) {
    t.mb = tile / p.n_tiles;
    t.nb = tile - t.mb * p.n_tiles;
  } else {
    t.nb = tile / p.m_tiles;
    t.mb = tile - t.nb * p.m_tiles;
  }
  return t;
}

// Work units of a launch.
__host__ __device__ __forceinline__ int head_units(const HeadParams& p) {
  return p.direct + (p.m_tiles * p.n_tiles - p.direct) * p.splits;
}

template <int MODE, int CG, int BN>
__global__ void __launch_bounds__(kThreads, 1)
    head_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const HeadParams p) {
  using S = HeadSmem<CG, BN>;
  constexpr int kStages = S::kStages, kBBytes = S::kBBytes, kStageBytes = S::kStageBytes;
  constexpr int TM = BM * CG;
  constexpr int kTmemCols = 2 * BN;
  constexpr bool kAmn = MODE == DW;                 // A read MN-major (its rows are the K index)
  constexpr bool kBmn = MODE == DX || MODE == DW;   // the same for B
  constexpr int kBoxes = (BN / CG) / 64;
  extern __shared__ uint8_t smem_raw[];
  let_next_begin();  // the small kernel that joins the tiles' results
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + kStages * kABytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);
  uint64_t* full = bars;
  uint64_t* empty = bars + kStages;
  uint64_t* tfull = bars + 2 * kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint8_t* sEpi = reinterpret_cast<uint8_t*>(bars + 32);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_ctarank() : 0;
  const bool leader = rank == 0;
  const int unit = blockIdx.x / CG, nunits = gridDim.x / CG;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], kEpiWarps * CG);
    }
    mbar_init(drain, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) tmem_alloc_cg<CG>(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int total_tiles = head_units(p);
  // The loss's logits are added up in runs of kRun K stages: each run has its own accumulator,
  // and the epilogue adds the runs in fp32. The tensor core's own additions truncate: over 4096
  // elements in one go the loss was off by 3.4e-6 of its size, in runs of 1024 by 6e-7. dz is
  // rounded to bf16, where one go is good enough.
  constexpr bool kRuns = MODE == STATS;
  auto runs_of = [&](const HeadTile& t) { return kRuns ? (t.kb1 - t.kb0 + kRun - 1) / kRun : 1; };
  auto run_end = [&](const HeadTile& t, int run) { return kRuns ? min(t.kb1, (run + 1) * kRun) : t.kb1; };

  if (warp == 0) {
    // ======================= TMA producer (each CTA loads its own rows of A and its part of B)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int64_t issued = 0;
      bool ok = true;
      for (int tile = unit; tile < total_tiles && ok; tile += nunits) {
        const HeadTile t = head_tile<MODE>(tile, p);
        const int am = t.mb * TM + (int)rank * BM, bn = t.nb * BN + (int)rank * (BN / CG);
        for (int kb = t.kb0; kb < t.kb1; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1, abort, p.timeout_ns, p.status)) { ok = false; break; }
          uint8_t* a_dst = sA + stage * kABytes;
          uint8_t* b_dst = sB + stage * kBBytes;
          uint32_t bar = 0;
          if constexpr (CG == 1) {
            mbar_arrive_expect_tx(&full[stage], kStageBytes);
          } else {
            if (leader) mbar_arrive_expect_tx(&full[stage], 2 * kStageBytes);
            bar = mapa_shared(smem_addr(&full[stage]), 0);
          }
          auto load = [&](const CUtensorMap* m, uint8_t* dst, int x, int y) {
            if constexpr (CG == 1) tma_load_2d(m, dst, &full[stage], x, y);
            else tma_load_2d_pair(m, dst, bar, x, y);
          };
          if constexpr (kAmn) {
            load(&tmA, a_dst, am, kb * BK);
            load(&tmA, a_dst + 8192, am + 64, kb * BK);
          } else {
            load(&tmA, a_dst, kb * BK, am);
          }
          if constexpr (kBmn) {
            const int y = (MODE == DX ? p.b_row0 : 0) + kb * BK;
#pragma unroll
            for (int j = 0; j < kBoxes; ++j) load(&tmB, b_dst + 8192 * j, bn + 64 * j, y);
          } else {
            load(&tmB, b_dst, kb * BK, p.b_row0 + bn);
          }
          ++issued;
          if (++stage == kStages) { stage = 0; phase ^= 1; }
        }
      }
      const int used = issued < kStages ? (int)issued : kStages;
      for (int i = 0; i < used; ++i) {
        const int s = (stage - 1 - i + 2 * kStages) % kStages;
        const uint32_t ph = (stage - 1 - i < 0) ? (phase ^ 1) : phase;
        if (ok) ok = mbar_wait(&empty[s], ph, abort, p.timeout_ns, p.status);
        if (!ok && (CG == 1 || leader)) mbar_wait_drain(&full[s], ph, p.timeout_ns, p.status);
      }
    }
  } else if (warp == 1) {
    // ======================= MMA issuer (the leader of a pair issues for both CTAs)
    if (lane == 0 && leader) {
      constexpr uint32_t idesc = idesc_make(1, TM, BN) | ((kAmn ? 1u : 0u) << 15) | ((kBmn ? 1u : 0u) << 16);
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (int tile = unit; tile < total_tiles && ok; tile += nunits) {
        const HeadTile t = head_tile<MODE>(tile, p);
        int kb = t.kb0;
        for (int run = 0; run < runs_of(t) && ok; ++run) {
          if (!mbar_wait(&tempty[acc], acc_phase ^ 1, abort, p.timeout_ns, p.status)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + acc * BN;
          const int first = kb, end = run_end(t, run);
          for (; kb < end; ++kb) {
            if (!mbar_wait(&full[stage], phase, abort, p.timeout_ns, p.status)) { ok = false; break; }
            tc_fence_after();
            const uint32_t a_addr = smem_addr(sA + stage * kABytes);
            const uint32_t b_addr = smem_addr(sB + stage * kBBytes);
#pragma unroll
            for (int k = 0; k < BK / 16; ++k) {
              const uint64_t ad = kAmn ? desc_mn(a_addr + k * 2048) : desc_k_sw128(a_addr + k * 32);
              const uint64_t bd = kBmn ? desc_mn(b_addr + k * 2048) : desc_k_sw128(b_addr + k * 32);
              const uint32_t accumulate = kb > first || k > 0;
              if constexpr (CG == 1) mma_bf16(d_tmem, ad, bd, idesc, accumulate);
              else mma_bf16_pair(d_tmem, ad, bd, idesc, accumulate);
            }
            if constexpr (CG == 1) mma_commit(&empty[stage]);
            else mma_commit_pair(&empty[stage], 0x3);
            if (++stage == kStages) { stage = 0; phase ^= 1; }
          }
          if (!ok) break;
          if constexpr (CG == 1) mma_commit(&tfull[acc]);
          else mma_commit_pair(&tfull[acc], 0x3);
          if (++acc == 2) { acc = 0; acc_phase ^= 1; }
        }
      }
      if constexpr (CG == 1) mma_commit(drain);
      else mma_commit_pair(drain, 0x3);
      mbar_wait_drain(drain, 0, p.timeout_ns, p.status);
    } else if (lane == 0 && CG == 2) {
      // the pair's MMAs write this CTA's TMEM and read its shared memory: stay until done
      mbar_wait_drain(drain, 0, p.timeout_ns, p.status);
    }
  } else {
    // ======================= epilogue (warps 2..9; TMEM lane quarter = warp % 4, half the columns each)
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    constexpr int kCols = BN / 2;
    const int cbase = half * kCols;
    const int wrow = (int)rank * BM + quarter * 32;
    uint8_t* stage = sEpi + (warp - 2) * 2048;
    const uint32_t tempty_leader = CG == 2 ? mapa_shared(smem_addr(&tempty[0]), 0) : 0;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int tile = unit; tile < total_tiles; tile += nunits) {
      const HeadTile t = head_tile<MODE>(tile, p);
      const int row0 = t.mb * TM + wrow, row = row0 + lane;  // the thread's row of the product
      const int col0 = t.nb * BN + cbase;                    // the warp's first column
      const bool live = row < p.M;
      auto wait_full = [&] {
        const bool ok = mbar_wait(&tfull[acc], acc_phase, abort, p.timeout_ns, p.status);
        tc_fence_after();
        return __all_sync(0xffffffffu, ok);
      };
      auto release = [&] {  // this accumulator may be written again
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (CG == 2 && !leader) mbar_arrive_cluster_relaxed(tempty_leader + acc * 8);
          else mbar_arrive_relaxed(&tempty[acc]);
        }
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      };
      const uint32_t t_lane = tmem_base + ((uint32_t)(quarter * 32) << 16) + cbase;

      if constexpr (MODE == STATS) {
        // this row's half of the tile's columns, out of TMEM before anything is made of it
        uint32_t zr[kCols / 32][32];
        const int runs = runs_of(t);
        bool ok = true;
        for (int run = 0; run < runs; ++run) {
          if (!(ok = wait_full())) break;
          const uint32_t t_row = t_lane + acc * BN;
          if (run == 0) {
#pragma unroll
            for (int c = 0; c < kCols / 32; ++c) tmem_ld32(t_row + 32 * c, zr[c]);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int c = 0; c < kCols; c += 16) {
              uint32_t v[16];
              tmem_ld16(t_row + c, v);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i)
                zr[c / 32][c % 32 + i] = __float_as_uint(__uint_as_float(zr[c / 32][c % 32 + i]) + __uint_as_float(v[i]));
            }
          }
          release();
        }
        if (!ok) break;
        auto z = [&](int i) { return __uint_as_float(zr[i / 32][i % 32]); };
        const int cols = p.N - col0;  // columns from here on that exist
        const int tgt = live ? __ldg(p.target + row) : -1;
        if (tgt >= col0 && tgt < min(col0 + kCols, p.N)) {
#pragma unroll
          for (int i = 0; i < kCols; ++i)
            if (col0 + i == tgt) p.target_logit[row] = z(i);
        }
        float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
        for (int i = 0; i < kCols; i += 2) {
          if (cols < kCols) {
            if (i >= cols) zr[i / 32][i % 32] = __float_as_uint(-INFINITY);
            if (i + 1 >= cols) zr[i / 32][i % 32 + 1] = __float_as_uint(-INFINITY);
          }
          m0 = fmaxf(m0, z(i));
          m1 = fmaxf(m1, z(i + 1));
        }
        const float mx = fmaxf(m0, m1) * kLog2e;
        const float base = mx == -INFINITY ? 0.0f : mx;
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int i = 0; i < kCols; i += 2) {
          s0 += ex2(fmaf(z(i), kLog2e, -base));
          s1 += ex2(fmaf(z(i + 1), kLog2e, -base));
        }
        if (live) p.part[(int64_t)(2 * t.nb + half) * p.M + row] = make_float2(mx, s0 + s1);
      } else {
        int tgt = -1;
        bool counts = false;
        float lse2 = 0.0f, g = 0.0f;
        if constexpr (MODE == DLOGITS) {
          if (live) tgt = __ldg(p.target + row);
          counts = tgt >= 0 && tgt < p.V;
          if (counts) {
            lse2 = __ldg(p.lse + row) * kLog2e;
            // the gradient of the mean: its factor 1 / count is left to the two products
            g = p.dloss ? __ldg(p.dloss + row) : 1.0f;
          }
        } else {
          g = p.factor ? __ldg(p.factor) : 1.0f;
        }
        if (!wait_full()) break;
        const bool none = MODE == DX && t.kb0 == t.kb1;  // a split without K stages: nothing in the accumulator
        const uint32_t t_row = t_lane + acc * BN;
        uint32_t nxt[32];
        tmem_ld32(t_row, nxt);
#pragma unroll 1
        for (int c0 = 0; c0 < kCols; c0 += 32) {
          float v[32];
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(nxt[i]);
          if (c0 + 32 < kCols) tmem_ld32(t_row + c0 + 32, nxt);  // next chunk in flight
          const int cc = col0 + c0;   // first column of the chunk
          const int cols = p.N - cc;  // columns from there on that exist
          if constexpr (MODE == DLOGITS) {
            const int at = tgt - p.b_row0 - cc;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              v[i] = ex2(fmaf(v[i], kLog2e, -lse2));
              if (i == at) v[i] -= 1.0f;
              v[i] = counts && i < cols ? v[i] * g : 0.0f;
            }
            stage_bf16(stage, lane, v);
            // columns past the vocabulary are written too, as zeros: they are K rows of the next products
            flush_rows_64B(stage, lane, static_cast<uint8_t*>(p.out) + ((int64_t)row0 * p.ldo + cc) * 2, p.ldo * 2,
                           p.M - row0);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = none ? 0.0f : v[i] * g;
            if (MODE == DX && t.slice >= 0) {
              uint8_t* out = reinterpret_cast<uint8_t*>(p.slices + ((int64_t)t.slice * TM + wrow) * BN + cbase + c0);
#pragma unroll
              for (int h = 0; h < 32; h += 16) {
                stage_f32(stage, lane, v + h);
                flush_rows_64B(stage, lane, out + 4 * h, BN * 4, 32);
              }
            } else if (p.out_f32) {
              uint8_t* out = static_cast<uint8_t*>(p.out) + ((int64_t)row0 * p.ldo + cc) * 4;
#pragma unroll
              for (int h = 0; h < 32; h += 16) {
                stage_f32(stage, lane, v + h);
                flush_edge(stage, lane, out + 4 * h, p.ldo * 4, p.M - row0, (cols - h) / 4, MODE == DX && p.add);
              }
            } else {
              stage_bf16(stage, lane, v);
              flush_edge(stage, lane, static_cast<uint8_t*>(p.out) + ((int64_t)row0 * p.ldo + cc) * 2, p.ldo * 2,
                         p.M - row0, cols / 8, false);
            }
          }
        }
        release();
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();  // neither CTA leaves while the pair still uses it
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc_cg<CG>(tmem_base, kTmemCols);
  }
}

bool bf16_box(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  return make_tmap(m, base, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, rows, cols, box_rows, 64);
}

template <int MODE, int CG, int BN>
cudaError_t launch_gemm(const CUtensorMap& a, const CUtensorMap& b, const HeadParams& p, cudaStream_t s) {
  auto kern = head_gemm_kernel<MODE, CG, BN>;
  const size_t smem = HeadSmem<CG, BN>::kBytes;
  static bool attr_set = false;  // per instantiation
  if (!attr_set) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    attr_set = true;
  }
  const int64_t tiles = head_units(p);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(CG * (num_sms() / CG));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 2 ? 1 : 0;
  int units = num_sms() / CG;
  if (CG == 2) {  // a persistent grid must be resident all at once: no more pairs than fit together
    static int max_pairs = 0;
    if (!max_pairs) {
      cudaError_t e = cudaOccupancyMaxActiveClusters(&max_pairs, kern, &cfg);
      if (e != cudaSuccess || max_pairs <= 0) return e != cudaSuccess ? e : cudaErrorInvalidConfiguration;
    }
    units = std::min(units, max_pairs);
  }
  cfg.gridDim = dim3((unsigned)(CG * std::min<int64_t>(units, tiles)));
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a, b, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Up to 128 tokens: one 128-row tile, single CTAs. Else 256-row tiles on CTA pairs.
bool small_tokens(int T) { return T <= BM; }

HeadParams base_params(int64_t M, int64_t N, int64_t K, int tm, int tn, DeviceStatus* st) {
  HeadParams p{};
  p.M = (int)M;
  p.N = (int)N;
  p.m_tiles = (int)ceil_div(M, tm);
  p.n_tiles = (int)ceil_div(N, tn);
  p.kblocks = (int)ceil_div(K, BK);
  p.direct = p.m_tiles * p.n_tiles;
  p.splits = 1;
  p.status = st;
  p.timeout_ns = kTimeoutNs;
  return p;
}

// dx of the tiles whose K was split: the sum of a tile's slices in order, written or added.
template <typename T>
__global__ void __launch_bounds__(256) join_slices_kernel(const HeadParams p, int tm, int tn, T* out) {
  after_previous();
  const int tile = p.direct + blockIdx.y, e = (blockIdx.x * 256 + threadIdx.x) * 4;  // 4 columns each
  const int nb = tile / p.m_tiles, mb = tile - nb * p.m_tiles;
  const int row = mb * tm + e / tn, col = nb * tn + e % tn;
  if (row >= p.M || col >= p.N) return;
  const float* s = p.slices + (int64_t)blockIdx.y * p.splits * tm * tn + e;
  float4 v = make_float4(0, 0, 0, 0);
#pragma unroll 4
  for (int k = 0; k < p.splits; ++k) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(s + (int64_t)k * tm * tn));
    v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
  }
  T* o = out + (int64_t)row * p.ldo + col;
  if constexpr (sizeof(T) == 4) {
    float4* d = reinterpret_cast<float4*>(o);
    if (p.add) {
      const float4 a = *d;
      v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
    }
    *d = v;
  } else {
    *reinterpret_cast<uint2*>(o) = make_uint2(pack2(v.x, v.y), pack2(v.z, v.w));
  }
}

}  // namespace

// Columns of a tile of the logits, for the number of (max, sum) halves.
int head_tile_cols(int T) { return small_tokens(T) ? 128 : 256; }

// The input gradient's tiles rarely fill whole rounds of the SMs (4096 x 4096 is 256 tiles of
// 256 x 256 on 76 CTA pairs: 3.37 rounds, so 4). The tiles of the last round are therefore
// split along K, by the number of ways that takes least time: rounds of stages of 64 at 0.14 us
// each against the slices' traffic at 0.08 us a tile, and the launch that adds them.
HeadSplit head_split(int64_t T, int64_t H, int64_t rows) {
  const bool small = small_tokens((int)std::min<int64_t>(T, INT32_MAX));
  const int tm = small ? BM : 2 * BM, tn = small ? 128 : 256, units = small ? 152 : 76;
  const int64_t tiles = ceil_div(T, tm) * ceil_div(H, tn), kblocks = ceil_div(rows, BK);
  HeadSplit best{tiles, 1, 0};
  const int64_t tail = tiles % units;
  double least = (tail ? 1.0 : 0.0) * kblocks * 0.14;
  for (int s = 2; s <= 32 && tail && s * 4 <= kblocks; ++s) {
    const double t = (double)ceil_div(tail * s, units) * ceil_div(kblocks, s) * 0.14 +
                     tail * s * 0.08 * (small ? 0.25 : 1.0) + 4.0;
    if (t < least) least = t, best = {tiles - tail, s, (size_t)(tail * s) * tm * tn * 4};
  }
  return best;
}

cudaError_t launch_head_stats(const moe_head_config_t& c, const void* x, const void* w, const int32_t* target,
                              float2* part, float* target_logit, DeviceStatus* st, cudaStream_t s) {
  const bool small = small_tokens(c.T);
  HeadParams p = base_params(c.T, c.V, c.H, small ? BM : 2 * BM, head_tile_cols(c.T), st);
  p.V = c.V;
  p.target = target;
  p.part = part;
  p.target_logit = target_logit;
  CUtensorMap a, b;
  if (!bf16_box(&a, x, c.T, c.H, BM) || !bf16_box(&b, w, c.V, c.H, 128)) return cudaErrorInvalidValue;
  return small ? launch_gemm<STATS, 1, 128>(a, b, p, s) : launch_gemm<STATS, 2, 256>(a, b, p, s);
}

// dz of the vocabulary rows [v0, v0 + rows) -> dl [T, ld] bf16; then dx and dw of the piece.
cudaError_t launch_head_piece(const moe_head_config_t& c, const void* x, const void* w, const int32_t* target,
                              const float* lse, const float* dloss, const float* mean, int64_t v0, int rows, void* dl,
                              int ld, void* dx, const HeadSplit& split, float* slices, bool dx_f32, bool add, void* dw,
                              DeviceStatus* st, cudaStream_t s) {
  const bool small = small_tokens(c.T);
  const int tm = small ? BM : 2 * BM, tn = head_tile_cols(c.T);
  CUtensorMap a, b;
  HeadParams p = base_params(c.T, rows, c.H, tm, tn, st);
  p.V = c.V;
  p.b_row0 = (int)v0;
  p.target = target;
  p.lse = lse;
  p.dloss = dloss;
  p.out = dl;
  p.ldo = ld;
  if (!bf16_box(&a, x, c.T, c.H, BM) || !bf16_box(&b, w, c.V, c.H, 128)) return cudaErrorInvalidValue;
  cudaError_t e = small ? launch_gemm<DLOGITS, 1, 128>(a, b, p, s) : launch_gemm<DLOGITS, 2, 256>(a, b, p, s);
  if (e != cudaSuccess) return e;
  if (dx) {  // M = T, N = H, K = the piece's vocabulary rows
    p = base_params(c.T, c.H, rows, tm, tn, st);
    p.b_row0 = (int)v0;
    p.direct = (int)split.direct;
    p.splits = split.splits;
    p.slices = slices;
    p.out = dx;
    p.ldo = c.H;
    p.out_f32 = dx_f32;
    p.add = add;
    p.factor = mean ? mean + 1 : nullptr;
    if (!bf16_box(&a, dl, c.T, ld, BM) || !bf16_box(&b, w, c.V, c.H, 64)) return cudaErrorInvalidValue;
    e = small ? launch_gemm<DX, 1, 128>(a, b, p, s) : launch_gemm<DX, 2, 256>(a, b, p, s);
    if (e != cudaSuccess) return e;
    if (split.splits > 1) {
      const dim3 grid((unsigned)(tm * tn / 1024), (unsigned)(p.m_tiles * p.n_tiles - p.direct));
      e = dx_f32 ? launch_after(join_slices_kernel<float>, grid, 256, s, p, tm, tn, static_cast<float*>(dx))
                 : launch_after(join_slices_kernel<__nv_bfloat16>, grid, 256, s, p, tm, tn, static_cast<__nv_bfloat16*>(dx));
      if (e != cudaSuccess) return e;
    }
  }
  if (dw) {  // M = the piece's vocabulary rows, N = H, K = T
    p = base_params(rows, c.H, c.T, 2 * BM, 256, st);
    p.out_f32 = c.grad_dtype == MOE_DTYPE_F32;
    p.out = static_cast<uint8_t*>(dw) + v0 * c.H * (p.out_f32 ? 4 : 2);
    p.ldo = c.H;
    p.factor = mean ? mean + 1 : nullptr;
    if (!bf16_box(&a, dl, c.T, ld, 64) || !bf16_box(&b, x, c.T, c.H, 64)) return cudaErrorInvalidValue;
    e = launch_gemm<DW, 2, 256>(a, b, p, s);
  }
  return e;
}

}  // namespace tc

namespace {

// ---- exact fp32 tiles of ST x ST outputs, K steps of 16, 256 threads with (ST / 16)^2 outputs
// each. ST = 64 is for products whose 128-tiles would leave SMs without two blocks (256 x 128 x
// 5003: 35 us for 80 blocks of 128 x 128). Rows go in pairs through fma.f32x2 (each half rounded
// on its own, as fmaf): with one FMA per instruction and two warps per scheduler the tiles were
// bound by issue (64 x 64 by 128 threads: 17 us).
constexpr int SK = 16;

struct SimtParams {
  int M, N, K;
  int splits, k_split;         // DX: K splits of k_split (a multiple of SK) each
  const void *A, *B;           // operand element (row, k) at row * r + k * k
  int64_t a_row, a_k, b_row, b_k;
  int a_f32, b_f32;            // element types (else bf16)
  int vec;                     // rows of both operands begin on multiples of 4 elements
  const int32_t* target;
  float2* part;
  float* target_logit;
  const float *lse, *dloss, *mean;
  int v0, V;
  void* out;
  int64_t ldo;
  int out_f32, add;
};

__device__ __forceinline__ float load_elem(const void* p, int64_t at, int f32) {
  return f32 ? static_cast<const float*>(p)[at] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at]);
}
__device__ __forceinline__ float4 load_elem4(const void* p, int64_t at, int f32) {
  if (f32) return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
  const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + at);
  return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                     __uint_as_float(v.y & 0xffff0000u));
}

enum { S_STATS = 0, S_DLOGITS = 1, S_STORE = 2 };

template <int MODE, int ST>
__global__ void __launch_bounds__(256) simt_kernel(const SimtParams p) {
  constexpr int TM = ST / 16, TN = ST / 16, LD = ST + 4;
  constexpr int kLoads = ST * SK / 4 / 256;  // of four elements per thread, operand and step
  let_next_begin();
  after_previous();
  __shared__ __align__(16) float sa[2][SK][LD], sb[2][SK][LD];
  const int m0 = blockIdx.x * ST, n0 = blockIdx.y * ST;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int k_lo = blockIdx.z * p.k_split, k_hi = min(p.K, k_lo + p.k_split);
  float2 acc2[TM / 2][TN];  // rows 2 i and 2 i + 1
#pragma unroll
  for (int i = 0; i < TM / 2; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc2[i][j] = make_float2(0.0f, 0.0f);
  // Four elements per thread and load, along the operand's contiguous direction.
  auto place = [&](int64_t kstep, int i, int* r, int* k) {
    const int e = threadIdx.x + i * 256;
    if (kstep == 1) *r = e / (SK / 4), *k = e % (SK / 4) * 4;
    else *r = e % (ST / 4) * 4, *k = e / (ST / 4);
  };
  auto fetch = [&](float4 (&v)[kLoads], const void* src, int64_t rstep, int64_t kstep, int f32, int r0, int rows, int k0) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      int r, k;
      place(kstep, i, &r, &k);
      const int64_t at = (int64_t)(r0 + r) * rstep + (int64_t)(k0 + k) * kstep;
      const bool along_k = kstep == 1;
      const int left = along_k ? (r0 + r < rows ? k_hi - (k0 + k) : 0) : (k0 + k < k_hi ? rows - (r0 + r) : 0);
      if (p.vec && left >= 4) {
        v[i] = load_elem4(src, at, f32);
      } else {
        const int64_t step = along_k ? kstep : rstep;
        v[i].x = left > 0 ? load_elem(src, at, f32) : 0.0f;
        v[i].y = left > 1 ? load_elem(src, at + step, f32) : 0.0f;
        v[i].z = left > 2 ? load_elem(src, at + 2 * step, f32) : 0.0f;
        v[i].w = left > 3 ? load_elem(src, at + 3 * step, f32) : 0.0f;
      }
    }
  };
  auto keep = [&](float (*dst)[LD], const float4 (&v)[kLoads], int64_t kstep) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      int r, k;
      place(kstep, i, &r, &k);
      if (kstep == 1) {
        dst[k][r] = v[i].x, dst[k + 1][r] = v[i].y, dst[k + 2][r] = v[i].z, dst[k + 3][r] = v[i].w;
      } else {
        *reinterpret_cast<float4*>(&dst[k][r]) = v[i];
      }
    }
  };
  float4 va[kLoads], vb[kLoads];
  if (k_lo < k_hi) {
    fetch(va, p.A, p.a_row, p.a_k, p.a_f32, m0, p.M, k_lo);
    fetch(vb, p.B, p.b_row, p.b_k, p.b_f32, n0, p.N, k_lo);
    keep(sa[0], va, p.a_k);
    keep(sb[0], vb, p.b_k);
  }
  __syncthreads();
  int buf = 0;
  for (int k0 = k_lo; k0 < k_hi; k0 += SK) {
    const bool more = k0 + SK < k_hi;
    if (more) {  // the next step's loads fly while this one is multiplied
      fetch(va, p.A, p.a_row, p.a_k, p.a_f32, m0, p.M, k0 + SK);
      fetch(vb, p.B, p.b_row, p.b_k, p.b_f32, n0, p.N, k0 + SK);
    }
#pragma unroll
    for (int k = 0; k < SK; ++k) {
      float2 a[TM / 2];
      float b[TN];
#pragma unroll
      for (int i = 0; i < TM; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(&sa[buf][k][ty * TM + i]);
        a[i / 2] = make_float2(v.x, v.y);
        a[i / 2 + 1] = make_float2(v.z, v.w);
      }
#pragma unroll
      for (int j = 0; j < TN; j += 4)
        *reinterpret_cast<float4*>(b + j) = *reinterpret_cast<const float4*>(&sb[buf][k][j * 16 + tx * 4]);
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const float2 bb = make_float2(b[j], b[j]);
#pragma unroll
        for (int i = 0; i < TM / 2; ++i) acc2[i][j] = __ffma2_rn(a[i], bb, acc2[i][j]);
      }
    }
    if (more) {
      keep(sa[buf ^ 1], va, p.a_k);
      keep(sb[buf ^ 1], vb, p.b_k);
    }
    __syncthreads();
    buf ^= 1;
  }
  auto acc = [&](int i, int j) { return i & 1 ? acc2[i / 2][j].y : acc2[i / 2][j].x; };
  // the thread's rows m0 + TM ty + i, columns n0 + 64 (j / 4) + 4 tx + j % 4
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int row = m0 + ty * TM + i;
    const bool live = row < p.M;
    auto col_of = [&](int j) { return n0 + j / 4 * 64 + tx * 4 + j % 4; };
    if constexpr (MODE == S_STATS) {
      constexpr float kLog2e = 1.4426950408889634f;
      const int tgt = live ? p.target[row] : -1;
      float m = -INFINITY;
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        if (col_of(j) < p.N) {
          if (col_of(j) == tgt) p.target_logit[row] = acc(i, j);
          m = fmaxf(m, acc(i, j) * kLog2e);
        }
      }
#pragma unroll
      for (int off = 8; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
      const float base = m == -INFINITY ? 0.0f : m;
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < TN; ++j)
        if (col_of(j) < p.N) s += exp2f(fmaf(acc(i, j), kLog2e, -base));
#pragma unroll
      for (int off = 8; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      if (tx == 0 && live) p.part[(int64_t)blockIdx.y * p.M + row] = make_float2(m, s);
    } else if (live) {
      float lse = 0.0f, g = 0.0f;
      int tgt = -1;
      bool counts = false;
      if constexpr (MODE == S_DLOGITS) {
        tgt = p.target[row];
        counts = tgt >= 0 && tgt < p.V;
        lse = p.lse[row];
        g = p.dloss ? p.dloss[row] : p.mean[1];
      }
#pragma unroll
      for (int j0 = 0; j0 < TN; j0 += 4) {
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] = acc(i, j0 + j);
          if constexpr (MODE == S_DLOGITS) {
            v[j] = expf(v[j] - lse);
            if (col_of(j0 + j) + p.v0 == tgt) v[j] -= 1.0f;
            v[j] = counts ? v[j] * g : 0.0f;
          }
        }
        const int col = col_of(j0);
        const int64_t at = ((int64_t)blockIdx.z * p.M + row) * p.ldo + col;
        if (p.out_f32 && p.ldo % 4 == 0 && col + 3 < p.N) {
          float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
          if (p.add) {
            const float4 w = *o;
            v[0] += w.x, v[1] += w.y, v[2] += w.z, v[3] += w.w;
          }
          *o = make_float4(v[0], v[1], v[2], v[3]);
          continue;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (col + j >= p.N) break;
          if (p.out_f32) {
            float* o = static_cast<float*>(p.out) + at + j;
            *o = p.add ? *o + v[j] : v[j];
          } else {
            static_cast<__nv_bfloat16*>(p.out)[at + j] = __float2bfloat16_rn(v[j]);
          }
        }
      }
    }
  }
}

// The tile of a product: 64 while the 128-tiles do not give every SM two blocks.
int simt_tile(int64_t M, int64_t N, int splits) {
  return ceil_div(M, 128) * ceil_div(N, 128) * splits >= 2 * 152 ? 128 : 64;
}

template <int MODE>
cudaError_t launch_simt(SimtParams p, cudaStream_t s) {
  p.k_split = (int)(ceil_div(ceil_div(p.K, p.splits), SK) * SK);
  const int st = simt_tile(p.M, p.N, p.splits);
  const dim3 grid((unsigned)ceil_div(p.M, st), (unsigned)ceil_div(p.N, st), (unsigned)p.splits);
  // a call begins with a plain launch (the logits), the products after it follow closely
  if (MODE == S_STORE)
    return st == 128 ? launch_after(simt_kernel<MODE, 128>, grid, 256, s, p) : launch_after(simt_kernel<MODE, 64>, grid, 256, s, p);
  if (st == 128) simt_kernel<MODE, 128><<<grid, 256, 0, s>>>(p);
  else simt_kernel<MODE, 64><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

// TOK tokens per block of 1024 threads, the other lanes over the halves: lse = max + log(sum),
// the loss, and in the block that finishes last their mean over the tokens that count and its
// reciprocal count. Few tokens take TOK = 4 (a token's 2000 halves of a large vocabulary in 8
// steps), many TOK = 32 (256 bytes of a row of halves per step). Every lane's running (max, sum)
// goes to shared memory, and one warp per token takes the maximum, then the sum.
template <int TOK>
__global__ void __launch_bounds__(1024)
    join_kernel(const float2* part, int parts, int T, int V, const int32_t* target, const float* target_logit,
                float* loss, float* lse, float* mean, uint32_t* ticket, DeviceStatus* st) {
  constexpr int kLanes = 1024 / TOK, kAhead = 4;
  __shared__ float2 lanes[TOK][kLanes + 1];
  __shared__ bool finish;
  after_previous();
  const int tok = threadIdx.x % TOK, lane = threadIdx.x / TOK, warp = threadIdx.x >> 5, wl = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * TOK + tok;
  float m = -INFINITY, s = 0.0f;
  if (t < T) {
    for (int i0 = lane; i0 < parts; i0 += kLanes * kAhead) {
      float2 v[kAhead];
      float m2 = m;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u * kLanes;
        v[u] = i < parts ? __ldg(part + (int64_t)i * T + t) : make_float2(-INFINITY, 0.0f);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) m2 = fmaxf(m2, v[u].x);
      const float base = m2 == -INFINITY ? 0.0f : m2;
      s *= exp2f(m - base);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) s = fmaf(v[u].y, exp2f(v[u].x - base), s);
      m = m2;
    }
  }
  lanes[tok][lane] = make_float2(m, s);
  __syncthreads();
  const int64_t tw = (int64_t)blockIdx.x * TOK + warp;  // the warp's token
  if (warp < TOK && tw < T) {
    float2 v[kLanes / 32];
    m = -INFINITY, s = 0.0f;
#pragma unroll
    for (int u = 0; u < kLanes / 32; ++u) {
      v[u] = lanes[warp][wl + 32 * u];
      m = fmaxf(m, v[u].x);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
    for (int u = 0; u < kLanes / 32; ++u) s = fmaf(v[u].y, exp2f(v[u].x - base), s);
#pragma unroll
    for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (wl == 0) {
      const float l = (m + log2f(s)) * 0.6931471805599453f;
      const int32_t tgt = target[tw];
      if (tgt >= V) set_status(st, MOE_ERR_DEVICE_BAD_INPUT, (int32_t)tw);
      lse[tw] = l;
      loss[tw] = tgt >= 0 && tgt < V ? l - target_logit[tw] : 0.0f;
      __threadfence();
    }
  }
  if (!mean) return;
  __syncthreads();
  if (threadIdx.x == 0) finish = atomicInc(ticket, gridDim.x - 1) == gridDim.x - 1;  // wraps to 0
  __syncthreads();
  if (!finish) return;
  __threadfence();
  __shared__ float sums[32];
  __shared__ int counts[32];
  float sum = 0.0f;
  int count = 0;
  for (int i = threadIdx.x; i < T; i += 1024) {
    const int32_t tgt = target[i];
    if (tgt >= 0 && tgt < V) {
      sum += __ldcg(loss + i);
      ++count;
    }
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, off);
    count += __shfl_xor_sync(0xffffffffu, count, off);
  }
  if (wl == 0) sums[warp] = sum, counts[warp] = count;
  __syncthreads();
  if (warp == 0) {
    double total = (double)sums[wl];
    int n = counts[wl];
#pragma unroll
    for (int off = 16; off; off >>= 1) {
      total += __shfl_xor_sync(0xffffffffu, total, off);
      n += __shfl_xor_sync(0xffffffffu, n, off);
    }
    if (wl == 0) {
      mean[0] = n ? (float)total / (float)n : 0.0f;
      mean[1] = n ? 1.0f / (float)n : 0.0f;
    }
  }
}

// dx = the sum of the K splits' slices [splits][T H], in order.
template <typename T>
__global__ void __launch_bounds__(256) join_dx_kernel(const float* slices, int splits, int64_t n, T* dx) {
  after_previous();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float v = 0.0f;
#pragma unroll 16
  for (int k = 0; k < splits; ++k) v += __ldg(slices + k * n + i);
  if constexpr (sizeof(T) == 4) dx[i] = v;
  else dx[i] = __float2bfloat16_rn(v);
}

bool head_tc(const moe_head_config_t& c) { return c.act_dtype == MOE_DTYPE_BF16 && c.H % 8 == 0; }

}  // namespace

// A piece holds at most 256 MB of dz unless the caller names its length; whole 256-column
// tiles. The SIMT input gradient splits K where its tiles alone would not fill the SMs, into
// slices [splits][T, H]; the tensor cores' split is head_split's.
HeadScratch head_scratch(const moe_head_config_t& c) {
  HeadScratch L{};
  const bool tc = head_tc(c);
  const int64_t esize = tc ? 2 : 4;
  const int64_t T = std::max(c.T, 1);
  int64_t piece = c.piece > 0 ? c.piece : std::max<int64_t>(4096, (256ll << 20) / (T * esize));
  piece = (int64_t)align_up((size_t)std::min<int64_t>(piece, c.V), 256);
  L.piece = piece;
  L.ld = (int)piece;
  const int64_t rows = std::min<int64_t>(piece, c.V);
  const bool one = piece >= c.V;
  size_t dx_bytes;
  if (tc) {
    L.split = tc::head_split(T, c.H, rows);
    dx_bytes = one ? 0 : (size_t)T * c.H * 4;
  } else {
    const int64_t tiles = ceil_div(T, 64) * ceil_div(c.H, 64);
    L.split = {0, (int)std::max<int64_t>(1, std::min<int64_t>({152 * 2 / tiles, rows / 64, 64})), 0};
    dx_bytes = one && L.split.splits == 1 ? 0 : (size_t)L.split.splits * T * c.H * 4;
  }
  size_t o = kWsHead;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes, 256);
    return at;
  };
  // (max, sum) of the halves of 128- or 256-column tiles, or of whole SIMT tiles
  L.part = take((size_t)ceil_div(c.V, 128) * 2 * T * 8);
  L.target_logit = take((size_t)T * 4);
  L.dlogits = take((size_t)T * piece * esize);
  L.dx = take(dx_bytes);
  L.slices = take(L.split.bytes);
  L.total = o;
  return L;
}

cudaError_t launch_head_loss(const moe_head_config_t& c, const void* x, const void* w, const int32_t* target,
                             float* loss, float* lse, float* mean, void* ws, DeviceStatus* st, cudaStream_t s) {
  if (c.T == 0) return mean ? cudaMemsetAsync(mean, 0, 8, s) : cudaSuccess;
  const HeadScratch L = head_scratch(c);
  char* b = static_cast<char*>(ws);
  auto* part = reinterpret_cast<float2*>(b + L.part);
  auto* tl = reinterpret_cast<float*>(b + L.target_logit);
  cudaError_t e;
  int parts;
  if (head_tc(c)) {
    parts = 2 * (int)ceil_div(c.V, tc::head_tile_cols(c.T));
    e = tc::launch_head_stats(c, x, w, target, part, tl, st, s);
  } else {
    parts = (int)ceil_div(c.V, simt_tile(c.T, c.V, 1));
    const int f32 = c.act_dtype == MOE_DTYPE_F32;
    SimtParams p{};
    p.M = c.T, p.N = c.V, p.K = c.H, p.splits = 1;
    p.A = x, p.B = w;
    p.a_row = p.b_row = c.H, p.a_k = p.b_k = 1;
    p.a_f32 = p.b_f32 = f32, p.vec = c.H % 4 == 0;
    p.target = target, p.part = part, p.target_logit = tl;
    e = launch_simt<S_STATS>(p, s);
  }
  if (e != cudaSuccess) return e;
  // the ticket lives in the head, which moe_workspace_init clears
  auto* ticket = reinterpret_cast<uint32_t*>(b + 320);
  if (c.T >= 1024)
    return launch_after(join_kernel<32>, (unsigned)ceil_div(c.T, 32), 1024, s, part, parts, c.T, c.V, target, tl, loss, lse,
                        mean, ticket, st);
  return launch_after(join_kernel<4>, (unsigned)ceil_div(c.T, 4), 1024, s, part, parts, c.T, c.V, target, tl, loss, lse, mean,
                      ticket, st);
}

cudaError_t launch_head_loss_backward(const moe_head_config_t& c, const void* x, const void* w, const int32_t* target,
                                      const float* lse, const float* dloss, const float* mean, void* dx, void* dw,
                                      void* ws, DeviceStatus* st, cudaStream_t s) {
  if (c.T == 0)
    return dw ? cudaMemsetAsync(dw, 0, (size_t)c.V * c.H * (c.grad_dtype == MOE_DTYPE_F32 ? 4 : 2), s) : cudaSuccess;
  const HeadScratch L = head_scratch(c);
  const bool tc = head_tc(c), one = L.piece >= c.V && (tc || L.split.splits == 1);
  char* b = static_cast<char*>(ws);
  float* slices = reinterpret_cast<float*>(b + L.dx);
  const int f32 = c.act_dtype == MOE_DTYPE_F32;
  for (int64_t v0 = 0; v0 < c.V; v0 += L.piece) {
    const int rows = (int)std::min<int64_t>(L.piece, c.V - v0);
    cudaError_t e;
    if (tc) {
      e = tc::launch_head_piece(c, x, w, target, lse, dloss, mean, v0, rows, b + L.dlogits, L.ld,
                                dx ? (one ? dx : slices) : nullptr, L.split, reinterpret_cast<float*>(b + L.slices),
                                !one, v0 > 0, dw, st, s);
      if (e != cudaSuccess) return e;
      continue;
    }
    SimtParams p{};
    p.M = c.T, p.N = rows, p.K = c.H, p.splits = 1;
    p.A = x, p.a_row = c.H, p.a_k = 1, p.a_f32 = f32;
    p.B = static_cast<const char*>(w) + v0 * c.H * (f32 ? 4 : 2), p.b_row = c.H, p.b_k = 1, p.b_f32 = f32;
    p.target = target, p.lse = lse, p.dloss = dloss, p.mean = mean, p.v0 = (int)v0, p.V = c.V;
    p.out = b + L.dlogits, p.ldo = L.ld, p.out_f32 = 1, p.vec = c.H % 4 == 0;
    if ((e = launch_simt<S_DLOGITS>(p, s)) != cudaSuccess) return e;
    SimtParams q{};
    q.A = b + L.dlogits, q.a_f32 = 1, q.splits = 1, q.vec = c.H % 4 == 0;
    if (dx) {
      q.M = c.T, q.N = c.H, q.K = rows, q.splits = L.split.splits;
      q.a_row = L.ld, q.a_k = 1;
      q.B = p.B, q.b_row = 1, q.b_k = c.H, q.b_f32 = f32;
      q.out = one ? dx : slices, q.ldo = c.H, q.out_f32 = one ? f32 : 1, q.add = v0 > 0;
      if ((e = launch_simt<S_STORE>(q, s)) != cudaSuccess) return e;
    }
    if (dw) {
      const int g32 = c.grad_dtype == MOE_DTYPE_F32;
      q.M = rows, q.N = c.H, q.K = c.T, q.splits = 1, q.add = 0;
      q.a_row = 1, q.a_k = L.ld;
      q.B = x, q.b_row = 1, q.b_k = c.H, q.b_f32 = f32;
      q.out = static_cast<char*>(dw) + v0 * c.H * (g32 ? 4 : 2), q.ldo = c.H, q.out_f32 = g32;
      if ((e = launch_simt<S_STORE>(q, s)) != cudaSuccess) return e;
    }
  }
  if (!dx || one) return cudaSuccess;
  const int64_t n = (int64_t)c.T * c.H;
  const int splits = tc ? 1 : L.split.splits;
  const unsigned grid = (unsigned)ceil_div(n, 256);
  const float* from = slices;
  return f32 ? launch_after(join_dx_kernel<float>, grid, 256, s, from, splits, n, static_cast<float*>(dx))
             : launch_after(join_dx_kernel<__nv_bfloat16>, grid, 256, s, from, splits, n, static_cast<__nv_bfloat16*>(dx));
}

}  // namespace moe
