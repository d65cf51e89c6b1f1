// The vocabulary head: softmax cross entropy of tokens x [T, H] against w [V, H], and its
// gradients, without ever holding the logits z = x w^T [T, V]:
//   lse_t = log sum_v exp z_tv;  loss_t = lse_t - z_{t,target}
//   dz_tv = (exp(z_tv - lse_t) - [v = target_t]) dloss_t;  dx = dz w;  dw = dz^T x
// Forward: one GEMM whose epilogue keeps, per token and half tile of columns, the running
// maximum and the sum of exponentials against it, without the target's; join_kernel puts the
// halves and the target's logit together. Backward: piece after piece of the vocabulary, the GEMM
// is run again and its epilogue turns the logits into dz (bf16, the operand of the next products),
// then dx += dz w_piece and dw_piece = dz^T x; all of it over the tokens that count alone, which
// gather_kernel puts one after the other. The logits are never whole. In the workspace, besides
// 8 bytes a token: (max, sum) of the half tiles, 16 bytes per token and 128 or 256 columns; the rows
// of x that count; one piece of dz; with several pieces dx in fp32; where dx may be split, its
// slices, up to 304 tiles of 256 x 256 fp32 (80 MB); of laid-out operands (below) x and a piece of w
// in all their planes.
//
// The target's logit is a dot product of its own, in fp32 (target_logits), the same bits in both
// directions. Where the model is nearly certain, the target's dz is p - 1 with p near 1, and lse is
// the target's logit but for a small part; what is left of their difference is the error of one
// against the other. With the tensor core's logits, which truncate (and by another amount in the
// backward's longer runs), dx of tokens with a loss of 3e-5 was off by 164 % of itself, of 5e-3 by
// 0.76 %; so by 1.1 % and 0.23 %, which is the rounding of lse and of dz. The dot products run beside
// the forward's GEMM and in the backward's first launch: nothing up to some hundred tokens, 8 us of
// 4096 x 4096 x 32000 forward (596 us).
//
// All products run on the tensor cores (tcgen05): warp 0 feeds a ring of shared-memory stages
// by TMA, warp 1 issues the MMAs into two TMEM accumulators, warps 2-9 are the epilogue of one
// accumulator while the other fills. Tiles are 256 x 256 on a CTA pair, or on one CTA 128 rows
// and 64 to 256 columns for up to 128 tokens, where reading w is all the time there is and the
// width is chosen to spread it evenly over the SMs. Edges need no special case in the operands: the TMA fills zeros
// past the last row and column.
//
// fp32 operands are split into three bf16 planes, v = v0 + v1 + v2 with 8 bits of the mantissa
// each, and a product takes the six plane products above 2^-24 of it: x0 w0, x0 w1, x1 w0,
// x0 w2, x1 w1, x2 w0, and the stages of 64 elements added in fp32. That is fp32 accuracy at a sixth of
// the bf16 rate; exact fp32 FMA tiles reached 23 to 36 TFLOP/s (1024 x 1024 x 8192, forward and
// backward: 2401 us, against 421). The planes of x and of one piece of w are laid out in the workspace, rows
// padded to a multiple of 16 bytes; bf16 operands of a width that is not a multiple of 8 are
// copied there too, as one plane (their dz has three).
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>

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
constexpr int kMaxStages = 12;  // of a ring whose stages are sized at run time
constexpr int kMaxSplits = 32;  // of the K of a tile of dx (a lane of a warp tries each)
constexpr int kNowhere = -(1 << 30);  // no column: far below the first of any tile

enum Mode { STATS = 0, DLOGITS = 1, DX = 2, DW = 3 };

// What the backward's gather_kernel finds: the tokens that count, and how the tiles of dx are split.
struct HeadPlan {
  int rows;    // tokens that count: rows of x's copy, of dz, and of dx before they go to their places
  int direct;  // DX: the first `direct` tiles are whole; the K of each further one is split over
  int splits;  //   `splits` units, which write fp32 tiles to `slices`
};

struct HeadParams {
  int M, N;            // rows and columns of the product that exist
  int m_tiles, n_tiles, kblocks;
  const HeadPlan* plan;  // the backward's: its rows stand for M (DLOGITS, DX) or K (DW)
  const int32_t* index;  // DLOGITS, DX: the token of each row (NULL: its number)
  float* slices;       // DX: of split tiles, [tile - direct][split][TM][BN]
  int v0;              // first vocabulary row of the piece
  int w_row0;          // its row in the map of w (0 where the piece was laid out by itself)
  int V;
  int a_planes, b_planes;  // of A and B in a K stage of 64 elements
  int terms;           // plane products per K stage, and the planes of A and B in each of them,
  uint32_t a_code, b_code;  //   four bits a term from the first on
  int a_plane, b_plane;  // rows from one plane of A and B to the next
  int a_bytes;         // of A in a stage: its map's box may have fewer than 128 rows
  const int32_t* target;
  // STATS: (max, sum) per token and half tile [2 n_tiles][T] - or, where all tiles have the same
  // rows (one m tile), per half of a CTA's or pair's tiles [2 units][T] - without the target's logit
  float2* part;
  int bn;              // STATS on single CTAs: columns of a tile, a multiple of 16
  int stages;          // of the ring, where they are sized at run time: there (a_bytes and bn rows of
                       //   w), and with planes (all those of a K stage)
  // DLOGITS
  const float *lse, *dloss;
  const float* target_logit;  // [T], from gather_kernel
  // outputs of the other modes, and their row length in elements
  void* out;
  int64_t ldo;
  int64_t out_plane;   // DLOGITS: elements from one plane of dz to the next
  int out_f32;         // DX, DW: fp32 output (else bf16)
  int scalar;          // DX, DW: the output's rows do not begin on 16-byte boundaries
  int add;             // DX: added to what out holds (a later piece of the vocabulary)
  const float* factor; // DX, DW: every value is multiplied by it (the mean's 1 / count), or NULL
  int follows;         // launched while the kernel before it in the call may still run
  DeviceStatus* status;
  uint64_t timeout_ns;
};

constexpr int kRingBytes = 192 * 1024;

template <int CG, int BN>
struct HeadSmem {
  static constexpr int kBBytes = (BN / CG) * BK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = kRingBytes / kStageBytes;
  static constexpr size_t kBytes = 1024 + kRingBytes + 256 + kEpiWarps * 2048;
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

// flush_rows_64B from row row0 of base on, with a column bound: the 16-byte pieces c >= pieces are
// left out. at (or NULL): where the rows go instead.
__device__ __forceinline__ void flush_edge(uint8_t* stage, int lane, uint8_t* base, int64_t stride, int row0,
                                           const int32_t* at, int live, int pieces, bool add) {
  __syncwarp();
  const int c = lane & 3;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int row = 8 * j + (lane >> 2);
    uint4 v = *reinterpret_cast<const uint4*>(stage + row * 64 + 16 * (c ^ ((row >> 1) & 3)));
    if (row < live && c < pieces) {
      uint4* dst = reinterpret_cast<uint4*>(base + (at ? at[row] : row0 + row) * stride + 16 * c);
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

// The same for rows that do not begin on 16-byte boundaries: element by element, cols of them.
template <typename T>
__device__ __forceinline__ void flush_scalar(const uint8_t* stage, int lane, T* base, int64_t ldo, int row0,
                                             const int32_t* at, int live, int cols, bool add) {
  __syncwarp();
  constexpr int kPer = 64 / sizeof(T);
#pragma unroll 4
  for (int j = 0; j < kPer; ++j) {
    const int e = lane + 32 * j, row = e / kPer, col = e % kPer, c = col * (int)sizeof(T) / 16;
    const T v = *reinterpret_cast<const T*>(stage + row * 64 + 16 * (c ^ ((row >> 1) & 3)) + col * sizeof(T) % 16);
    if (row < live && col < cols) {
      T* dst = base + (at ? at[row] : row0 + row) * ldo + col;
      if constexpr (sizeof(T) == 4) *dst = add ? *dst + v : v;
      else *dst = v;
    }
  }
  __syncwarp();
}

// The product as this launch finds it (with a plan, known on the device only).
struct HeadShape {
  int M, m_tiles, n_tiles, kblocks;
  int direct, splits;
};
template <int MODE>
__device__ __forceinline__ HeadShape head_shape(const HeadParams& p, int tm) {
  HeadShape h{p.M, p.m_tiles, p.n_tiles, p.kblocks, 0, 1};
  if (MODE != STATS) {
    const int rows = p.plan->rows;
    if (MODE == DW) h.kblocks = (rows + BK - 1) / BK;
    else h.M = rows, h.m_tiles = (rows + tm - 1) / tm;
  }
  h.direct = h.m_tiles * h.n_tiles;
  if (MODE == DX) h.direct = p.plan->direct, h.splits = p.plan->splits;
  return h;
}

struct HeadTile {
  int mb, nb, slice, kb0, kb1;  // slice: -1, or the tile's place in `slices`
};

// Which tiles run side by side, and so share operands through L2. Logits and dx: the m tiles
// (a tile of w is read once, x or a K slice of dz stays in L2). dw: the n tiles (the columns of
// dz are read once, x stays in L2; with the m tiles first, dz came from DRAM once per n tile,
// 4.2 GB for 4096 x 4096 x 32000, and the product took 700 us).
template <int MODE>
__device__ __forceinline__ HeadTile head_tile(int unit_index, const HeadShape& h) {
  HeadTile t;
  int tile = unit_index;
  t.slice = -1;
  t.kb0 = 0;
  t.kb1 = h.kblocks;
  if (MODE == DX && unit_index >= h.direct) {
    t.slice = unit_index - h.direct;
    const int split = t.slice % h.splits;
    tile = h.direct + t.slice / h.splits;
    t.kb0 = (int)((int64_t)h.kblocks * split / h.splits);
    t.kb1 = (int)((int64_t)h.kblocks * (split + 1) / h.splits);
  }
  if (MODE == DW) {
    t.mb = tile / h.n_tiles;
    t.nb = tile - t.mb * h.n_tiles;
  } else {
    t.nb = tile / h.m_tiles;
    t.mb = tile - t.nb * h.m_tiles;
  }
  return t;
}

// NP planes: 1, or up to 3 per operand with p.terms products per K stage (the smallest first).
template <int MODE, int CG, int BN, int NP>
__global__ void __launch_bounds__(kThreads, 1)
    head_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const HeadParams p) {
  using S = HeadSmem<CG, BN>;
  constexpr int kBBytes = S::kBBytes;
  constexpr int TM = BM * CG;
  constexpr int kTmemCols = 2 * BN;
  constexpr bool kAmn = MODE == DW;                 // A read MN-major (its rows are the K index)
  constexpr bool kBmn = MODE == DX || MODE == DW;   // the same for B
  constexpr int kBoxes = (BN / CG) / 64;
  // Few tokens: the tile's width is chosen so that the SMs' rounds come out even, and a stage has
  // only the rows that there are, so that the ring is deep. The MMA reads 128 rows of A all the
  // same: into the next stages, for rows of the product that are not stored.
  constexpr bool kFlex = MODE == STATS && CG == 1 && NP == 1;
  constexpr int kMostStages = kFlex ? kMaxStages : S::kStages;
  const int bn_cols = kFlex ? p.bn : BN;
  const int kStages = kFlex || NP == 3 ? p.stages : S::kStages;
  // a stage's planes lie one after the other, and a plane of A or B takes
  const int a_bytes = kFlex ? p.a_bytes : kABytes, b_bytes = kFlex ? bn_cols * BK * 2 : kBBytes;
  const int a_planes = NP == 3 ? p.a_planes : 1, b_planes = NP == 3 ? p.b_planes : 1;
  const int a_stride = a_planes * a_bytes, b_stride = b_planes * b_bytes;
  extern __shared__ uint8_t smem_raw[];
  let_next_begin();
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + kStages * a_stride;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kRingBytes);
  uint64_t* full = bars;
  uint64_t* empty = bars + kMostStages;
  uint64_t* tfull = bars + 2 * kMostStages;
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
  after_previous();  // nothing of memory was touched before
  const uint32_t tmem_base = *tmem_slot;
  const HeadShape h = head_shape<MODE>(p, TM);
  const int total_tiles = h.direct + (h.m_tiles * h.n_tiles - h.direct) * h.splits;
  // The loss's logits and all sums of planes are added up in runs: each has its own accumulator, and
  // the epilogue adds the runs in fp32. The tensor core's own additions truncate: over 4096 elements
  // in one go the loss was off by 3.4e-6 of its size, in runs of 1024 by 7e-7, of 512 by 3.6e-7, of
  // 256 by 1.8e-7. 256 where reading w leaves the time (32 x 4096 x 131072: 171 us, 168 with 512),
  // 512 from 128 tokens on (4096 x 4096 x 32000: 590 us, 566 with 1024, 645 with 256). All six
  // products of one K stage of planes are a run, the big one last (dw of 256 x 128 x 5003: off by
  // 4e-7, and 1.1e-6 with two stages; 1024 x 1024 x 8192 forward and backward 421 us, and 389).
  // Where dz is rounded to bf16 for the next products (which leaves dw off by up to 1.6e-3 by norm,
  // in fp32 too), one go is good enough: those 256 steps of 16 lose 0.2 half units of fp32 each, so a
  // sum over 131072 tokens 1.1e-4. The target's dz, which could not bear it, has its own logit.
  constexpr bool kRuns = MODE == STATS || NP == 3;
  const int terms = NP == 3 ? p.terms : 1;
  const int run_stages = NP == 3 ? min(4, 6 / terms) : CG == 1 ? 4 : 8;
  auto runs_of = [&](const HeadTile& t) { return kRuns ? (t.kb1 - t.kb0 + run_stages - 1) / run_stages : 1; };
  auto run_end = [&](const HeadTile& t, int run) { return kRuns ? min(t.kb1, t.kb0 + (run + 1) * run_stages) : t.kb1; };

  if (warp == 0) {
    // ======================= TMA producer (each CTA loads its own rows of A and its part of B)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int64_t issued = 0;
      bool ok = true;
      for (int tile = unit; tile < total_tiles && ok; tile += nunits) {
        const HeadTile t = head_tile<MODE>(tile, h);
        const int am = t.mb * TM + (int)rank * BM, bn = t.nb * bn_cols + (int)rank * (BN / CG);
        for (int kb = t.kb0; kb < t.kb1; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1, abort, p.timeout_ns, p.status)) { ok = false; break; }
          uint32_t bar = 0;
          if constexpr (CG == 1) {
            mbar_arrive_expect_tx(&full[stage], a_planes * p.a_bytes + b_stride);
          } else {
            if (leader) mbar_arrive_expect_tx(&full[stage], 2 * (a_stride + b_stride));
            bar = mapa_shared(smem_addr(&full[stage]), 0);
          }
          auto load = [&](const CUtensorMap* m, uint8_t* dst, int x, int y) {
            if constexpr (CG == 1) tma_load_2d(m, dst, &full[stage], x, y);
            else tma_load_2d_pair(m, dst, bar, x, y);
          };
          for (int pl = 0; pl < a_planes; ++pl) {
            uint8_t* dst = sA + stage * a_stride + pl * a_bytes;
            const int pa = NP == 3 ? pl * p.a_plane : 0;
            if constexpr (kAmn) {
              load(&tmA, dst, am, pa + kb * BK);
              load(&tmA, dst + 8192, am + 64, pa + kb * BK);
            } else {
              load(&tmA, dst, kb * BK, pa + am);
            }
          }
          for (int pl = 0; pl < b_planes; ++pl) {
            uint8_t* dst = sB + stage * b_stride + pl * b_bytes;
            const int pb = NP == 3 ? pl * p.b_plane : 0;
            if constexpr (kBmn) {
              const int y = pb + (MODE == DX ? p.w_row0 : 0) + kb * BK;
#pragma unroll
              for (int j = 0; j < kBoxes; ++j) load(&tmB, dst + 8192 * j, bn + 64 * j, y);
            } else {
              load(&tmB, dst, kb * BK, pb + p.w_row0 + bn);
            }
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
      const uint32_t idesc = idesc_make(1, TM, bn_cols) | ((kAmn ? 1u : 0u) << 15) | ((kBmn ? 1u : 0u) << 16);
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (int tile = unit; tile < total_tiles && ok; tile += nunits) {
        const HeadTile t = head_tile<MODE>(tile, h);
        int kb = t.kb0;
        for (int run = 0; run < runs_of(t) && ok; ++run) {
          if (!mbar_wait(&tempty[acc], acc_phase ^ 1, abort, p.timeout_ns, p.status)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + acc * BN;
          const int first = kb, end = run_end(t, run);
          for (; kb < end; ++kb) {
            if (!mbar_wait(&full[stage], phase, abort, p.timeout_ns, p.status)) { ok = false; break; }
            tc_fence_after();
            const uint32_t a_stage = smem_addr(sA + stage * a_stride), b_stage = smem_addr(sB + stage * b_stride);
            for (int term = 0; term < terms; ++term) {
              const uint32_t a_addr = a_stage + (NP == 3 ? (p.a_code >> (4 * term) & 3) * a_bytes : 0);
              const uint32_t b_addr = b_stage + (NP == 3 ? (p.b_code >> (4 * term) & 3) * b_bytes : 0);
#pragma unroll
              for (int k = 0; k < BK / 16; ++k) {
                const uint64_t ad = kAmn ? desc_mn(a_addr + k * 2048) : desc_k_sw128(a_addr + k * 32);
                const uint64_t bd = kBmn ? desc_mn(b_addr + k * 2048) : desc_k_sw128(b_addr + k * 32);
                const uint32_t accumulate = kb > first || term > 0 || k > 0;
                if constexpr (CG == 1) mma_bf16(d_tmem, ad, bd, idesc, accumulate);
                else mma_bf16_pair(d_tmem, ad, bd, idesc, accumulate);
              }
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
    float run_max = -INFINITY, run_sum = 0.0f;  // STATS with one m tile: of all tiles so far
    for (int tile = unit; tile < total_tiles; tile += nunits) {
      const HeadTile t = head_tile<MODE>(tile, h);
      const int row0 = t.mb * TM + wrow, row = row0 + lane;  // the thread's row of the product
      const int col0 = t.nb * bn_cols + cbase;               // the warp's first column
      const bool live = row < h.M;
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

      // dz or output values of the 32 columns from c0 of this warp's share on
      int tgt = -1;
      bool counts = false;
      float lse = 0.0f, g = 0.0f, hit = 0.0f;  // hit: DLOGITS, the target's p - 1
      if constexpr (MODE == STATS || MODE == DLOGITS) {
        const int token = MODE == DLOGITS && live ? p.index[row] : row;
        if (live) tgt = __ldg(p.target + token);
        counts = tgt >= 0 && tgt < p.V;
        tgt = counts ? tgt - p.v0 : kNowhere;  // the target's column of this piece, or outside it
        if (MODE == DLOGITS && counts) {
          lse = __ldg(p.lse + token);
          // the gradient of the mean: its factor 1 / count is left to the two products
          g = p.dloss ? __ldg(p.dloss + token) : 1.0f;
          if (tgt >= col0 && tgt < col0 + kCols) hit = expm1f(p.target_logit[token] - lse);
        }
      } else {
        g = p.factor ? __ldg(p.factor) : 1.0f;
      }
      auto finish = [&](float (&v)[32], int c0) {
        const int cc = col0 + c0;   // first column of the chunk
        const int cols = p.N - cc;  // columns from there on that exist
        if constexpr (MODE == DLOGITS) {
          const int at = tgt - cc;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            // fp32 outputs follow p to its last bits; a dz that is rounded to bf16 does not
            const float e = NP == 3 ? expf(v[i] - lse) : ex2((v[i] - lse) * kLog2e);
            const float pr = i == at ? hit : e;
            v[i] = counts && i < cols ? pr * g : 0.0f;
          }
          // columns past the vocabulary, and rows up to a whole K stage of dw, are written too, as
          // zeros: they are K rows of the next products
          __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + (int64_t)row0 * p.ldo + cc;
#pragma unroll
          for (int pl = 0; pl < NP; ++pl) {
            stage_bf16(stage, lane, v);
            flush_rows_64B(stage, lane, reinterpret_cast<uint8_t*>(out + pl * p.out_plane), p.ldo * 2, (h.M + BK - 1) / BK * BK - row0);
            if (pl + 1 < NP)
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] -= __bfloat162float(__float2bfloat16_rn(v[i]));
          }
        } else {
          const int32_t* at = MODE == DX && p.index ? p.index + row0 : nullptr;  // the places of the warp's rows
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] *= g;
          if (MODE == DX && t.slice >= 0) {
            uint8_t* out = reinterpret_cast<uint8_t*>(p.slices + ((int64_t)t.slice * TM + wrow) * BN + cbase + c0);
#pragma unroll
            for (int q = 0; q < 32; q += 16) {
              stage_f32(stage, lane, v + q);
              flush_rows_64B(stage, lane, out + 4 * q, BN * 4, 32);
            }
          } else if (p.out_f32) {
            float* out = static_cast<float*>(p.out) + cc;
            const bool add = MODE == DX && p.add;
#pragma unroll
            for (int q = 0; q < 32; q += 16) {
              stage_f32(stage, lane, v + q);
              if (NP == 3 && p.scalar) flush_scalar(stage, lane, out + q, p.ldo, row0, at, h.M - row0, cols - q, add);
              else flush_edge(stage, lane, reinterpret_cast<uint8_t*>(out + q), p.ldo * 4, row0, at, h.M - row0, (cols - q) / 4, add);
            }
          } else {
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + cc;
            stage_bf16(stage, lane, v);
            if (NP == 3 && p.scalar) flush_scalar(stage, lane, out, p.ldo, row0, at, h.M - row0, cols, false);
            else flush_edge(stage, lane, reinterpret_cast<uint8_t*>(out), p.ldo * 2, row0, at, h.M - row0, cols / 8, false);
          }
        }
      };

      if constexpr (kRuns) {
        // this row's half of the tile's columns, out of TMEM before anything is made of it
        uint32_t zr[kCols / 32][32];
        const int runs = runs_of(t);
        bool ok = true;
        if (runs == 0) {  // no K stages: of a split, or no token counts
#pragma unroll
          for (int i = 0; i < kCols; ++i) zr[i / 32][i % 32] = 0u;
        }
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
        if constexpr (MODE == STATS) {
          // columns from here on that exist, in this tile
          const int cols = min(p.N - col0, bn_cols - cbase);
          if (tgt >= col0 && tgt < col0 + min(kCols, cols)) {  // its logit joins the sum later
#pragma unroll
            for (int i = 0; i < kCols; ++i)
              if (col0 + i == tgt) zr[i / 32][i % 32] = __float_as_uint(-INFINITY);
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
          // z - max is exact near the maximum; z log2 e - max log2 e would carry the rounding of the
          // second product, several U, into every term
          const float mx = fmaxf(m0, m1), base = mx == -INFINITY ? 0.0f : mx;
          float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
          for (int i = 0; i < kCols; i += 2) {
            s0 += ex2((z(i) - base) * kLog2e);
            s1 += ex2((z(i + 1) - base) * kLog2e);
          }
          if (p.m_tiles > 1) {
            if (live) p.part[(int64_t)(2 * t.nb + half) * p.M + row] = make_float2(mx, s0 + s1);
          } else {
            const float m = fmaxf(run_max, mx), m_base = m == -INFINITY ? 0.0f : m;
            run_sum = fmaf(run_sum, ex2((run_max - m_base) * kLog2e), (s0 + s1) * ex2((mx - m_base) * kLog2e));
            run_max = m;
          }
        } else {
#pragma unroll
          for (int c0 = 0; c0 < kCols; c0 += 32) {
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = z(c0 + i);
            finish(v, c0);
          }
        }
      } else {
        if (!wait_full()) break;
        const bool none = t.kb0 == t.kb1;  // no K stages (of a split, or no token counts): nothing in the accumulator
        const uint32_t t_row = t_lane + acc * BN;
        uint32_t nxt[32];
        tmem_ld32(t_row, nxt);
#pragma unroll 1
        for (int c0 = 0; c0 < kCols; c0 += 32) {
          float v[32];
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = none ? 0.0f : __uint_as_float(nxt[i]);
          if (c0 + 32 < kCols) tmem_ld32(t_row + c0 + 32, nxt);  // next chunk in flight
          finish(v, c0);
        }
        release();
      }
    }
    if (MODE == STATS && p.m_tiles == 1 && wrow + lane < p.M)
      p.part[(int64_t)(2 * unit + half) * p.M + wrow + lane] = make_float2(run_max, run_sum);
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

// *walkers: the CTAs, or pairs, that walk the tiles. p.follows: not the first launch of its call.
template <int MODE, int CG, int BN, int NP>
cudaError_t launch_gemm(const CUtensorMap& a, const CUtensorMap& b, const HeadParams& p, int* walkers, cudaStream_t s) {
  auto kern = head_gemm_kernel<MODE, CG, BN, NP>;
  const size_t smem = HeadSmem<CG, BN>::kBytes;
  static std::atomic<bool> attr_set{false};  // per instantiation
  if (!attr_set.load(std::memory_order_relaxed)) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    attr_set.store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(CG * (num_sms() / CG));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int units = std::min(num_sms(), 152) / CG;  // the workspace has room for the sums of that many
  if (CG == 2) {  // a persistent grid must be resident all at once: no more pairs than fit together
    static std::atomic<int> max_pairs{0};
    int pairs = max_pairs.load(std::memory_order_relaxed);
    if (!pairs) {
      cudaError_t e = cudaOccupancyMaxActiveClusters(&pairs, kern, &cfg);
      if (e != cudaSuccess || pairs <= 0) return e != cudaSuccess ? e : cudaErrorInvalidConfiguration;
      max_pairs.store(pairs, std::memory_order_relaxed);
    }
    units = std::min(units, pairs);
  }
  // as many as the tiles there may be (those of dx up to split 32 ways)
  units = (int)std::min<int64_t>(units, (int64_t)p.m_tiles * p.n_tiles * (MODE == DX ? kMaxSplits : 1));
  if (walkers) *walkers = units;
  cfg.gridDim = dim3((unsigned)(CG * units));
  cfg.numAttrs = p.follows ? 2 : 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a, b, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Up to 128 tokens: one 128-row tile, single CTAs. Else 256-row tiles on CTA pairs. Planes take
// 128 columns a tile: the runs' sums of 64 columns per warp stay in registers.
bool small_tokens(int64_t T) { return T <= BM; }
int tile_rows(int64_t T) { return small_tokens(T) ? BM : 2 * BM; }
int tile_cols(int64_t T, int planes) { return small_tokens(T) || planes == 3 ? 128 : 256; }

template <int MODE>
cudaError_t launch_mode(int T, int planes, const CUtensorMap& a, const CUtensorMap& b, const HeadParams& p, cudaStream_t s,
                        int* walkers = nullptr) {
  if constexpr (MODE != DW) {
    if (small_tokens(T)) {
      if (planes == 3) return launch_gemm<MODE, 1, 128, 3>(a, b, p, walkers, s);
      return launch_gemm<MODE, 1, MODE == STATS ? 256 : 128, 1>(a, b, p, walkers, s);
    }
  }
  return planes == 3 ? launch_gemm<MODE, 2, 128, 3>(a, b, p, walkers, s) : launch_gemm<MODE, 2, 256, 1>(a, b, p, walkers, s);
}

// Columns of a logits tile of the forward. Up to 128 tokens, where the time is that of reading w:
// the width, of 64 to 256, with the fewest columns in the rounds that the SMs take together
// (32000 vocabulary rows on 152 SMs: one round of 224 instead of two of 128).
int stats_cols(int64_t T, int64_t V, int planes) {
  if (!small_tokens(T) || planes == 3) return tile_cols(T, planes);
  int best = 128;
  int64_t least = INT64_MAX;
  for (int bn = 256; bn >= 64; bn -= 16) {
    const int64_t cost = ceil_div(ceil_div(V, bn), num_sms()) * (bn + 4);  // a little for every tile
    if (cost < least) least = cost, best = bn;
  }
  return best;
}

// Rows of A's box, and so of a stage's A: what up to 128 tokens fill of the tile. The rest of it
// holds whatever was there, for rows of the product that are not stored. (A box of 128 rows of
// which 120 and more lie outside the tensor is slow to fill: the logits of 1 x 4096 x 32000 took
// 73 us with it, 58 with a box of 16.)
int a_box(int64_t T) { return T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : BM; }

HeadParams base_params(int64_t M, int64_t N, int64_t K, int tm, int tn, DeviceStatus* st) {
  HeadParams p{};
  p.M = (int)M;
  p.N = (int)N;
  p.m_tiles = (int)ceil_div(M, tm);
  p.n_tiles = (int)ceil_div(N, tn);
  p.kblocks = (int)ceil_div(K, BK);
  p.a_bytes = kABytes;
  p.status = st;
  p.timeout_ns = kTimeoutNs;
  return p;
}

// dx of the tiles whose K was split: the sum of a tile's slices in order, written or added.
template <typename T>
__global__ void __launch_bounds__(256) join_slices_kernel(const HeadParams p, int tm, int tn, T* out) {
  let_next_begin();
  after_previous();
  const HeadShape h = head_shape<DX>(p, tm);
  const int tile = h.direct + blockIdx.y, e = (blockIdx.x * 256 + threadIdx.x) * 4;  // 4 columns each
  if (tile >= h.m_tiles * h.n_tiles) return;
  const int nb = tile / h.m_tiles, mb = tile - nb * h.m_tiles;
  const int row = mb * tm + e / tn, col = nb * tn + e % tn;
  if (row >= h.M || col >= p.N) return;
  const float* s = p.slices + (int64_t)blockIdx.y * h.splits * tm * tn + e;
  float4 v = make_float4(0, 0, 0, 0);
#pragma unroll 4
  for (int k = 0; k < h.splits; ++k) {
    const float4 a = *reinterpret_cast<const float4*>(s + (int64_t)k * tm * tn);
    v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
  }
  T* o = out + (int64_t)(p.index ? p.index[row] : row) * p.ldo + col;
  if (p.scalar) {
    const float f[4] = {v.x, v.y, v.z, v.w};
    for (int i = 0; i < 4 && col + i < p.N; ++i) {
      if constexpr (sizeof(T) == 4) o[i] = p.add ? o[i] + f[i] : f[i];
      else o[i] = __float2bfloat16_rn(f[i]);
    }
  } else if constexpr (sizeof(T) == 4) {
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

// Eight columns from c on of a row of H as fp32 (zeros past H).
template <typename T>
__device__ __forceinline__ void load8(const T* row, int c, int H, float (&v)[8]) {
  const bool whole = H % 8 == 0;  // they are all there, and aligned
  if (whole && sizeof(T) == 4) {
    const float4* q = reinterpret_cast<const float4*>(row + c);
    const float4 a = __ldg(q), b = __ldg(q + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else if (whole) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(row + c));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < H ? static_cast<float>(row[c + i]) : 0.0f;
  }
}

// Their NP planes at dst, `plane` elements apart.
template <int NP>
__device__ __forceinline__ void store_planes(__nv_bfloat16* dst, int64_t plane, float (&v)[8]) {
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    *reinterpret_cast<uint4*>(dst + p * plane) =
        make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
    if (p + 1 < NP)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] -= __bfloat162float(__float2bfloat16_rn(v[i]));
  }
}

// The planes of rows [0, rows) of src [., H] in dst [planes][rows_pad][Hp] bf16: zeros past H and
// from `rows` to `zero_to` (the K stages of the products read that far). Eight columns a thread.
template <typename T, int NP>
__global__ void __launch_bounds__(256)
    planes_kernel(const T* src, int rows, int H, __nv_bfloat16* dst, int64_t plane, int Hp, int zero_to) {
  let_next_begin();
  after_previous();
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int per = Hp / 8, row = (int)(e / per), c = (int)(e % per) * 8;
  if (row >= zero_to) return;
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (row < rows) load8(src + (int64_t)row * H, c, H, v);
  store_planes<NP>(dst + (int64_t)row * Hp + c, plane, v);
}

// The input gradient's tiles rarely fill whole rounds of the SMs (4096 x 4096 is 256 tiles of
// 256 x 256 on 76 CTA pairs: 3.37 rounds, so 4). The tiles of the last round are therefore
// split along K, by the number of ways that takes least time: rounds of stages of 64 (0.14 us
// with 256 columns, half of that with 128) against the slices' traffic (0.08 us for a tile of
// 256 x 256) and the launch that adds them. At most four rounds of slices.
struct SplitRule {
  int tm, tn, units, planes, n_tiles, kblocks;
  bool can;  // there is room for slices
  __host__ __device__ float stage() const { return 0.14f * tn / 256 * (planes == 3 ? 6 : 1); }
  __host__ __device__ float slice() const { return 0.08f * tm * tn / 65536; }
  // Whether a split into any number could pay, for any number of rows.
  bool could_pay() const { return kblocks * stage() > 4.0f + 2.0f * sqrtf(kblocks * stage() * slice()); }
  // By a whole warp, a number of splits per lane.
  __device__ HeadPlan of(int rows) const {
    const int lane = threadIdx.x & 31, s = lane + 1;
    const int tiles = (rows + tm - 1) / tm * n_tiles, tail = tiles % units;
    float least = INFINITY;
    if (s == 1) least = kblocks * stage();
    else if (can && tail && s * 4 <= kblocks && tail * s <= 4 * units)
      least = (float)((tail * s + units - 1) / units) * ((kblocks + s - 1) / s) * stage() + tail * s * slice() + 4.0f;
    int best = s;
#pragma unroll
    for (int off = 16; off; off >>= 1) {
      const float other = __shfl_xor_sync(0xffffffffu, least, off);
      const int at = __shfl_xor_sync(0xffffffffu, best, off);
      if (other < least || (other == least && at < best)) least = other, best = at;
    }
    return {rows, best > 1 ? tiles - tail : tiles, best};
  }
  // Room for the slices of any number of rows up to `rows`.
  int64_t most_slices(int64_t rows) const {
    return std::min<int64_t>(kMaxSplits * ceil_div(rows, tm) * n_tiles, 4 * units);
  }
};
SplitRule split_rule(int64_t T, int64_t H, int64_t rows, int planes) {
  const int tm = tile_rows(T), tn = tile_cols(T, planes);
  SplitRule r{tm, tn, small_tokens(T) ? 152 : 76, planes, (int)ceil_div(H, tn), (int)ceil_div(rows, BK), false};
  r.can = r.could_pay();
  return r;
}

// The logits of the targets, logit[t] = x_t . w_target in fp32 for the tokens that count, from token
// `first` on: `warps` warps to a token (1, or 4 for rows of more than four pieces a lane), 8 sums a
// lane, then their tree. By a whole block of kWarps warps; the same bits wherever a token stands.
int target_warps(int H) { return H <= 1024 ? 1 : 4; }
template <int kWarps, typename T>
__device__ __forceinline__ void target_logits(const T* x, const T* w, const int32_t* target, int64_t first, int rows, int H,
                                              int V, int warps, float* logit) {
  __shared__ float part[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = first + warp / warps;
  const int32_t v = t < rows ? __ldg(target + t) : -1;
  const bool counts = v >= 0 && v < V;
  float r = 0.0f;
  if (counts) {
    const T *xr = x + t * H, *wr = w + (int64_t)v * H;
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
    for (int c = (warp % warps * 32 + lane) * 8; c < H; c += warps * 256) {
      float a[8], b[8];
      load8(xr, c, H, a);
      load8(wr, c, H, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] = fmaf(a[i], b[i], sum[i]);
    }
    r = ((sum[0] + sum[1]) + (sum[2] + sum[3])) + ((sum[4] + sum[5]) + (sum[6] + sum[7]));
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) r += __shfl_xor_sync(0xffffffffu, r, off);
  if (warps > 1) {
    if (lane == 0) part[warp] = r;
    __syncthreads();
    const float* p = part + warp / 4 * 4;
    r = (p[0] + p[1]) + (p[2] + p[3]);
  }
  if (counts && lane == 0 && warp % warps == 0) logit[t] = r;
}

// The forward's, launched behind the GEMM, beside which its small blocks run: nothing that may still
// run reads or writes what it touches, so it waits for the kernels before it only at its end. (In
// join_kernel the dot products took 8 us of 64 x 4096 x 32000, which takes 55.)
constexpr int kTargetWarps = 4;
template <typename T>
__global__ void __launch_bounds__(32 * kTargetWarps)
    target_kernel(const T* x, const T* w, const int32_t* target, int rows, int H, int V, int warps, float* logit) {
  let_next_begin();
  target_logits<kTargetWarps>(x, w, target, (int64_t)blockIdx.x * (kTargetWarps / warps), rows, H, V, warps, logit);
  after_previous();  // this kernel's end is also that of those before it
}

// The backward's first kernel: the rows of x whose tokens count, one after the other, in dst
// [planes][rows_pad][Hp] (with zeros up to a whole K stage), their tokens in index, the plan, and
// zeros in the rows of dx whose tokens do not count. What is left out costs the products nothing
// (1500 x 2048 x 50257 with 60 % left out, forward and backward: 515 us, 743 with zeros for them),
// and a NaN or infinity in a padded row of x meets no other row. A block takes 16 tokens and 512
// columns; it counts those of the tokens before its own by itself, from the first or, beyond 65536
// tokens, from the last whole chunk of 4096 on and over the chunks' counts (chunk; else NULL). The
// blocks past the first `gathers` of a slab form the targets' logits instead, 8 or 2 tokens each.
constexpr int kGather = 16, kGatherCols = 512, kItems = kGather * kGatherCols / 8 / 256;
constexpr int kChunk = 4096, kCountFrom = 65536;
__global__ void __launch_bounds__(256) count_kernel(const int32_t* target, int rows, int V, int32_t* chunk) {
  let_next_begin();
  __shared__ int32_t sum;
  if (threadIdx.x == 0) sum = 0;
  __syncthreads();
  const int64_t first = (int64_t)blockIdx.x * kChunk;
  int n = 0;
  for (int64_t i = first + threadIdx.x; i < min((int64_t)rows, first + kChunk); i += 256) {
    const int32_t t = __ldg(target + i);
    n += t >= 0 && t < V;
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) n += __shfl_xor_sync(0xffffffffu, n, off);
  if ((threadIdx.x & 31) == 0) atomicAdd(&sum, n);
  __syncthreads();
  if (threadIdx.x == 0) chunk[blockIdx.x] = sum;
}

template <typename T, int NP>
__global__ void __launch_bounds__(256)
    gather_kernel(const T* x, const T* w, const int32_t* target, int rows, int H, int V, __nv_bfloat16* dst, int64_t plane, int Hp,
                  const int32_t* chunk, int32_t* index, HeadPlan* plan, T* dx, SplitRule rule, int gathers, int warps,
                  float* logit) {
  let_next_begin();
  if (chunk) after_previous();
  if ((int)blockIdx.x >= gathers) {
    const int64_t block = (int64_t)(blockIdx.x - gathers) * gridDim.y + blockIdx.y;
    target_logits<8>(x, w, target, block * (8 / warps), rows, H, V, warps, logit);
    return;
  }
  __shared__ int32_t before, place[kGather];
  const int first = blockIdx.x * kGather, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int live = min(kGather, rows - first);
  const int c0 = blockIdx.y * kGatherCols, per = min(kGatherCols, Hp - c0) / 8;  // 8 columns an item
  auto counts = [&](int32_t t) { return t >= 0 && t < V; };
  // everything is on its way before the first wait: the rows, their targets and those before them
  float v[kItems][8];
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int e = threadIdx.x + i * 256, r = e / per;
    if (r < live) load8(x + (int64_t)(first + r) * H, c0 + e % per * 8, H, v[i]);
  }
  const uint32_t mask = __ballot_sync(0xffffffffu, lane < live && counts(__ldg(target + first + min(lane, live - 1))));
  if (threadIdx.x == 0) before = 0;
  __syncthreads();
  int n = 0;
  const int whole = chunk ? first / kChunk : 0;
  for (int i = threadIdx.x; i < whole; i += 256) n += chunk[i];
  for (int i = whole * kChunk + threadIdx.x * 4; i < first; i += 1024) {
    const int4 t = __ldg(reinterpret_cast<const int4*>(target + i));  // first is a multiple of 16
    n += (int)counts(t.x) + (int)counts(t.y) + (int)counts(t.z) + (int)counts(t.w);
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) n += __shfl_xor_sync(0xffffffffu, n, off);
  if (lane == 0 && n) atomicAdd(&before, n);
  __syncthreads();
  if (warp == 0 && lane < kGather) {
    const int at = before + __popc(mask & ((1u << lane) - 1));
    const bool in = mask >> lane & 1;
    place[lane] = in ? at : -1;
    if (in && blockIdx.y == 0) index[at] = first + lane;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int e = threadIdx.x + i * 256, r = e / per, c = c0 + e % per * 8;
    if (r >= live) continue;
    if (place[r] >= 0) {
      store_planes<NP>(dst + (int64_t)place[r] * Hp + c, plane, v[i]);
    } else if (dx) {
      T* o = dx + (int64_t)(first + r) * H + c;
      if (H % 8 == 0) {
#pragma unroll
        for (int q = 0; q < (int)sizeof(T) / 2; ++q) reinterpret_cast<uint4*>(o)[q] = make_uint4(0, 0, 0, 0);
      } else {
        for (int q = 0; q < 8 && c + q < H; ++q) o[q] = T(0.0f);
      }
    }
  }
  if ((int)blockIdx.x == gathers - 1) {
    const int total = before + __popc(mask);
    if (blockIdx.y == 0 && warp == 7) {
      const HeadPlan made = rule.of(total);
      if (lane == 0) *plan = made;
    }
    float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const int to = (total + BK - 1) / BK * BK;
    for (int e = threadIdx.x; e < (to - total) * per; e += 256)
      store_planes<NP>(dst + (int64_t)(total + e / per) * Hp + c0 + e % per * 8, plane, zero);
  }
}

cudaError_t launch_planes(const void* src, int f32, int rows, int H, void* dst, int64_t plane, int Hp, int zero_to,
                          bool follows, cudaStream_t s) {
  const dim3 grid((unsigned)ceil_div((int64_t)zero_to * (Hp / 8), 256));
  auto* d = static_cast<__nv_bfloat16*>(dst);
  const auto* xf = static_cast<const float*>(src);
  const auto* xb = static_cast<const __nv_bfloat16*>(src);
  if (follows)
    return f32 ? launch_after(planes_kernel<float, 3>, grid, 256, s, xf, rows, H, d, plane, Hp, zero_to)
               : launch_after(planes_kernel<__nv_bfloat16, 1>, grid, 256, s, xb, rows, H, d, plane, Hp, zero_to);
  if (f32) planes_kernel<float, 3><<<grid, 256, 0, s>>>(xf, rows, H, d, plane, Hp, zero_to);
  else planes_kernel<__nv_bfloat16, 1><<<grid, 256, 0, s>>>(xb, rows, H, d, plane, Hp, zero_to);
  return cudaGetLastError();
}

// TOK tokens per block of 1024 threads, the other lanes over the halves: lse = max + log(sum),
// the target's logit among them, the loss, and in the block that finishes last their mean over the tokens that count and its
// reciprocal count. Few tokens take TOK = 4 (a token's 2000 halves of a large vocabulary in 8
// steps), many TOK = 32 (256 bytes of a row of halves per step). Every lane's running (max, sum)
// goes to shared memory, and one warp per token takes the maximum, then the sum.
template <int TOK>
__global__ void __launch_bounds__(1024)
    join_kernel(const float2* part, int parts, int T, int V, const int32_t* target, const float* target_logit, float* loss, float* lse, float* mean, uint32_t* ticket, DeviceStatus* st) {
  constexpr int kLanes = 1024 / TOK, kAhead = 4;
  __shared__ float2 lanes[TOK][kLanes + 1];
  __shared__ bool finish;
  const int tok = threadIdx.x % TOK, lane = threadIdx.x / TOK, warp = threadIdx.x >> 5, wl = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * TOK + tok, tw = (int64_t)blockIdx.x * TOK + warp;  // tw: the warp's token
  const int32_t tgt = warp < TOK && tw < T ? __ldg(target + tw) : -1;
  const bool keep = tgt >= 0 && tgt < V;
  after_previous();
  const float hit = keep ? target_logit[tw] : 0.0f;
  float m = -INFINITY, s = 0.0f;
  if (t < T) {
    for (int i0 = lane; i0 < parts; i0 += kLanes * kAhead) {
      float2 v[kAhead];
      float m2 = m;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u * kLanes;
        v[u] = i < parts ? part[(int64_t)i * T + t] : make_float2(-INFINITY, 0.0f);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) m2 = fmaxf(m2, v[u].x);
      const float base = m2 == -INFINITY ? 0.0f : m2;
      s *= expf(m - base);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) s = fmaf(v[u].y, expf(v[u].x - base), s);
      m = m2;
    }
  }
  lanes[tok][lane] = make_float2(m, s);
  __syncthreads();
  if (warp < TOK && tw < T) {
    float2 v[kLanes / 32];
    m = keep ? hit : -INFINITY, s = 0.0f;
#pragma unroll
    for (int u = 0; u < kLanes / 32; ++u) {
      v[u] = lanes[warp][wl + 32 * u];
      m = fmaxf(m, v[u].x);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
    for (int u = 0; u < kLanes / 32; ++u) s = fmaf(v[u].y, expf(v[u].x - base), s);
#pragma unroll
    for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (keep) s += expf(hit - base);
    if (wl == 0) {
      const float l = m + logf(s);
      if (tgt >= V) set_status(st, MOE_ERR_DEVICE_BAD_INPUT, (int32_t)tw);
      lse[tw] = l;
      loss[tw] = keep ? l - hit : 0.0f;
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

// dx = the sums of the pieces, from fp32 (x of one type or the other), at their tokens' rows.
template <typename T>
__global__ void __launch_bounds__(256)
    store_dx_kernel(const float* sums, int64_t n, int H, const int32_t* index, const HeadPlan* plan, T* dx) {
  after_previous();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, row = i / H;
  if (i >= n || row >= plan->rows) return;
  T* o = dx + (int64_t)index[row] * H + i % H;
  if constexpr (sizeof(T) == 4) *o = sums[i];
  else *o = __float2bfloat16_rn(sums[i]);
}

// The plane products of a GEMM: all six of fp32 operands; those of an operand of three planes (A)
// with one of one; or one. A K stage brings every plane once for all of them (by itself for each
// product, 256 x 128 tiles asked for 94 bytes a clock and SM, more than L2 gives: 1024 x 1024 x 8192
// fp32, forward and backward, 506 us; 421 so).
void set_terms(HeadParams* p, int a_planes, int b_planes, bool pair) {
  p->a_planes = a_planes;
  p->b_planes = b_planes;
  p->stages = kRingBytes / (a_planes * kABytes + b_planes * (pair ? HeadSmem<2, 128>::kBBytes : HeadSmem<1, 128>::kBBytes));
  if (a_planes == 3 && b_planes == 3) {  // (0,2) (1,1) (2,0) (0,1) (1,0) (0,0)
    p->terms = 6;
    p->a_code = 0x010210;
    p->b_code = 0x001012;
  } else if (a_planes == 3) {  // (2,0) (1,0) (0,0)
    p->terms = 3;
    p->a_code = 0x012;
    p->b_code = 0;
  } else {
    p->terms = 1;
    p->a_code = p->b_code = 0;
  }
}

// x and one piece of w as the tensor maps read them: in place, or laid out in the workspace.
struct Operands {
  int planes;          // of dz, and the kernel's: 1 in place, 3 where laid out
  int in_planes;       // of x and w
  bool laid_out;
  int64_t cols;        // of a row: H, or H padded to a multiple of 8
  int64_t x_rows, w_rows, dl_rows;     // of the maps
  int64_t x_plane, w_plane, dl_plane;  // rows from a plane to the next
  const void *x, *w;
};

}  // namespace
}  // namespace tc

namespace {

bool is_f32(const moe_head_config_t& c) { return c.act_dtype == MOE_DTYPE_F32; }
bool laid_out(const moe_head_config_t& c) { return is_f32(c) || c.H % 8; }
int planes_of(const moe_head_config_t& c) { return laid_out(c) ? 3 : 1; }  // of dz
int in_planes_of(const moe_head_config_t& c) { return is_f32(c) ? 3 : 1; }   // of x and w
int64_t padded_tokens(const moe_head_config_t& c) { return align_up((size_t)c.T, 64); }  // whole K stages of dw

tc::Operands operands(const moe_head_config_t& c, const HeadScratch& L, const void* x, const void* w, char* ws) {
  tc::Operands o{};
  o.planes = planes_of(c);
  o.in_planes = in_planes_of(c);
  o.laid_out = laid_out(c);
  o.cols = o.laid_out ? (int64_t)align_up((size_t)c.H, 8) : c.H;
  o.x_plane = o.laid_out ? padded_tokens(c) : c.T;
  o.dl_plane = padded_tokens(c);
  o.w_plane = o.laid_out ? L.piece : c.V;
  o.x_rows = o.in_planes * o.x_plane;
  o.w_rows = o.in_planes * o.w_plane;
  o.dl_rows = o.planes * o.dl_plane;
  o.x = o.laid_out ? ws + L.x : x;
  o.w = o.laid_out ? ws + L.w : w;
  return o;
}

// Lays out x, and rows [v0, v0 + rows) of w, where the products need it.
cudaError_t lay_out_x(const moe_head_config_t& c, const tc::Operands& o, const void* x, cudaStream_t s) {
  if (!o.laid_out) return cudaSuccess;
  return tc::launch_planes(x, is_f32(c), c.T, c.H, const_cast<void*>(o.x), o.x_plane * o.cols, (int)o.cols, (int)o.x_plane, false, s);
}
// x's rows that count to o.x, the targets' logits, and what else the backward's first kernel does.
template <typename T, int NP>
cudaError_t launch_gather(const moe_head_config_t& c, const tc::Operands& o, const void* x, const void* w, const int32_t* target,
                          int32_t* index, tc::HeadPlan* plan, void* dx, float* logit, const tc::SplitRule& rule, cudaStream_t s) {
  const int gathers = (int)ceil_div(c.T, tc::kGather), slabs = (int)ceil_div(o.cols, tc::kGatherCols);
  const int warps = tc::target_warps(c.H);
  const dim3 grid((unsigned)(gathers + ceil_div(ceil_div(c.T, 8 / warps), slabs)), (unsigned)slabs);
  const auto *from = static_cast<const T*>(x), *wt = static_cast<const T*>(w);
  auto* to = static_cast<__nv_bfloat16*>(const_cast<void*>(o.x));
  auto* none = static_cast<T*>(dx);
  const int64_t plane = o.x_plane * o.cols;
  if (c.T <= tc::kCountFrom) {
    tc::gather_kernel<T, NP><<<grid, 256, 0, s>>>(from, wt, target, c.T, c.H, c.V, to, plane, (int)o.cols, nullptr, index, plan, none,
                                                  rule, gathers, warps, logit);
    return cudaGetLastError();
  }
  int32_t* chunk = index + padded_tokens(c);
  tc::count_kernel<<<(unsigned)ceil_div(c.T, tc::kChunk), 256, 0, s>>>(target, c.T, c.V, chunk);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_after(tc::gather_kernel<T, NP>, grid, 256, s, from, wt, target, c.T, c.H, c.V, to, plane, (int)o.cols, chunk, index,
                      plan, none, rule, gathers, warps, logit);
}

cudaError_t lay_out_w(const moe_head_config_t& c, const tc::Operands& o, const void* w, int64_t v0, int rows, cudaStream_t s) {
  if (!o.laid_out) return cudaSuccess;
  return tc::launch_planes(static_cast<const char*>(w) + v0 * c.H * (is_f32(c) ? 4 : 2), is_f32(c), rows, c.H,
                           const_cast<void*>(o.w), o.w_plane * o.cols, (int)o.cols, (int)align_up((size_t)rows, 64), true, s);
}

}  // namespace

// A piece holds at most 256 MB of dz and laid-out w unless the caller names its length; whole
// 256-column tiles.
HeadScratch head_scratch(const moe_head_config_t& c) {
  HeadScratch L{};
  const bool lay = laid_out(c);
  const int64_t T = std::max<int64_t>(padded_tokens(c), 1), Hp = align_up((size_t)c.H, 8), np = planes_of(c), ip = in_planes_of(c);
  const int64_t row_bytes = 2 * np * (T + (lay ? Hp : 0));
  int64_t piece = c.piece > 0 ? c.piece : std::max<int64_t>(4096, (256ll << 20) / row_bytes);
  piece = (int64_t)align_up((size_t)std::min<int64_t>(piece, c.V), 256);
  L.piece = piece;
  L.ld = (int)piece;
  size_t o = kWsHead;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes, 256);
    return at;
  };
  // (max, sum) of the halves of 128- or 256-column tiles; one m tile: of the CTAs, for every piece
  L.part = take((size_t)std::max<int64_t>(ceil_div(c.V, 128), T <= 256 ? ceil_div(c.V, lay ? piece : c.V) * 152 : 0) * 2 * T * 8);
  L.target_logit = take((size_t)T * 4);
  L.plan = take(sizeof(tc::HeadPlan));
  L.index = take((size_t)(T + ceil_div(T, tc::kChunk)) * 4);  // and the chunks' counts
  L.x = take((size_t)(ip * T * Hp * 2));
  L.w = take(lay ? (size_t)(ip * piece * Hp * 2) : 0);
  L.dlogits = take((size_t)(np * T * piece * 2));
  L.dx = take(piece >= c.V ? 0 : (size_t)T * c.H * 4);
  const tc::SplitRule rule = tc::split_rule(T, c.H, std::min<int64_t>(piece, c.V), (int)np);
  L.slices = take(rule.can ? (size_t)rule.most_slices(T) * rule.tm * rule.tn * 4 : 0);
  L.total = o;
  return L;
}

cudaError_t launch_head_loss(const moe_head_config_t& c, const void* x, const void* w, const int32_t* target,
                             float* loss, float* lse, float* mean, void* ws, DeviceStatus* st, cudaStream_t s) {
  if (c.T == 0) return mean ? cudaMemsetAsync(mean, 0, 8, s) : cudaSuccess;
  using namespace tc;
  const HeadScratch L = head_scratch(c);
  char* b = static_cast<char*>(ws);
  auto* part = reinterpret_cast<float2*>(b + L.part);
  const Operands o = operands(c, L, x, w, b);
  const int tm = tile_rows(c.T), tn = stats_cols(c.T, c.V, o.planes);
  cudaError_t e = lay_out_x(c, o, x, s);
  int parts = 0, walkers = 0;
  const int64_t step = o.laid_out ? L.piece : c.V;  // w in place needs no pieces here
  for (int64_t v0 = 0; v0 < c.V && e == cudaSuccess; v0 += step) {
    const int rows = (int)std::min<int64_t>(step, c.V - v0);
    if ((e = lay_out_w(c, o, w, v0, rows, s)) != cudaSuccess) break;
    HeadParams p = base_params(c.T, rows, c.H, tm, tn, st);
    p.v0 = (int)v0;
    p.V = c.V;
    set_terms(&p, o.in_planes, o.in_planes, !small_tokens(c.T));
    p.a_bytes = a_box(c.T) * BK * 2;
    p.a_plane = (int)o.x_plane;
    p.b_plane = (int)o.w_plane;
    p.target = target;
    p.follows = o.laid_out || v0 > 0;
    p.bn = tn;
    if (o.planes == 1) p.stages = std::min<int>(kMaxStages, kRingBytes / (a_box(c.T) * BK * 2 + tn * BK * 2));
    p.part = part + (int64_t)parts * c.T;
    CUtensorMap ma, mb;
    if (!bf16_box(&ma, o.x, o.x_rows, o.cols, a_box(c.T)) || !bf16_box(&mb, o.w, o.w_rows, o.cols, tn / (tm / BM)))
      return cudaErrorInvalidValue;
    e = launch_mode<STATS>(c.T, o.planes, ma, mb, p, s, &walkers);
    parts += 2 * (p.m_tiles > 1 ? p.n_tiles : walkers);
  }
  if (e != cudaSuccess) return e;
  auto* ticket = reinterpret_cast<uint32_t*>(b + kHeadTicket);
  const float2* from = part;
  auto* logit = reinterpret_cast<float*>(b + L.target_logit);
  auto targets = [&](auto kern, auto* xt) {
    const int warps = target_warps(c.H);
    return launch_after(kern, (unsigned)ceil_div(c.T, kTargetWarps / warps), 32 * kTargetWarps, s, xt, static_cast<decltype(xt)>(w),
                        target, c.T, c.H, c.V, warps, logit);
  };
  e = is_f32(c) ? targets(target_kernel<float>, static_cast<const float*>(x))
                : targets(target_kernel<__nv_bfloat16>, static_cast<const __nv_bfloat16*>(x));
  if (e != cudaSuccess) return e;
  const float* logits = logit;
  if (c.T >= 1024)
    return launch_after(join_kernel<32>, (unsigned)ceil_div(c.T, 32), 1024, s, from, parts, c.T, c.V, target, logits, loss, lse,
                        mean, ticket, st);
  return launch_after(join_kernel<4>, (unsigned)ceil_div(c.T, 4), 1024, s, from, parts, c.T, c.V, target, logits, loss, lse, mean,
                      ticket, st);
}

cudaError_t launch_head_loss_backward(const moe_head_config_t& c, const void* x, const void* w, const int32_t* target,
                                      const float* lse, const float* dloss, const float* mean, void* dx, void* dw,
                                      void* ws, DeviceStatus* st, cudaStream_t s) {
  const int g32 = c.grad_dtype == MOE_DTYPE_F32, f32 = is_f32(c);
  if (c.T == 0) return dw ? cudaMemsetAsync(dw, 0, (size_t)c.V * c.H * (g32 ? 4 : 2), s) : cudaSuccess;
  using namespace tc;
  const HeadScratch L = head_scratch(c);
  const bool one = L.piece >= c.V;  // dx needs no sum over pieces
  char* b = static_cast<char*>(ws);
  Operands o = operands(c, L, b + L.x, w, b);
  o.x_plane = padded_tokens(c);
  o.x_rows = o.in_planes * o.x_plane;
  const int tm = tile_rows(c.T), tn = tile_cols(c.T, o.planes);
  void* dl = b + L.dlogits;
  float* dx_sums = reinterpret_cast<float*>(b + L.dx);
  const float* factor = mean ? mean + 1 : nullptr;
  auto* plan = reinterpret_cast<HeadPlan*>(b + L.plan);
  auto* index = reinterpret_cast<int32_t*>(b + L.index);
  auto* logit = reinterpret_cast<float*>(b + L.target_logit);
  const SplitRule rule = split_rule(c.T, c.H, std::min<int64_t>(L.piece, c.V), o.planes);
  cudaError_t e = f32 ? launch_gather<float, 3>(c, o, x, w, target, index, plan, dx, logit, rule, s)
                      : launch_gather<__nv_bfloat16, 1>(c, o, x, w, target, index, plan, dx, logit, rule, s);
  for (int64_t v0 = 0; v0 < c.V && e == cudaSuccess; v0 += L.piece) {
    const int rows = (int)std::min<int64_t>(L.piece, c.V - v0);
    if ((e = lay_out_w(c, o, w, v0, rows, s)) != cudaSuccess) break;
    const int w_row0 = o.laid_out ? 0 : (int)v0;
    CUtensorMap ma, mb;
    // dz of the piece: M = T, N = its rows, K = H
    HeadParams p = base_params(c.T, rows, c.H, tm, tn, st);
    p.v0 = (int)v0;
    p.w_row0 = w_row0;
    p.V = c.V;
    set_terms(&p, o.in_planes, o.in_planes, !small_tokens(c.T));
    p.a_bytes = a_box(c.T) * BK * 2;
    p.a_plane = (int)o.x_plane;
    p.b_plane = (int)o.w_plane;
    p.target = target;
    p.lse = lse;
    p.dloss = dloss;
    p.target_logit = logit;
    p.plan = plan;
    p.index = index;
    p.follows = 1;
    p.out = dl;
    p.ldo = L.ld;
    p.out_plane = o.dl_plane * L.ld;
    if (!bf16_box(&ma, o.x, o.x_rows, o.cols, a_box(c.T)) || !bf16_box(&mb, o.w, o.w_rows, o.cols, tn / (tm / BM)))
      return cudaErrorInvalidValue;
    if ((e = launch_mode<DLOGITS>(c.T, o.planes, ma, mb, p, s)) != cudaSuccess) break;
    if (dx) {  // M = T, N = H, K = the piece's rows
      p = base_params(c.T, c.H, rows, tm, tn, st);
      p.w_row0 = w_row0;
      set_terms(&p, o.planes, o.in_planes, !small_tokens(c.T));
      p.a_bytes = a_box(c.T) * BK * 2;
      p.a_plane = (int)o.dl_plane;
      p.b_plane = (int)o.w_plane;
      p.follows = 1;
      p.plan = plan;
      p.index = one ? index : nullptr;  // the sums of pieces stay one row after the other
      p.slices = reinterpret_cast<float*>(b + L.slices);
      p.out = one ? dx : dx_sums;
      p.ldo = c.H;
      p.out_f32 = !one || f32;
      p.scalar = c.H * (p.out_f32 ? 4 : 2) % 16 != 0;
      p.add = v0 > 0;
      p.factor = factor;
      if (!bf16_box(&ma, dl, o.dl_rows, L.ld, a_box(c.T)) || !bf16_box(&mb, o.w, o.w_rows, o.cols, 64)) return cudaErrorInvalidValue;
      if ((e = launch_mode<DX>(c.T, o.planes, ma, mb, p, s)) != cudaSuccess) break;
      if (rule.can) {  // how many tiles are is known on the device; fewer than a round
        const dim3 grid((unsigned)(tm * tn / 1024), (unsigned)std::min(p.m_tiles * p.n_tiles, rule.units - 1));
        e = p.out_f32 ? launch_after(join_slices_kernel<float>, grid, 256, s, p, tm, tn, static_cast<float*>(p.out))
                      : launch_after(join_slices_kernel<__nv_bfloat16>, grid, 256, s, p, tm, tn, static_cast<__nv_bfloat16*>(p.out));
        if (e != cudaSuccess) break;
      }
    }
    if (dw) {  // M = the piece's rows, N = H, K = T
      const int wn = o.planes == 3 ? 128 : 256;
      p = base_params(rows, c.H, c.T, 2 * BM, wn, st);
      set_terms(&p, o.planes, o.in_planes, true);
      p.a_plane = (int)o.dl_plane;
      p.b_plane = (int)o.x_plane;
      p.follows = 1;
      p.plan = plan;
      p.out_f32 = g32;
      p.out = static_cast<char*>(dw) + v0 * c.H * (g32 ? 4 : 2);
      p.ldo = c.H;
      p.scalar = c.H * (g32 ? 4 : 2) % 16 != 0;
      p.factor = factor;
      if (!bf16_box(&ma, dl, o.dl_rows, L.ld, 64) || !bf16_box(&mb, o.x, o.x_rows, o.cols, 64)) return cudaErrorInvalidValue;
      e = launch_mode<DW>(c.T, o.planes, ma, mb, p, s);
    }
  }
  if (e != cudaSuccess || !dx || one) return e;
  const int64_t n = (int64_t)c.T * c.H;
  const unsigned grid = (unsigned)ceil_div(n, 256);
  const float* from = dx_sums;
  const int32_t* rows_at = index;
  const HeadPlan* from_plan = plan;
  return f32 ? launch_after(store_dx_kernel<float>, grid, 256, s, from, n, c.H, rows_at, from_plan, static_cast<float*>(dx))
             : launch_after(store_dx_kernel<__nv_bfloat16>, grid, 256, s, from, n, c.H, rows_at, from_plan, static_cast<__nv_bfloat16*>(dx));
}

}  // namespace moe
