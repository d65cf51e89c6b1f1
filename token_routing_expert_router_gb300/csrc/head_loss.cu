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

enum Mode { STATS = 0, DLOGITS = 1, DX = 2, DW = 3 };

struct HeadParams {
  int M, N;            // rows and columns of the product that exist
  int m_tiles, n_tiles, kblocks;
  int splits;          // DX: K splits, each with its own slice of out
  int b_row0;          // first vocabulary row of the piece (STATS: 0)
  int V;
  const int32_t* target;
  // STATS: (max, sum) per token and half tile [2 n_tiles][T], and the target's logit [T]
  float2* part;
  float* target_logit;
  // DLOGITS
  const float *lse, *dloss, *mean;
  // outputs of the other modes, and their row length in elements
  void* out;
  int64_t ldo;
  int out_f32;         // DX, DW: fp32 output (else bf16)
  int add;             // DX: added to what out holds (a later piece of the vocabulary)
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

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
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
  int mb, nb, split, kb0, kb1;
};

// m tiles run fastest: they share a tile of w (or of x) through L2.
__device__ __forceinline__ HeadTile head_tile(int tile, const HeadParams& p) {
  HeadTile t;
  const int per = p.m_tiles * p.n_tiles;
  t.split = tile / per;
  const int local = tile - t.split * per;
  t.nb = local / p.m_tiles;
  t.mb = local - t.nb * p.m_tiles;
  t.kb0 = (int)((int64_t)p.kblocks * t.split / p.splits);
  t.kb1 = (int)((int64_t)p.kblocks * (t.split + 1) / p.splits);
  return t;
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
  const int total_tiles = p.m_tiles * p.n_tiles * p.splits;

  if (warp == 0) {
    // ======================= TMA producer (each CTA loads its own rows of A and its part of B)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int64_t issued = 0;
      bool ok = true;
      for (int tile = unit; tile < total_tiles && ok; tile += nunits) {
        const HeadTile t = head_tile(tile, p);
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
        const HeadTile t = head_tile(tile, p);
        if (!mbar_wait(&tempty[acc], acc_phase ^ 1, abort, p.timeout_ns, p.status)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * BN;
        for (int kb = t.kb0; kb < t.kb1; ++kb) {
          if (!mbar_wait(&full[stage], phase, abort, p.timeout_ns, p.status)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a_addr = smem_addr(sA + stage * kABytes);
          const uint32_t b_addr = smem_addr(sB + stage * kBBytes);
#pragma unroll
          for (int k = 0; k < BK / 16; ++k) {
            const uint64_t ad = kAmn ? desc_mn(a_addr + k * 2048) : desc_k_sw128(a_addr + k * 32);
            const uint64_t bd = kBmn ? desc_mn(b_addr + k * 2048) : desc_k_sw128(b_addr + k * 32);
            const uint32_t accumulate = kb > t.kb0 || k > 0;
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
      const HeadTile t = head_tile(tile, p);
      const int row0 = t.mb * TM + wrow, row = row0 + lane;  // the thread's row of the product
      const int col0 = t.nb * BN + cbase;                    // the warp's first column
      const bool live = row < p.M;
      int tgt = -1;
      float lse2 = 0.0f, g = 0.0f;
      if constexpr (MODE == STATS || MODE == DLOGITS) {
        if (live) tgt = __ldg(p.target + row);
        if constexpr (MODE == DLOGITS) {
          if (live) {
            lse2 = __ldg(p.lse + row) * kLog2e;
            g = p.dloss ? __ldg(p.dloss + row) : __ldg(p.mean + 1);
          }
          if (tgt < 0 || tgt >= p.V) tgt = -1;
          else tgt -= p.b_row0;  // column of this piece
        }
      }
      const bool counts = MODE == DLOGITS && live && __ldg(p.target + row) >= 0 && __ldg(p.target + row) < p.V;
      bool ok = mbar_wait(&tfull[acc], acc_phase, abort, p.timeout_ns, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t t_row = tmem_base + ((uint32_t)(quarter * 32) << 16) + acc * BN + cbase;
      uint32_t nxt[32];
      tmem_ld32(t_row, nxt);
      float mx = -INFINITY, sum = 0.0f;  // STATS: running maximum (of z log2 e) and sum
#pragma unroll 1
      for (int c0 = 0; c0 < kCols; c0 += 32) {
        uint32_t v[32];
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = MODE == DX && t.kb0 == t.kb1 ? 0u : nxt[i];  // a split without K stages
        if (c0 + 32 < kCols) tmem_ld32(t_row + c0 + 32, nxt);
        const int cc = col0 + c0;            // first column of the chunk
        const int cols = p.N - cc;           // columns from there on that exist
        if constexpr (MODE == STATS) {
          if (__any_sync(0xffffffffu, (uint32_t)(tgt - cc) < 32u) && tgt < p.N) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (cc + i == tgt) p.target_logit[row] = __uint_as_float(v[i]);
          }
          float z[32], m = mx;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            z[i] = __uint_as_float(v[i]) * kLog2e;
            if (cols < 32 && i >= cols) z[i] = -INFINITY;
            m = fmaxf(m, z[i]);
          }
          const float base = m == -INFINITY ? 0.0f : m;
          float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            s0 += exp2f(z[i] - base);
            s1 += exp2f(z[i + 1] - base);
          }
          sum = fmaf(sum, exp2f(mx - base), s0 + s1);
          mx = m;
        } else if constexpr (MODE == DLOGITS) {
          uint32_t w[16];
          const int at = tgt - cc;
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float d[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float pr = exp2f(fmaf(__uint_as_float(v[i + e]), kLog2e, -lse2));
              if (tgt >= 0 && i + e == at) pr -= 1.0f;
              d[e] = counts && i + e < cols ? pr * g : 0.0f;
            }
            w[i / 2] = pack2(d[0], d[1]);
          }
#pragma unroll
          for (int q = 0; q < 4; ++q)
            stage_piece(stage, lane, q, make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]));
          // columns past the vocabulary are written too, as zeros: they are K rows of the next products
          flush_rows_64B(stage, lane, static_cast<uint8_t*>(p.out) + ((int64_t)row0 * p.ldo + cc) * 2, p.ldo * 2,
                         p.M - row0);
        } else if (p.out_f32) {
          uint8_t* out = static_cast<uint8_t*>(p.out) +
                         (((int64_t)t.split * p.M + row0) * p.ldo + cc) * 4;
#pragma unroll
          for (int h2 = 0; h2 < 2; ++h2) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              stage_piece(stage, lane, q, make_uint4(v[16 * h2 + 4 * q], v[16 * h2 + 4 * q + 1], v[16 * h2 + 4 * q + 2],
                                                     v[16 * h2 + 4 * q + 3]));
            flush_edge(stage, lane, out + 64 * h2, p.ldo * 4, p.M - row0, (cols - 16 * h2) / 4, MODE == DX && p.add);
          }
        } else {
          uint8_t* out = static_cast<uint8_t*>(p.out) + ((int64_t)row0 * p.ldo + cc) * 2;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            stage_piece(stage, lane, q,
                        make_uint4(pack2(__uint_as_float(v[8 * q]), __uint_as_float(v[8 * q + 1])),
                                   pack2(__uint_as_float(v[8 * q + 2]), __uint_as_float(v[8 * q + 3])),
                                   pack2(__uint_as_float(v[8 * q + 4]), __uint_as_float(v[8 * q + 5])),
                                   pack2(__uint_as_float(v[8 * q + 6]), __uint_as_float(v[8 * q + 7]))));
          flush_edge(stage, lane, out, p.ldo * 2, p.M - row0, cols / 8, false);
        }
      }
      if (MODE == STATS && live) p.part[(int64_t)(2 * t.nb + half) * p.M + row] = make_float2(mx, sum);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2 && !leader) mbar_arrive_cluster_relaxed(tempty_leader + acc * 8);
        else mbar_arrive_relaxed(&tempty[acc]);
      }
      if (++acc == 2) { acc = 0; acc_phase ^= 1; }
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
  const int64_t tiles = (int64_t)p.m_tiles * p.n_tiles * p.splits;
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

HeadParams base_params(DeviceStatus* st) {
  HeadParams p{};
  p.splits = 1;
  p.status = st;
  p.timeout_ns = kTimeoutNs;
  return p;
}

}  // namespace

// Columns of a tile of the logits, for the number of (max, sum) halves.
int head_tile_cols(int T) { return small_tokens(T) ? 128 : 256; }

cudaError_t launch_head_stats(const moe_head_config_t& c, const void* x, const void* w, const int32_t* target,
                              float2* part, float* target_logit, DeviceStatus* st, cudaStream_t s) {
  HeadParams p = base_params(st);
  const bool small = small_tokens(c.T);
  const int bn = head_tile_cols(c.T);
  p.M = c.T;
  p.N = c.V;
  p.V = c.V;
  p.m_tiles = (int)ceil_div(c.T, small ? BM : 2 * BM);
  p.n_tiles = (int)ceil_div(c.V, bn);
  p.kblocks = (int)ceil_div(c.H, BK);
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
                              int ld, void* dx, int splits, bool dx_f32, bool add, void* dw, DeviceStatus* st,
                              cudaStream_t s) {
  const bool small = small_tokens(c.T);
  CUtensorMap a, b;
  HeadParams p = base_params(st);
  const int bn = head_tile_cols(c.T);
  p.M = c.T;
  p.N = rows;
  p.V = c.V;
  p.b_row0 = (int)v0;
  p.m_tiles = (int)ceil_div(c.T, small ? BM : 2 * BM);
  p.n_tiles = (int)ceil_div(rows, bn);
  p.kblocks = (int)ceil_div(c.H, BK);
  p.target = target;
  p.lse = lse;
  p.dloss = dloss;
  p.mean = mean;
  p.out = dl;
  p.ldo = ld;
  if (!bf16_box(&a, x, c.T, c.H, BM) || !bf16_box(&b, w, c.V, c.H, 128)) return cudaErrorInvalidValue;
  cudaError_t e = small ? launch_gemm<DLOGITS, 1, 128>(a, b, p, s) : launch_gemm<DLOGITS, 2, 256>(a, b, p, s);
  if (e != cudaSuccess) return e;
  if (dx) {  // M = T, N = H, K = the piece's vocabulary rows
    p = base_params(st);
    p.M = c.T;
    p.N = c.H;
    p.b_row0 = (int)v0;
    p.m_tiles = (int)ceil_div(c.T, small ? BM : 2 * BM);
    p.n_tiles = (int)ceil_div(c.H, small ? 128 : 256);
    p.kblocks = (int)ceil_div(rows, BK);
    p.splits = splits;
    p.out = dx;
    p.ldo = c.H;
    p.out_f32 = dx_f32;
    p.add = add;
    if (!bf16_box(&a, dl, c.T, ld, BM) || !bf16_box(&b, w, c.V, c.H, 64)) return cudaErrorInvalidValue;
    e = small ? launch_gemm<DX, 1, 128>(a, b, p, s) : launch_gemm<DX, 2, 256>(a, b, p, s);
    if (e != cudaSuccess) return e;
  }
  if (dw) {  // M = the piece's vocabulary rows, N = H, K = T
    p = base_params(st);
    p.M = rows;
    p.N = c.H;
    p.m_tiles = (int)ceil_div(rows, 2 * BM);
    p.n_tiles = (int)ceil_div(c.H, 256);
    p.kblocks = (int)ceil_div(c.T, BK);
    p.out_f32 = c.grad_dtype == MOE_DTYPE_F32;
    p.out = static_cast<uint8_t*>(dw) + v0 * c.H * (p.out_f32 ? 4 : 2);
    p.ldo = c.H;
    if (!bf16_box(&a, dl, c.T, ld, 64) || !bf16_box(&b, x, c.T, c.H, 64)) return cudaErrorInvalidValue;
    e = launch_gemm<DW, 2, 256>(a, b, p, s);
  }
  return e;
}

}  // namespace tc

namespace {

// ---- exact fp32 tiles: 128 x 128 outputs per block, 8 x 8 per thread, K steps of 16
constexpr int ST = 128, SK = 16;

struct SimtParams {
  int M, N, K;
  int splits;                  // DX: K splits
  const void *A, *B;           // operand element (row, k) at row * r + k * k
  int64_t a_row, a_k, b_row, b_k;
  int a_f32, b_f32;            // element types (else bf16)
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

enum { S_STATS = 0, S_DLOGITS = 1, S_STORE = 2 };

template <int MODE>
__global__ void __launch_bounds__(256) simt_kernel(const SimtParams p) {
  __shared__ float sa[SK][ST + 4], sb[SK][ST + 4];
  const int m0 = blockIdx.x * ST, n0 = blockIdx.y * ST;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int k_lo = (int)((int64_t)p.K * blockIdx.z / p.splits), k_hi = (int)((int64_t)p.K * (blockIdx.z + 1) / p.splits);
  float acc[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
  // consecutive threads read along the operand's contiguous direction
  auto fill = [&](float (*dst)[ST + 4], const void* src, int64_t rstep, int64_t kstep, int f32, int r0, int rows, int k0) {
#pragma unroll
    for (int i = 0; i < ST * SK / 256; ++i) {
      const int e = threadIdx.x + i * 256;
      const int r = kstep == 1 ? e / SK : e % ST, k = kstep == 1 ? e % SK : e / ST;
      float v = 0.0f;
      if (r0 + r < rows && k0 + k < k_hi) v = load_elem(src, (int64_t)(r0 + r) * rstep + (int64_t)(k0 + k) * kstep, f32);
      dst[k][r] = v;
    }
  };
  for (int k0 = k_lo; k0 < k_hi; k0 += SK) {
    fill(sa, p.A, p.a_row, p.a_k, p.a_f32, m0, p.M, k0);
    fill(sb, p.B, p.b_row, p.b_k, p.b_f32, n0, p.N, k0);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < SK; ++k) {
      float a[8], b[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = sa[k][ty * 8 + i], b[i] = sb[k][tx + 16 * i];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    __syncthreads();
  }
  // the thread's rows m0 + 8 ty + i, columns n0 + tx + 16 j
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = m0 + ty * 8 + i;
    const bool live = row < p.M;
    if constexpr (MODE == S_STATS) {
      constexpr float kLog2e = 1.4426950408889634f;
      const int tgt = live ? p.target[row] : -1;
      float m = -INFINITY;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int col = n0 + tx + 16 * j;
        if (col < p.N) {
          if (col == tgt) p.target_logit[row] = acc[i][j];
          m = fmaxf(m, acc[i][j] * kLog2e);
        }
      }
#pragma unroll
      for (int off = 8; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
      const float base = m == -INFINITY ? 0.0f : m;
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (n0 + tx + 16 * j < p.N) s += exp2f(fmaf(acc[i][j], kLog2e, -base));
#pragma unroll
      for (int off = 8; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      if (tx == 0 && live) p.part[(int64_t)blockIdx.y * p.M + row] = make_float2(m, s);
    } else if constexpr (MODE == S_DLOGITS) {
      if (live) {
        const int tgt = p.target[row];
        const bool counts = tgt >= 0 && tgt < p.V;
        const float lse = p.lse[row], g = p.dloss ? p.dloss[row] : p.mean[1];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int col = n0 + tx + 16 * j;
          if (col < p.N) {
            float pr = expf(acc[i][j] - lse);
            if (col + p.v0 == tgt) pr -= 1.0f;
            static_cast<float*>(p.out)[(int64_t)row * p.ldo + col] = counts ? pr * g : 0.0f;
          }
        }
      }
    } else if (live) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int col = n0 + tx + 16 * j;
        if (col >= p.N) continue;
        const int64_t at = ((int64_t)blockIdx.z * p.M + row) * p.ldo + col;
        if (p.out_f32) {
          float* o = static_cast<float*>(p.out) + at;
          *o = p.add ? *o + acc[i][j] : acc[i][j];
        } else {
          static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(acc[i][j]);
        }
      }
    }
  }
}

template <int MODE>
cudaError_t launch_simt(const SimtParams& p, cudaStream_t s) {
  simt_kernel<MODE><<<dim3((unsigned)ceil_div(p.M, ST), (unsigned)ceil_div(p.N, ST), (unsigned)p.splits), 256, 0, s>>>(p);
  return cudaGetLastError();
}

// Four tokens per block, 256 lanes of halves each: lse = max + log(sum), the loss, and in the
// block that finishes last their mean over the tokens that count and its reciprocal count.
constexpr int kJoinTokens = 4;
__global__ void __launch_bounds__(1024)
    join_kernel(const float2* part, int parts, int T, int V, const int32_t* target, const float* target_logit,
                float* loss, float* lse, float* mean, uint32_t* ticket, DeviceStatus* st) {
  __shared__ float sm[32][kJoinTokens], ss[32][kJoinTokens];
  __shared__ bool finish;
  const int tok = threadIdx.x & 3, lane = threadIdx.x >> 2, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kJoinTokens + tok;
  float m = -INFINITY, s = 0.0f;
  auto merge = [&](float m2, float s2) {
    const float n = fmaxf(m, m2), base = n == -INFINITY ? 0.0f : n;
    s = fmaf(s, exp2f(m - base), s2 * exp2f(m2 - base));
    m = n;
  };
  if (t < T) {
#pragma unroll 4
    for (int i = lane; i < parts; i += 256) {
      const float2 v = __ldg(part + (int64_t)i * T + t);
      merge(v.x, v.y);
    }
  }
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) merge(__shfl_xor_sync(0xffffffffu, m, off), __shfl_xor_sync(0xffffffffu, s, off));
  if ((threadIdx.x & 31) < kJoinTokens) sm[warp][tok] = m, ss[warp][tok] = s;
  __syncthreads();
  if (warp == 0) {
    m = -INFINITY, s = 0.0f;
    for (int i = lane; i < 32; i += 8) merge(sm[i][tok], ss[i][tok]);
#pragma unroll
    for (int off = 4; off < 32; off <<= 1)
      merge(__shfl_xor_sync(0xffffffffu, m, off), __shfl_xor_sync(0xffffffffu, s, off));
    if (threadIdx.x < kJoinTokens && t < T) {
      const float l = (m + log2f(s)) * 0.6931471805599453f;
      const int32_t tgt = target[t];
      if (tgt >= V) set_status(st, MOE_ERR_DEVICE_BAD_INPUT, (int32_t)t);
      lse[t] = l;
      loss[t] = tgt >= 0 && tgt < V ? l - target_logit[t] : 0.0f;
      __threadfence();
    }
  }
  if (!mean) return;
  __syncthreads();
  if (threadIdx.x == 0) finish = atomicInc(ticket, gridDim.x - 1) == gridDim.x - 1;  // wraps to 0
  __syncthreads();
  if (!finish) return;
  __threadfence();
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
  __shared__ int counts[32];
  if ((threadIdx.x & 31) == 0) sm[warp][0] = sum, counts[warp] = count;
  __syncthreads();
  if (threadIdx.x == 0) {
    double total = 0.0;
    int n = 0;
    for (int i = 0; i < 32; ++i) total += (double)sm[i][0], n += counts[i];
    mean[0] = n ? (float)(total / n) : 0.0f;
    mean[1] = n ? 1.0f / (float)n : 0.0f;
  }
}

// dx = the sum of the K splits' slices [splits][T H], in order.
template <typename T>
__global__ void __launch_bounds__(256) join_dx_kernel(const float* slices, int splits, int64_t n, T* dx) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float v = 0.0f;
  for (int k = 0; k < splits; ++k) v += slices[k * n + i];
  if constexpr (sizeof(T) == 4) dx[i] = v;
  else dx[i] = __float2bfloat16_rn(v);
}

bool head_tc(const moe_head_config_t& c) { return c.act_dtype == MOE_DTYPE_BF16 && c.H % 8 == 0; }

}  // namespace

// A piece holds at most 256 MB of dz unless the caller names its length; whole 256-column
// tiles. The input gradient's K is split where its tiles alone would not fill the SMs.
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
  int64_t tiles, units, most;
  if (tc) {
    const bool small = c.T <= 128;
    tiles = small ? ceil_div(c.H, 128) : ceil_div(T, 256) * ceil_div(c.H, 256);
    units = small ? 152 : 76;
    most = ceil_div(rows, 64) / 8;  // at least 8 K stages a split
  } else {
    tiles = ceil_div(T, ST) * ceil_div(c.H, ST);
    units = 152 * 2;
    most = rows / 64;
  }
  L.splits = (int)std::max<int64_t>(1, std::min<int64_t>({units / tiles, most, 64}));
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
  L.dx = take((size_t)L.splits * T * c.H * 4);
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
    parts = (int)ceil_div(c.V, ST);
    const int f32 = c.act_dtype == MOE_DTYPE_F32;
    SimtParams p{};
    p.M = c.T, p.N = c.V, p.K = c.H, p.splits = 1;
    p.A = x, p.B = w;
    p.a_row = p.b_row = c.H, p.a_k = p.b_k = 1;
    p.a_f32 = p.b_f32 = f32;
    p.target = target, p.part = part, p.target_logit = tl;
    e = launch_simt<S_STATS>(p, s);
  }
  if (e != cudaSuccess) return e;
  // the ticket lives in the head, which moe_workspace_init clears
  join_kernel<<<(unsigned)ceil_div(c.T, kJoinTokens), 1024, 0, s>>>(part, parts, c.T, c.V, target, tl, loss, lse, mean,
                                                                   reinterpret_cast<uint32_t*>(b + 320), st);
  return cudaGetLastError();
}

cudaError_t launch_head_loss_backward(const moe_head_config_t& c, const void* x, const void* w, const int32_t* target,
                                      const float* lse, const float* dloss, const float* mean, void* dx, void* dw,
                                      void* ws, DeviceStatus* st, cudaStream_t s) {
  if (c.T == 0)
    return dw ? cudaMemsetAsync(dw, 0, (size_t)c.V * c.H * (c.grad_dtype == MOE_DTYPE_F32 ? 4 : 2), s) : cudaSuccess;
  const HeadScratch L = head_scratch(c);
  const bool tc = head_tc(c), one = L.piece >= c.V && L.splits == 1;
  char* b = static_cast<char*>(ws);
  float* slices = reinterpret_cast<float*>(b + L.dx);
  const int f32 = c.act_dtype == MOE_DTYPE_F32;
  for (int64_t v0 = 0; v0 < c.V; v0 += L.piece) {
    const int rows = (int)std::min<int64_t>(L.piece, c.V - v0);
    cudaError_t e;
    if (tc) {
      e = tc::launch_head_piece(c, x, w, target, lse, dloss, mean, v0, rows, b + L.dlogits, L.ld,
                                dx ? (one ? dx : slices) : nullptr, L.splits, !one, v0 > 0, dw, st, s);
      if (e != cudaSuccess) return e;
      continue;
    }
    SimtParams p{};
    p.M = c.T, p.N = rows, p.K = c.H, p.splits = 1;
    p.A = x, p.a_row = c.H, p.a_k = 1, p.a_f32 = f32;
    p.B = static_cast<const char*>(w) + v0 * c.H * (f32 ? 4 : 2), p.b_row = c.H, p.b_k = 1, p.b_f32 = f32;
    p.target = target, p.lse = lse, p.dloss = dloss, p.mean = mean, p.v0 = (int)v0, p.V = c.V;
    p.out = b + L.dlogits, p.ldo = L.ld, p.out_f32 = 1;
    if ((e = launch_simt<S_DLOGITS>(p, s)) != cudaSuccess) return e;
    SimtParams q{};
    q.A = b + L.dlogits, q.a_f32 = 1, q.splits = 1;
    if (dx) {
      q.M = c.T, q.N = c.H, q.K = rows, q.splits = L.splits;
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
  const unsigned grid = (unsigned)ceil_div(n, 256);
  if (f32) join_dx_kernel<float><<<grid, 256, 0, s>>>(slices, L.splits, n, static_cast<float*>(dx));
  else join_dx_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(slices, L.splits, n, static_cast<__nv_bfloat16*>(dx));
  return cudaGetLastError();
}

}  // namespace moe
