// Tensor-core pieces of the attention kernels (attn_tc.cu, attn_tc_bwd.cu): tiles of [rows, heads,
// channels] tensors by TMA, products with their first operand in tensor memory, packed fp32 pairs.
#pragma once

#include <cudaTypedefs.h>

#include "attn.cuh"
#include "tc_common.cuh"

namespace moe {
namespace tc {
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // gemm_tc.cu
}

namespace attn {

using namespace tc;

constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Box (x, y, z) of a [rows][heads][channels] map: first channel, head, row.
__device__ __forceinline__ void tma_load_3d(const CUtensorMap* m, void* dst, uint64_t* bar, int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// ---- products. A thread's worth of them, but the whole warp comes here and `one` says which lane issues:
// in a branch of a single lane every operand would be moved to a uniform register before every
// instruction, 140 cycles a product of 128 x 128 x 16 where the tensor core takes 64. Descriptors are
// given by their lower word (the address, to which a step adds) and their upper one (the layout).
constexpr uint32_t kRowsDesc = (1024u >> 4) | (1u << 14) | (2u << 29);  // upper word: 128-byte swizzle, 8 rows 1024 bytes apart

// One value of the warp, for the compiler to see.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// Lower word of a K-major operand: a slab of 64 K elements, rows of 128 bytes; 16 K elements are 32 bytes.
__device__ __forceinline__ uint32_t k_desc(uint32_t saddr) { return (saddr >> 4) | (1u << 16); }
// Of an MN-major one: blocks of 64 MN elements 16384 bytes apart, rows (K) of 128 bytes; 16 rows are 2048.
__device__ __forceinline__ uint32_t mn_desc(uint32_t saddr) { return (saddr >> 4) | ((16384u >> 4) << 16); }

// D[tmem] (+)= A[smem] B[smem]
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_desc, uint32_t b_desc, uint32_t idesc, bool accumulate,
                                       bool one) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %4};\n\t"
      "mov.b64 b, {%2, %4};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_desc), "r"(b_desc), "r"(idesc), "r"(kRowsDesc), "r"((uint32_t)accumulate), "r"((uint32_t)one)
      : "memory");
}

// D[tmem] (+)= A[tmem] B[smem]: A is 128 lanes of K elements, two bf16 to a column.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_desc, uint32_t idesc, bool accumulate,
                                       bool one) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %4};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_desc), "r"(idesc), "r"(kRowsDesc), "r"((uint32_t)accumulate), "r"((uint32_t)one)
      : "memory");
}

// The barrier gets an arrival when everything issued before has completed.
__device__ __forceinline__ void commit(uint64_t* bar, bool one) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar)),
      "r"((uint32_t)one)
      : "memory");
}

// The counterpart of tmem_ld32 / tmem_ld16.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 2^x (the PTX instruction, relative error 2^-22).
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// (a, b) -> (a, b) * f + c, as one packed FMA.
__device__ __forceinline__ void scale2(float& a, float& b, float f, float c) {
  asm("{\n\t.reg .b64 x, s, t;\n\t"
      "mov.b64 x, {%0, %1};\n\t"
      "mov.b64 s, {%2, %2};\n\t"
      "mov.b64 t, {%3, %3};\n\t"
      "fma.rn.f32x2 x, x, s, t;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(f), "f"(c));
}
// (a, b) += (x, y)
__device__ __forceinline__ void add2(float& a, float& b, float x, float y) {
  asm("{\n\t.reg .b64 p, q;\n\t"
      "mov.b64 p, {%0, %1};\n\t"
      "mov.b64 q, {%2, %3};\n\t"
      "add.rn.f32x2 p, p, q;\n\t"
      "mov.b64 {%0, %1}, p;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y));
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// Zeros in rows [live, rows) of a tile of `slabs` slabs of 64 channels (rows of 128 bytes), by one
// warp, in the async proxy's sight afterwards: a row that is not the sequence's may hold NaN, and
// would reach a product's sums even times zero.
__device__ __forceinline__ void clear_rows(uint8_t* tile, int slabs, int rows, int live, int lane) {
  for (int s = 0; s < slabs; ++s)
    for (int i = live * 8 + lane; i < rows * 8; i += 32)
      *reinterpret_cast<uint4*>(tile + s * rows * 128 + i * 16) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncwarp();
}

// ---- forward: 128 keys a tile
constexpr int kThreads = 384;
constexpr int BK = 128;
constexpr int kSmem = 227 * 1024;

template <int DP>
struct Fwd {
  static constexpr int kSlabs = DP / 64;
  static constexpr int kTile = 128 * DP * 2;  // bytes of a tile of Q, K or V
  static constexpr int kQ = DP == 64 ? 2 : 1;   // buffers of an item's Q: the next one's where there is room
  static constexpr int kNK = DP == 64 ? 4 : 2, kNV = DP == 64 ? 4 : 3;  // tiles of K and of V
  static constexpr size_t kBytes = 1024 + (2 * kQ + kNK + kNV) * kTile + 512;
  static_assert(kBytes + 1024 <= kSmem);
};

// A row's softmax so far: sums of exp2(c (s - top)), even and odd columns.
struct Running {
  float top = -INFINITY, sum0 = 0.0f, sum1 = 0.0f;
  bool far = false;  // some row of the warp has a maximum beyond 2^24 (base 2)
};

// One tile of scores at my_s (this thread's lane) becomes P. P is rounded to bf16 (2^-8 of it at most): the tensor
// cores take both operands of a product in one type, and V is bf16; the sums are of the exponentials before it. By norm
// o is off by 0.19 to 0.24 %, where its own rounding alone makes 0.17. Columns from `end` on are not seen (the
// whole warp gives BK where every row sees every column). O at my_o is scaled, where it holds anything
// (`begun`) and a row's maximum has grown by more than 2^8.
template <int DP>
__device__ __forceinline__ void softmax_step(uint32_t my_s, uint32_t my_o, float c, int end, bool begun, Running& w) {
  uint32_t r[4][32];
#pragma unroll
  for (int q = 0; q < 4; ++q) tmem_ld32(my_s + 32 * q, r[q]);
  tmem_ld_wait();
  if (__any_sync(0xffffffffu, end < BK)) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int l = 0; l < 32; ++l)
        if (32 * q + l >= end) r[q][l] = 0xff800000u;
  }
  float mx[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    mx[q] = __uint_as_float(r[q][0]);
#pragma unroll
    for (int l = 1; l < 32; ++l) mx[q] = fmaxf(mx[q], __uint_as_float(r[q][l]));
  }
  const float most = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
  const bool grow = most > w.top + 8.0f / c;
  if (__any_sync(0xffffffffu, grow)) {
    const float f = grow ? ex2((w.top - most) * c) : 1.0f;  // 0 for the row's first key
    if (grow) w.top = most;
    w.far = __any_sync(0xffffffffu, w.top != -INFINITY && fabsf(w.top * c) > 0x1p24f);
    w.sum0 *= f, w.sum1 *= f;
    if (begun) {  // the products up to the last tile are in O: these scores were issued behind them
#pragma unroll 1
      for (int col = 0; col < DP; col += 8) {  // few at a time: the scores are in registers
        uint32_t o[8];
        tmem_ld8(my_o + col, o);
        tmem_ld_wait();
#pragma unroll
        for (int l = 0; l < 8; ++l) o[l] = __float_as_uint(__uint_as_float(o[l]) * f);
        tmem_st8(my_o + col, o);
      }
    }
  }
  const float base = w.top == -INFINITY ? 0.0f : -w.top * c;  // no key yet: exp2(-inf) = 0
  // base's rounding is a factor of all the row's exponentials, too large a one where scores are: there the
  // difference is formed first, from the scores as they lie in tensor memory (P goes over those that are read)
  if (w.far) {
    const float least = w.top == -INFINITY ? 0.0f : w.top;
#pragma unroll 1
    for (int col = 0; col < BK; col += 16) {
      uint32_t s[16], v[8];
      tmem_ld16(my_s + col, s);
      tmem_ld_wait();
#pragma unroll
      for (int l = 0; l < 16; l += 2) {
        const float x = col + l < end ? ex2((__uint_as_float(s[l]) - least) * c) : 0.0f;
        const float y = col + l + 1 < end ? ex2((__uint_as_float(s[l + 1]) - least) * c) : 0.0f;
        w.sum0 += x, w.sum1 += y;
        v[l / 2] = pack2(x, y);
      }
      tmem_st8(my_s + col / 2, v);
    }
    tmem_st_wait();
    return;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t v[16];
#pragma unroll
    for (int l = 0; l < 32; l += 2) {
      float x = __uint_as_float(r[q][l]), y = __uint_as_float(r[q][l + 1]);
      scale2(x, y, c, base);
      x = ex2(x), y = ex2(y);
      add2(w.sum0, w.sum1, x, y);
      v[l / 2] = pack2(x, y);
    }
    tmem_st16(my_s + 16 * q, v);
  }
  tmem_st_wait();
}

// Query heads of a group that are packed into a tile's rows: row r is query r / pack, head r % pack.
inline int heads_packed(int group) {
  int p = 1;
  while (p < 128 && group % (2 * p) == 0) p *= 2;
  return p;
}

// A map over rows of `heads` heads of D channels, ld elements apart; boxes of 64 channels, box_heads
// heads, box_rows rows, zeros past the edges.
inline bool head_map(CUtensorMap* m, const void* base, int64_t rows, int heads, int D, int64_t ld, int box_heads, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)ld * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  cuuint32_t estr[3] = {1, 1, 1};
  auto run = [&] {
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  if (run()) return true;
  // a driver call, which needs a current context: a host thread's first CUDA call makes it so
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && run();
}

}  // namespace attn
}  // namespace moe
