// Rotary positions: every pair (a, b) of a head's rotated channels turns by angle = pos * f_i,
//   (a, b) -> m (a cos - b sin, b cos + a sin);   backward: by -angle,
// q and k in one launch, with v and a cache's rows to store into where a serving step wants them.
//
// Angles. A frequency is kept as turns per position in 64-bit fixed point (2^64 = one turn), so
// that pos * f modulo a turn is one integer product, exact at any position; what is lost is the
// frequency's own rounding in fp64, 2^-54 of it, times the position (1e-10 turns at 10^6). The
// nearest quarter turn comes off in integers, what is left (an eighth of a turn at most) goes to
// fp32 and two Taylor series. In fp32 the product alone would be off by 0.03 radians at position 10^6.
//
// Memory bound: every element is read and written once. A thread has one place in the heads (two
// pieces of up to 16 bytes: the two halves of lane-wise pairs, or two neighbouring pieces) of one token
// and turns it in up to four heads. The block forms its tokens' cosines and sines once, in shared
// memory, while all loads of the heads are in flight. The piece is the widest power of two that divides
// what is rotated, its place, the head, the row lengths and the addresses. 8192 tokens of 32 + 8 heads of
// 128 with their values: 38 us, 5.3 TB/s; 4095 tokens of 129 heads of 192: 69 us, 5.9 TB/s.
#include "step.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;  // of a block, at most
constexpr int kHeads = 4;      // of a thread, at most

struct RopeParams {
  int T, Hq, Hk, Hv, D, rot, first;
  int slots;
  int items_qk, items_v;      // places of a head
  int groups_qk, groups_v;    // heads are dealt out to this many threads of a place
  int tokens, chunk;          // of a block: tokens, and how many of a token's threads
  float magnitude, sign;
  const void *q, *k, *v;
  void *qo, *ko, *vo;
  int64_t ld_q, ld_k, ld_v, ld_qo, ld_ko, ld_vo;
  const int32_t *pos, *slot;
  const uint64_t* table;
  DeviceStatus* status;
};

template <typename T, int N>
struct alignas(sizeof(T) * N) Piece {
  T v[N];
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float& d, float v) { d = v; }
__device__ __forceinline__ void from_f(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }

// cos and sin of pos * f, both times m. The upper half of pos * f modulo a turn is enough (2^-32 turns);
// the quarter turns come off, and up to an eighth of a turn, x = pi / 4 radians, is left: the sine's
// Taylor series to x^9 leaves 1.8e-9 there, the cosine's to x^10 1.2e-10.
__device__ __forceinline__ float2 turn(int32_t pos, uint64_t f, float m, float sign) {
  const uint32_t n = pos < 0 ? 0u - (uint32_t)pos : (uint32_t)pos;
  if (pos < 0) sign = -sign;
  const uint32_t phase = __umulhi(n, (uint32_t)f) + n * (uint32_t)(f >> 32);
  const uint32_t quarter = (phase + (1u << 29)) >> 30;
  const int32_t rest = (int32_t)(phase - (quarter << 30));  // |rest| <= 2^29
  const float x = __int2float_rn(rest) * 1.4629180792671596e-9f;  // 2 pi / 2^32
  const float z = x * x;
  float s = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
  s = fmaf(z, s, 8.3333333e-3f);
  s = fmaf(z, s, -1.6666667e-1f);
  s = fmaf(x * z, s, x);
  float c = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
  c = fmaf(z, c, -1.3888889e-3f);
  c = fmaf(z, c, 4.1666667e-2f);
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.0f);
  const float cs = quarter & 1 ? s : c, sn = quarter & 1 ? c : s;
  const int q = quarter & 3;
  return make_float2(m * (q == 1 || q == 2 ? -cs : cs), sign * m * (q >= 2 ? -sn : sn));
}

// Two neighbouring elements as fp32, and back with one rounding each.
__device__ __forceinline__ float2 load2(const float* v) { return make_float2(v[0], v[1]); }
__device__ __forceinline__ float2 load2(const __nv_bfloat16* v) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(v));
}
__device__ __forceinline__ void store2(float* v, float a, float b) { v[0] = a, v[1] = b; }
__device__ __forceinline__ void store2(__nv_bfloat16* v, float a, float b) {
  *reinterpret_cast<__nv_bfloat162*>(v) = __floats2bfloat162_rn(a, b);
}

template <typename T, int VEC, bool INTERLEAVED, int HEADS>
__global__ void __launch_bounds__(kThreads, HEADS == 4 ? 7 : HEADS == 3 ? 8 : 12) rope_kernel(const RopeParams p) {
  using P = Piece<T, VEC>;
  constexpr bool kInside = INTERLEAVED && VEC > 1;  // pairs lie inside a piece
  extern __shared__ float2 sTurn[];                 // [tokens][rot / 2]
  const int half = p.rot / 2;
  const int per_qk = p.groups_qk * p.items_qk, per_token = per_qk + p.groups_v * p.items_v;
  const int mine = (int)threadIdx.x / p.chunk;      // the thread's token of the block
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens, t = t0 + mine;
  int r = blockIdx.y * p.chunk + (int)threadIdx.x - mine * p.chunk;
  const bool active = mine < p.tokens && t < p.T && r < per_token;
  const bool value = r >= per_qk;
  if (value) r -= per_qk;
  const int items = value ? p.items_v : p.items_qk, step = value ? p.groups_v : p.groups_qk;
  const int group = r / items, piece = r - group * items;
  const int heads = !active ? 0 : value ? p.Hv : p.Hq + p.Hk;  // none: loads and stores nothing

  // the two pieces' first channels (b < 0: none), and the first pair of table (-1: copied)
  int a, b, pair = -1;
  const int nrot = kInside ? (p.rot / VEC + 1) / 2 : half / VEC;
  if (value) {
    a = piece * 2 * VEC;
    b = a + VEC < p.D ? a + VEC : -1;
  } else if (piece < nrot) {
    pair = piece * VEC;
    a = p.first + (kInside ? piece * 2 * VEC : INTERLEAVED ? 2 * piece : piece * VEC);
    b = kInside ? (a + VEC < p.first + p.rot ? a + VEC : -1) : INTERLEAVED ? a + 1 : a + half;
  } else {
    // the channels that stay, those behind the rotated ones counted on from those before
    const int c = (piece - nrot) * 2 * VEC, c2 = c + VEC;
    a = c < p.first ? c : c + p.rot;
    b = c2 < p.D - p.rot ? (c2 < p.first ? c2 : c2 + p.rot) : -1;
  }
  int64_t row = t;  // of k_out and v_out
  if (p.slot && active) {
    row = __ldg(p.slot + t);
    if (row >= p.slots) {
      if (r == 0) set_status(p.status, MOE_ERR_DEVICE_BAD_INPUT, (int32_t)t);
      row = -1;
    }
  }

  P x[HEADS], y[HEADS];
#pragma unroll
  for (int j = 0; j < HEADS; ++j) {
    const int h = group + j * step;
    if (h < heads) {
      const T* src = value ? static_cast<const T*>(p.v) + t * p.ld_v + (int64_t)h * p.D
                     : h < p.Hq ? static_cast<const T*>(p.q) + t * p.ld_q + (int64_t)h * p.D
                                : static_cast<const T*>(p.k) + t * p.ld_k + (int64_t)(h - p.Hq) * p.D;
      x[j] = *reinterpret_cast<const P*>(src + a);
      if (b >= 0) y[j] = *reinterpret_cast<const P*>(src + b);
    }
  }
  for (int i = threadIdx.x; i < p.tokens * half; i += blockDim.x) {
    const int u = i / half;
    if (t0 + u < p.T) sTurn[i] = turn(__ldg(p.pos + t0 + u), __ldg(p.table + (i - u * half)), p.magnitude, p.sign);
  }
  __syncthreads();
  const float2* cs = sTurn + mine * half + pair;  // of the place's pairs
#pragma unroll
  for (int j = 0; j < HEADS; ++j) {
    const int h = group + j * step;
    if (h >= heads) continue;
    T* dst;
    if (!value && h < p.Hq) dst = static_cast<T*>(p.qo) + t * p.ld_qo + (int64_t)h * p.D;
    else if (row < 0) continue;
    else if (value) dst = static_cast<T*>(p.vo) + row * p.ld_vo + (int64_t)h * p.D;
    else dst = static_cast<T*>(p.ko) + row * p.ld_ko + (int64_t)(h - p.Hq) * p.D;
    if (pair >= 0) {
      if constexpr (kInside) {
        auto rotate = [](T* v, float2 c) {
          const float2 u = load2(v);
          store2(v, u.x * c.x - u.y * c.y, u.y * c.x + u.x * c.y);
        };
#pragma unroll
        for (int l = 0; l < VEC / 2; ++l) {
          rotate(x[j].v + 2 * l, cs[l]);
          if (b >= 0) rotate(y[j].v + 2 * l, cs[VEC / 2 + l]);
        }
      } else if constexpr (VEC > 1) {
#pragma unroll
        for (int l = 0; l < VEC; l += 2) {
          const float2 u = load2(x[j].v + l), w = load2(y[j].v + l), c = cs[l], d = cs[l + 1];
          store2(x[j].v + l, u.x * c.x - w.x * c.y, u.y * d.x - w.y * d.y);
          store2(y[j].v + l, w.x * c.x + u.x * c.y, w.y * d.x + u.y * d.y);
        }
      } else {
        const float u = to_f(x[j].v[0]), w = to_f(y[j].v[0]);
        from_f(x[j].v[0], u * cs->x - w * cs->y);
        from_f(y[j].v[0], w * cs->x + u * cs->y);
      }
    }
    *reinterpret_cast<P*>(dst + a) = x[j];
    if (b >= 0) *reinterpret_cast<P*>(dst + b) = y[j];
  }
}

// Turns per position of every pair. YaRN (Peng et al. 2023): with r = trained_len f / 2 pi whole
// turns within the trained length, f is kept from r = beta_fast on, divided by the factor up to
// r = beta_slow, and mixed linearly in r between (much model code mixes linearly in the pair's index
// instead: its callers fill the table).
__global__ void rope_table_kernel(const moe_rope_freq_t c, uint64_t* table) {
  for (int i = threadIdx.x; i < c.rot / 2; i += blockDim.x) {
    const double turns = pow(c.base, -2.0 * i / c.rot) / 6.283185307179586476925;
    double f = turns;
    if (c.scaling == MOE_ROPE_LINEAR) f = turns / c.factor;
    if (c.scaling == MOE_ROPE_YARN) {
      const double r = c.trained_len * turns;
      const double keep = fmin(1.0, fmax(0.0, (r - c.beta_slow) / (c.beta_fast - c.beta_slow)));
      f = turns * keep + turns / c.factor * (1.0 - keep);
    }
    f -= floor(f);
    table[i] = (uint64_t)__double2ull_rn(f * 18446744073709551616.0);
  }
}

struct Launch {
  dim3 grid;
  unsigned threads;
  size_t smem;
  int heads;
};

template <typename T, int VEC, bool INTERLEAVED>
void launch_heads(const RopeParams& p, const Launch& l, cudaStream_t s) {
  if (l.heads == 4) rope_kernel<T, VEC, INTERLEAVED, 4><<<l.grid, l.threads, l.smem, s>>>(p);
  else if (l.heads == 3) rope_kernel<T, VEC, INTERLEAVED, 3><<<l.grid, l.threads, l.smem, s>>>(p);
  else if (l.heads == 2) rope_kernel<T, VEC, INTERLEAVED, 2><<<l.grid, l.threads, l.smem, s>>>(p);
  else rope_kernel<T, VEC, INTERLEAVED, 1><<<l.grid, l.threads, l.smem, s>>>(p);
}

template <typename T, int VEC>
void launch_vec(const RopeParams& p, int layout, const Launch& l, cudaStream_t s) {
  if (layout == MOE_ROPE_INTERLEAVED) launch_heads<T, VEC, true>(p, l, s);
  else launch_heads<T, VEC, false>(p, l, s);
}

cudaError_t launch(RopeParams p, int layout, bool bf16, cudaStream_t s) {
  const int es = bf16 ? 2 : 4;
  // the widest piece: every place that one may begin at is a multiple of it
  auto fits = [&](int vec) {
    const uint64_t bytes = (uint64_t)vec * es;
    uint64_t at = 0;
    for (const void* q : {p.q, p.k, p.v, (const void*)p.qo, (const void*)p.ko, (const void*)p.vo}) at |= (uint64_t)q;
    for (int64_t ld : {p.ld_q, p.ld_k, p.ld_v, p.ld_qo, p.ld_ko, p.ld_vo}) at |= (uint64_t)ld * es;
    if (at % bytes) return false;
    const int unit = layout == MOE_ROPE_INTERLEAVED ? p.rot : p.rot / 2;
    return p.D % vec == 0 && p.first % vec == 0 && unit % vec == 0;
  };
  int vec = 16 / es;
  while (vec > 1 && !fits(vec)) vec /= 2;
  const bool wide = layout == MOE_ROPE_INTERLEAVED && vec > 1;
  const int nrot = wide ? (p.rot / vec + 1) / 2 : p.rot / 2 / vec;
  p.items_qk = nrot + ((p.D - p.rot) / vec + 1) / 2;
  p.items_v = (p.D / vec + 1) / 2;
  // several heads a thread, where that leaves every SM its threads
  Launch l{};
  int per_token = 0;
  auto deal = [&](int heads) {
    l.heads = heads;
    p.groups_qk = (int)ceil_div(p.Hq + p.Hk, heads);
    p.groups_v = (int)ceil_div(p.Hv, heads);
    per_token = p.groups_qk * p.items_qk + p.groups_v * p.items_v;
  };
  // as many as come out even: 40 heads four at a time take 38 us (8192 tokens with their values) and 47
  // three at a time, 18 heads 33 and 30 us (16384 tokens)
  int best = kHeads;
  for (int h = kHeads - 1; h > 1; --h)
    if (ceil_div(p.Hq + p.Hk, h) * h < ceil_div(p.Hq + p.Hk, best) * best) best = h;
  deal(best);
  if ((int64_t)p.T * per_token < (int64_t)tc::num_sms() * 512) deal(1);
  // whole tokens a block, or a part of one
  p.chunk = min(per_token, kThreads);
  p.tokens = max(1, min(kThreads / p.chunk, 40 * 1024 / max(1, p.rot / 2 * (int)sizeof(float2))));
  l.grid = dim3((unsigned)ceil_div(p.T, p.tokens), (unsigned)ceil_div(per_token, p.chunk));
  l.threads = (unsigned)((p.tokens * p.chunk + 31) / 32 * 32);
  l.smem = (size_t)p.tokens * (p.rot / 2) * sizeof(float2);
  if (l.grid.y > 65535) return cudaErrorInvalidConfiguration;
  if (bf16) {
    if (vec == 8) launch_vec<__nv_bfloat16, 8>(p, layout, l, s);
    else if (vec == 4) launch_vec<__nv_bfloat16, 4>(p, layout, l, s);
    else if (vec == 2) launch_vec<__nv_bfloat16, 2>(p, layout, l, s);
    else launch_vec<__nv_bfloat16, 1>(p, layout, l, s);
  } else {
    if (vec == 4) launch_vec<float, 4>(p, layout, l, s);
    else if (vec == 2) launch_vec<float, 2>(p, layout, l, s);
    else launch_vec<float, 1>(p, layout, l, s);
  }
  return cudaGetLastError();
}

int64_t dense(int64_t ld, int heads, int D) { return ld ? ld : (int64_t)heads * D; }

}  // namespace

cudaError_t launch_rope_table(const moe_rope_freq_t& c, uint64_t* table, cudaStream_t s) {
  rope_table_kernel<<<1, 128, 0, s>>>(c, table);
  return cudaGetLastError();
}

cudaError_t launch_rope(const moe_rope_config_t& c, const void* q, const void* k, const void* v, const int32_t* pos,
                        const int32_t* slot, const uint64_t* table, void* q_out, void* k_out, void* v_out,
                        DeviceStatus* st, cudaStream_t s) {
  RopeParams p{c.T, c.Hq, c.Hk, v_out ? c.Hk : 0, c.D, c.rot, c.first, c.slots};
  p.magnitude = c.magnitude;
  p.sign = 1.0f;
  p.q = q, p.k = k, p.v = v_out ? v : nullptr;
  p.qo = q_out, p.ko = k_out, p.vo = v_out;
  p.ld_q = dense(c.ld_q, c.Hq, c.D), p.ld_k = dense(c.ld_k, c.Hk, c.D);
  p.ld_qo = dense(c.ld_q_out, c.Hq, c.D), p.ld_ko = dense(c.ld_k_out, c.Hk, c.D);
  if (v_out) p.ld_v = dense(c.ld_v, c.Hk, c.D), p.ld_vo = dense(c.ld_v_out, c.Hk, c.D);
  p.pos = pos, p.slot = slot, p.table = table, p.status = st;
  return launch(p, c.layout, c.act_dtype == MOE_DTYPE_BF16, s);
}

cudaError_t launch_rope_backward(const moe_rope_config_t& c, const void* dq_out, const void* dk_out, const int32_t* pos,
                                 const uint64_t* table, void* dq, void* dk, cudaStream_t s) {
  RopeParams p{c.T, c.Hq, c.Hk, 0, c.D, c.rot, c.first, 0};
  p.magnitude = c.magnitude;
  p.sign = -1.0f;
  p.q = dq_out, p.k = dk_out, p.qo = dq, p.ko = dk;
  p.ld_q = dense(c.ld_q_out, c.Hq, c.D), p.ld_k = dense(c.ld_k_out, c.Hk, c.D);
  p.ld_qo = dense(c.ld_q, c.Hq, c.D), p.ld_ko = dense(c.ld_k, c.Hk, c.D);
  p.pos = pos, p.table = table;
  return launch(p, c.layout, c.act_dtype == MOE_DTYPE_BF16, s);
}

}  // namespace moe
