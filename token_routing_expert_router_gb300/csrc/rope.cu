// Rotary positions: every pair (a, b) of a head's rotated channels turns by angle = pos * f_i,
//   (a, b) -> m (a cos - b sin, b cos + a sin);   backward: by -angle,
// q and k in one launch, with v and a cache's rows to store into where a serving step wants them.
//
// Angles. A frequency is kept as turns per position in 64-bit fixed point (2^64 = one turn), so
// that pos * f modulo a turn is one integer product, exact at any position; what is lost is the
// frequency's own rounding in fp64, 2^-54 of it, times the position (1e-10 turns at 10^6). The
// nearest quarter turn comes off in integers, what is left (an eighth of a turn at most) goes to
// fp32 and sincospif. In fp32 the product alone would be off by 0.03 radians at position 10^6.
//
// Memory bound: every element is read and written once, cos and sin are formed once per token and
// pair and shared by all heads through shared memory. An item is two pieces of up to 16 bytes: the
// two halves of lane-wise pairs, or two neighbouring pieces. The piece is the widest power of two
// that divides what is rotated, its place, the head, the row lengths and the addresses.
#include "step.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;  // of a block

struct RopeParams {
  int T, Hq, Hk, Hv, D, rot, first;
  int slots;
  int tokens;           // of a block
  int items_qk, items_v;  // of a head
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

// cos and sin of pos * f, both times m.
__device__ __forceinline__ float2 turn(int32_t pos, uint64_t f, float m, float sign) {
  const uint64_t phase = (uint64_t)(int64_t)pos * f;
  const uint32_t quarter = (uint32_t)((phase + (1ull << 61)) >> 62);
  const int64_t rest = (int64_t)(phase - ((uint64_t)quarter << 62));  // |rest| <= 2^61: an eighth of a turn
  float s, c;
  sincospif(__ll2float_rn(rest) * 0x1p-63f, &s, &c);
  const float cs = quarter & 1 ? s : c, sn = quarter & 1 ? c : s;
  return make_float2(m * (quarter == 1 || quarter == 2 ? -cs : cs), sign * m * (quarter >= 2 ? -sn : sn));
}

template <typename T, int VEC, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  using P = Piece<T, VEC>;
  extern __shared__ float2 sTurn[];  // [tokens][rot / 2]
  __shared__ int sRow[kMaxTokens];   // the row of k_out and v_out, or -1
  const int half = p.rot / 2;
  const int t0 = blockIdx.x * p.tokens, tokens = min(p.tokens, p.T - t0);
  for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
    const int t = i / half;
    sTurn[i] = turn(__ldg(p.pos + t0 + t), __ldg(p.table + (i - t * half)), p.magnitude, p.sign);
  }
  if ((int)threadIdx.x < tokens) {
    int row = t0 + threadIdx.x;
    if (p.slot) {
      row = __ldg(p.slot + row);
      if (row >= p.slots) {
        if (blockIdx.y == 0) set_status(p.status, MOE_ERR_DEVICE_BAD_INPUT, t0 + threadIdx.x);
        row = -1;
      }
    }
    sRow[threadIdx.x] = row;
  }
  __syncthreads();

  const int n_qk = (p.Hq + p.Hk) * p.items_qk, per_token = n_qk + p.Hv * p.items_v;
  const int total = tokens * per_token, step = kThreads * gridDim.y;
  // the first piece that is not rotated, and where the pieces behind the rotated ones begin
  const int nrot = INTERLEAVED && VEC > 1 ? (p.rot / VEC + 1) / 2 : half / VEC;

  struct Item {
    const T *a, *b;
    T *oa, *ob;       // NULL: no such piece
    const float2* cs;  // NULL: copied
  };
  auto locate = [&](int idx) {
    Item it{};
    const int t = idx / per_token;
    int r = idx - t * per_token;
    const T* src;
    T* dst;
    int piece;
    bool plain = false;
    const int64_t row = t0 + t;
    if (r < n_qk) {
      const int h = r / p.items_qk;
      piece = r - h * p.items_qk;
      if (h < p.Hq) {
        src = static_cast<const T*>(p.q) + row * p.ld_q + (int64_t)h * p.D;
        dst = static_cast<T*>(p.qo) + row * p.ld_qo + (int64_t)h * p.D;
      } else {
        src = static_cast<const T*>(p.k) + row * p.ld_k + (int64_t)(h - p.Hq) * p.D;
        dst = sRow[t] < 0 ? nullptr : static_cast<T*>(p.ko) + sRow[t] * p.ld_ko + (int64_t)(h - p.Hq) * p.D;
      }
    } else {
      r -= n_qk;
      const int h = r / p.items_v;
      piece = r - h * p.items_v;
      plain = true;
      src = static_cast<const T*>(p.v) + row * p.ld_v + (int64_t)h * p.D;
      dst = sRow[t] < 0 ? nullptr : static_cast<T*>(p.vo) + sRow[t] * p.ld_vo + (int64_t)h * p.D;
    }
    if (!dst) return it;
    int a, b;  // first channels of the two pieces, b < 0: none
    if (plain) {
      a = piece * 2 * VEC;
      b = a + VEC < p.D ? a + VEC : -1;
    } else if (piece < nrot) {
      it.cs = sTurn + t * half;
      if constexpr (INTERLEAVED) {
        a = p.first + piece * 2 * VEC;
        b = a + VEC < p.first + p.rot ? a + VEC : -1;
        it.cs += piece * VEC;
      } else {
        a = p.first + piece * VEC;
        b = a + half;
        it.cs += piece * VEC;
      }
    } else {
      // the channels that stay, those behind the rotated ones counted on from those before
      const int c = (piece - nrot) * 2 * VEC, left = p.D - p.rot;
      a = c < p.first ? c : c + p.rot;
      const int c2 = c + VEC;
      b = c2 < left ? (c2 < p.first ? c2 : c2 + p.rot) : -1;
    }
    it.a = src + a;
    it.oa = dst + a;
    it.b = b < 0 ? nullptr : src + b;
    it.ob = b < 0 ? nullptr : dst + b;
    return it;
  };
  auto rotate = [&](const Item& it, P& a, P& b) {
    if (!it.cs) return;
    if constexpr (INTERLEAVED && VEC > 1) {
#pragma unroll
      for (int l = 0; l < VEC; l += 2) {
        const float2 cs = it.cs[l / 2];
        const float x = to_f(a.v[l]), y = to_f(a.v[l + 1]);
        from_f(a.v[l], x * cs.x - y * cs.y);
        from_f(a.v[l + 1], y * cs.x + x * cs.y);
      }
      if (it.b) {
#pragma unroll
        for (int l = 0; l < VEC; l += 2) {
          const float2 cs = it.cs[VEC / 2 + l / 2];
          const float x = to_f(b.v[l]), y = to_f(b.v[l + 1]);
          from_f(b.v[l], x * cs.x - y * cs.y);
          from_f(b.v[l + 1], y * cs.x + x * cs.y);
        }
      }
    } else {
#pragma unroll
      for (int l = 0; l < VEC; ++l) {
        const float2 cs = it.cs[l];
        const float x = to_f(a.v[l]), y = to_f(b.v[l]);
        from_f(a.v[l], x * cs.x - y * cs.y);
        from_f(b.v[l], y * cs.x + x * cs.y);
      }
    }
  };

  constexpr int kAhead = 4;  // items whose loads are in flight at once
  for (int base = blockIdx.y * kThreads + threadIdx.x; base < total; base += kAhead * step) {
    Item it[kAhead];
    P a[kAhead], b[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      it[j] = base + j * step < total ? locate(base + j * step) : Item{};
      if (it[j].a) a[j] = *reinterpret_cast<const P*>(it[j].a);
      if (it[j].b) b[j] = *reinterpret_cast<const P*>(it[j].b);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (!it[j].a) continue;
      rotate(it[j], a[j], b[j]);
      *reinterpret_cast<P*>(it[j].oa) = a[j];
      if (it[j].b) *reinterpret_cast<P*>(it[j].ob) = b[j];
    }
  }
}

// Turns per position of every pair. YaRN (Peng et al. 2023): with r = trained_len f / 2 pi whole
// turns within the trained length, f is kept from r = beta_fast on, divided by the factor up to
// r = beta_slow, and mixed linearly between.
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

template <typename T, int VEC>
void launch_vec(const RopeParams& p, int layout, dim3 grid, size_t smem, cudaStream_t s) {
  if (layout == MOE_ROPE_INTERLEAVED) rope_kernel<T, VEC, true><<<grid, kThreads, smem, s>>>(p);
  else rope_kernel<T, VEC, false><<<grid, kThreads, smem, s>>>(p);
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
  const int64_t per_token = (int64_t)(p.Hq + p.Hk) * p.items_qk + (int64_t)p.Hv * p.items_v;
  // a block has about four items a thread; where the tokens are few, several blocks share them
  const int sms = tc::num_sms();
  p.tokens = (int)max((int64_t)1, min((int64_t)kMaxTokens, ceil_div(4 * kThreads, per_token)));
  while (p.tokens > 1 && ceil_div(p.T, p.tokens) < 2 * sms) --p.tokens;
  while (p.tokens > 1 && (size_t)p.tokens * (p.rot / 2) * 8 > 40 * 1024) --p.tokens;
  const int64_t blocks = ceil_div(p.T, p.tokens);
  const int64_t most = ceil_div(per_token * p.tokens, kThreads);
  const int64_t split = max((int64_t)1, min(most, min((int64_t)64, 2 * (int64_t)sms / blocks)));
  const dim3 grid((unsigned)blocks, (unsigned)split);
  const size_t smem = (size_t)p.tokens * (p.rot / 2) * sizeof(float2);
  if (bf16) {
    if (vec == 8) launch_vec<__nv_bfloat16, 8>(p, layout, grid, smem, s);
    else if (vec == 4) launch_vec<__nv_bfloat16, 4>(p, layout, grid, smem, s);
    else if (vec == 2) launch_vec<__nv_bfloat16, 2>(p, layout, grid, smem, s);
    else launch_vec<__nv_bfloat16, 1>(p, layout, grid, smem, s);
  } else {
    if (vec == 4) launch_vec<float, 4>(p, layout, grid, smem, s);
    else if (vec == 2) launch_vec<float, 2>(p, layout, grid, smem, s);
    else launch_vec<float, 1>(p, layout, grid, smem, s);
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
