// The attention entry points' choice of variant, and their workspaces.
#include "attn_plan.cuh"

namespace moe {

namespace {

attn::AttnArgs args_of(const moe_attn_config_t& c, const void* q, const void* k, const void* v, const AttnSeqs& at,
                       const void* o, float* lse, DeviceStatus* st) {
  attn::AttnArgs a{};
  a.Tq = c.Tq, a.Tk = c.Tk, a.B = c.B, a.Hq = c.Hq, a.Hkv = c.Hkv, a.D = c.D, a.group = c.Hq / c.Hkv;
  a.causal = c.causal, a.max_q = c.max_q ? c.max_q : c.Tq;
  a.scale = c.scale;
  a.ld_q = c.ld_q ? c.ld_q : (int64_t)c.Hq * c.D;
  a.ld_k = c.ld_k ? c.ld_k : (int64_t)c.Hkv * c.D;
  a.ld_v = c.ld_v ? c.ld_v : (int64_t)c.Hkv * c.D;
  a.ld_o = c.ld_o ? c.ld_o : (int64_t)c.Hq * c.D;
  a.q = q, a.k = k, a.v = v;
  a.q_start = at.q_start, a.k_start = at.k_start, a.k_len = at.k_len;
  a.o = const_cast<void*>(o);
  a.lse = lse;
  a.status = st;
  return a;
}

}  // namespace

namespace attn {

bool tc_rows(const AttnArgs& a, bool backward) {
  uint64_t at = (uint64_t)a.q | (uint64_t)a.k | (uint64_t)a.v | (uint64_t)a.o;
  if (backward) at |= (uint64_t)a.d_o | (uint64_t)a.dq | (uint64_t)a.dk | (uint64_t)a.dv;
  at |= (uint64_t)(2 * a.D) | (uint64_t)(2 * a.ld_q) | (uint64_t)(2 * a.ld_k) | (uint64_t)(2 * a.ld_v) | (uint64_t)(2 * a.ld_o);
  return at % 16 == 0;
}

// Equal shares of all key tiles instead of tiles of 256 rows. Rows: (query, head) pairs of a sequence and pack
// of heads. Measured with 32 query and 8 key heads of 128 (tiles, shares):
//   few rows: 64 requests of 1 query over 2048 keys 107 and 94 us, 1 over 8192 89 and 18, 1 over 128 7 and 9;
//   128 rows: 1 request over 8192 89 and 35, 8 over 8192 96 and 89, 64 over 2048 114 and 121;
//   16 tiles: 64 queries over 8192 121 and 36, over 300 14 and 12;
//   72 tiles: 512 queries over 8192 121 and 97, over 512 16 and 39. The lengths are on the device: shares
//   only where a request may have very many keys, by the room that k has. With few keys in much room that is
//   the wrong side: 512 queries over 512 keys take 18 us in a cache of 4096 rows, 42 in one of 8192 or more.
bool stream_rule(const AttnArgs& a) {
  int pack = 1;
  while (pack < 128 && a.group % (2 * pack) == 0) pack *= 2;
  const int64_t rows = (int64_t)a.max_q * pack;
  const int64_t tiles = (a.Tq / (256 / pack) + a.B) * (int64_t)(a.Hq / pack);
  if (rows <= 64) return true;
  if (rows <= 128) return tiles < 304;
  return tiles <= 24 || (tiles < 76 && a.k_start && a.Tk / 8192 >= a.B);
}

}  // namespace attn

AttnScratch attn_scratch(const moe_attn_config_t& c, bool backward) {
  const attn::AttnArgs a = args_of(c, nullptr, nullptr, nullptr, AttnSeqs{}, nullptr, nullptr, nullptr);
  AttnScratch s{};
  size_t at = kWsHead;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align_up(bytes, 256);
    return here;
  };
  const bool tensor_cores = c.act_dtype == MOE_DTYPE_BF16 && c.D % 8 == 0;  // where rows are aligned
  const size_t DP = c.D <= 64 ? 64 : 128, rows = (size_t)c.Hq * c.Tq;
  if (backward) s.delta = s.neg_delta = take(rows * sizeof(float));
  if (tensor_cores && backward) {
    s.neg_lse = take(rows * sizeof(float));
    s.dq_plan = take(attn::plan_bytes(attn::dq_tiles(a)));
    s.dkv_plan = take(attn::plan_bytes(attn::dkv_tiles(a)));
    s.first = take((size_t)2 * (c.B + 1) * sizeof(int));
    s.part = take((size_t)attn::kMostPieces * 2 * 128 * DP * sizeof(float));
  } else if (tensor_cores) {
    s.plan = take(attn::plan_bytes(attn::forward_tiles(a)));
    s.first = take((size_t)(c.B + 1) * sizeof(int));
    s.stat = take((size_t)2 * attn::kMaxStreamCtas * 128 * sizeof(float2));
    s.part = take((size_t)2 * attn::kMaxStreamCtas * 128 * DP * sizeof(float));
  } else if (!backward && c.act_dtype == MOE_DTYPE_F32) {
    s.stat = take((size_t)attn::kMostFewParts * 16 * sizeof(float2));
    s.part = take((size_t)attn::kMostFewParts * 16 * c.D * sizeof(float));
  }
  s.total = at;
  return s;
}

cudaError_t launch_attn(const moe_attn_config_t& c, const void* q, const void* k, const void* v, const AttnSeqs& at,
                        void* o, float* lse, void* ws, DeviceStatus* st, cudaStream_t s) {
  if (c.Tq == 0 || c.B == 0) return cudaSuccess;
  const attn::AttnArgs a = args_of(c, q, k, v, at, o, lse, st);
  char* b = static_cast<char*>(ws);
  const AttnScratch L = attn_scratch(c, false);
  if (c.act_dtype == MOE_DTYPE_F32 && attn::few_rule(a))
    return attn::launch_few(a, reinterpret_cast<float2*>(b + L.stat), reinterpret_cast<float*>(b + L.part), s);
  if (c.act_dtype != MOE_DTYPE_BF16 || !attn::tc_rows(a, false)) return attn::launch_simt(a, c.act_dtype == MOE_DTYPE_BF16, s);
  if (!attn::stream_rule(a)) return attn::launch_tc(a, reinterpret_cast<attn::TilePlan*>(b + L.plan),
                                                     reinterpret_cast<int*>(b + L.first), reinterpret_cast<int*>(b + kAttnQueue), s);
  return attn::launch_stream(a, {reinterpret_cast<uint32_t*>(b + kAttnTickets), reinterpret_cast<float2*>(b + L.stat),
                                 reinterpret_cast<float*>(b + L.part)}, s);
}

cudaError_t launch_attn_backward(const moe_attn_config_t& c, const void* q, const void* k, const void* v,
                                 const AttnSeqs& at, const void* o, const float* lse, const void* d_o, void* dq, void* dk,
                                 void* dv, void* ws, DeviceStatus* st, cudaStream_t s) {
  if (c.B == 0 || (c.Tq == 0 && c.Tk == 0)) return cudaSuccess;
  attn::AttnArgs a = args_of(c, q, k, v, at, o, const_cast<float*>(lse), st);
  a.d_o = d_o, a.dq = dq, a.dk = dk, a.dv = dv;
  char* b = static_cast<char*>(ws);
  const AttnScratch L = attn_scratch(c, true);
  a.delta = reinterpret_cast<float*>(b + L.delta);
  if (c.act_dtype != MOE_DTYPE_BF16 || !attn::tc_rows(a, true)) return attn::launch_simt_backward(a, c.act_dtype == MOE_DTYPE_BF16, s);
  auto floats = [&](size_t at) { return reinterpret_cast<float*>(b + at); };
  return attn::launch_tc_backward(a, {reinterpret_cast<attn::TilePlan*>(b + L.dq_plan), reinterpret_cast<attn::TilePlan*>(b + L.dkv_plan),
                                      reinterpret_cast<int*>(b + L.first),
                                      floats(L.neg_lse), floats(L.neg_delta), floats(L.part),
                                      reinterpret_cast<uint32_t*>(b + kAttnTickets)}, s);
}

}  // namespace moe
