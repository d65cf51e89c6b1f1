// The C ABI of the operators around the layer (include/moe.h, last section): host-side
// validation and workspace sizes. Nothing here allocates, synchronises or throws.
#include <math.h>

#include "step.cuh"

using namespace moe;

namespace {

bool ok16(const void* p) { return p != nullptr && ((uintptr_t)p & 15u) == 0; }
bool opt16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool act_ok(int32_t d) { return d == MOE_DTYPE_F32 || d == MOE_DTYPE_BF16; }
moe_status_t status_of_launch(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

moe_status_t validate(const moe_norm_config_t* c) {
  if (!c || c->T < 0 || c->H < 1 || !act_ok(c->act_dtype)) return MOE_ERR_INVALID_ARG;
  if (!(c->eps > 0.0f) || !isfinite(c->eps) || !isfinite(c->res_scale)) return MOE_ERR_INVALID_ARG;
  return c->H > kNormMaxH ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

moe_status_t validate(const moe_head_config_t* c) {
  if (!c || c->T < 0 || c->H < 1 || c->V < 1 || c->piece < 0) return MOE_ERR_INVALID_ARG;
  if (!act_ok(c->act_dtype) || !act_ok(c->grad_dtype)) return MOE_ERR_INVALID_ARG;
  // tile and row numbers are 32-bit, with room for a grid's last step
  if (c->T > (1 << 28) || c->H > (1 << 20) || c->V > (1 << 23)) return MOE_ERR_UNSUPPORTED;
  if (ceil_div(c->T, 128) * ceil_div(c->V, 128) > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  return ceil_div(c->T, 128) * ceil_div(c->H, 128) > (1 << 26) ? MOE_ERR_UNSUPPORTED : MOE_OK;  // times 32 splits
}

moe_status_t validate(const moe_embed_config_t* c) {
  if (!c || c->T < 0 || c->H < 1 || c->V < 1 || !isfinite(c->scale)) return MOE_ERR_INVALID_ARG;
  if (!act_ok(c->act_dtype) || !act_ok(c->grad_dtype)) return MOE_ERR_INVALID_ARG;
  if (c->T > (1 << 30) || c->H > (1 << 20) || c->V > kEmbedMaxV) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status_t validate(const moe_grad_t* g, int32_t count) {
  if (count < 0 || (count > 0 && !g)) return MOE_ERR_INVALID_ARG;
  for (int32_t i = 0; i < count; ++i) {
    if (g[i].n < 0 || !act_ok(g[i].dtype)) return MOE_ERR_INVALID_ARG;
    if (g[i].n == 0) continue;
    const uintptr_t mask = g[i].dtype == MOE_DTYPE_BF16 ? 1 : 3;
    if (!g[i].grad || ((uintptr_t)g[i].grad & mask) || ((uintptr_t)g[i].out & mask)) return MOE_ERR_INVALID_ARG;
    if (g[i].n > ((int64_t)1 << 40)) return MOE_ERR_UNSUPPORTED;
  }
  return MOE_OK;
}

DeviceStatus* word(void* ws) { return static_cast<DeviceStatus*>(ws); }

moe_status_t clip(const moe_grad_t* grads, int32_t count, float max_norm, float* norm, void* ws, moe_stream_t stream) {
  const moe_status_t v = validate(grads, count);
  if (v != MOE_OK) return v;
  if (!ok16(norm) || !ok16(ws)) return MOE_ERR_INVALID_ARG;
  return status_of_launch(launch_grad_clip(grads, count, max_norm, norm, ws, word(ws), (cudaStream_t)stream));
}

}  // namespace

extern "C" {

moe_status_t moe_block_norm(const moe_norm_config_t* cfg, const void* x, const void* y, const float* w_post,
                            const float* w_next, const float* gate, const float* token_gate, void* r, void* n,
                            moe_stream_t stream) {
  const moe_status_t v = validate(cfg);
  if (v != MOE_OK) return v;
  if ((!r && !n) || (n && !w_next) || (!y && (w_post || gate || token_gate))) return MOE_ERR_INVALID_ARG;
  if (cfg->T == 0) return MOE_OK;
  if (!ok16(x) || !opt16(y) || !opt16(w_post) || !opt16(w_next) || !opt16(gate) || !opt16(token_gate) || !opt16(r) ||
      !opt16(n))
    return MOE_ERR_INVALID_ARG;
  const NormIn in{x, y, w_post, w_next, gate, token_gate};
  return status_of_launch(launch_block_norm(*cfg, in, r, n, (cudaStream_t)stream));
}

moe_status_t moe_block_norm_workspace_size(const moe_norm_config_t* cfg, size_t* bytes) {
  const moe_status_t v = validate(cfg);
  if (v != MOE_OK) return v;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = kWsHead + align_up(norm_part_bytes(*cfg), 256);
  return MOE_OK;
}

moe_status_t moe_block_norm_backward(const moe_norm_config_t* cfg, const void* r, const void* y, const float* w_post,
                                     const float* w_next, const float* gate, const float* token_gate, const void* dr,
                                     const void* dn, void* dx, void* dy, const moe_norm_grads_t* grads, void* ws,
                                     moe_stream_t stream) {
  const moe_status_t v = validate(cfg);
  if (v != MOE_OK) return v;
  const moe_norm_grads_t g = grads ? *grads : moe_norm_grads_t{};
  const bool columns = g.dw_post || g.dw_next || g.dgate;
  if (!y && (w_post || gate || token_gate || dy || g.dw_post || g.dgate || g.dtoken_gate)) return MOE_ERR_INVALID_ARG;
  if ((dn != nullptr) != (w_next != nullptr) && cfg->T > 0) return MOE_ERR_INVALID_ARG;
  if ((g.dw_post && !w_post) || (g.dw_next && !w_next)) return MOE_ERR_INVALID_ARG;
  if (!opt16(g.dw_post) || !opt16(g.dw_next) || !opt16(g.dgate) || !opt16(g.dtoken_gate)) return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 && (!opt16(r) || !opt16(y) || !opt16(w_post) || !opt16(w_next) || !opt16(gate) || !opt16(token_gate) ||
                     !opt16(dr) || !opt16(dn) || !opt16(dx) || !opt16(dy) || (w_next && !r) || (!dr && !dn) ||
                     (columns && !ok16(ws))))
    return MOE_ERR_INVALID_ARG;
  NormBwd b{r, y, w_post, w_next, gate, token_gate, dr, dn, dx, dy, g.dw_post, g.dw_next, g.dgate, g.dtoken_gate};
  float* part = columns ? reinterpret_cast<float*>(static_cast<char*>(ws) + kWsHead) : nullptr;
  return status_of_launch(launch_block_norm_backward(*cfg, b, part, (cudaStream_t)stream));
}

moe_status_t moe_head_workspace_size(const moe_head_config_t* cfg, size_t* bytes) {
  const moe_status_t v = validate(cfg);
  if (v != MOE_OK) return v;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = head_scratch(*cfg).total;
  return MOE_OK;
}

moe_status_t moe_head_loss(const moe_head_config_t* cfg, const void* x, const void* w, const int32_t* target,
                           float* loss, float* lse, float* mean, void* ws, moe_stream_t stream) {
  const moe_status_t v = validate(cfg);
  if (v != MOE_OK) return v;
  if (!opt16(mean)) return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 && (!ok16(x) || !ok16(w) || !ok16(target) || !ok16(loss) || !ok16(lse) || !ok16(ws)))
    return MOE_ERR_INVALID_ARG;
  return status_of_launch(launch_head_loss(*cfg, x, w, target, loss, lse, mean, ws, word(ws), (cudaStream_t)stream));
}

moe_status_t moe_head_loss_backward(const moe_head_config_t* cfg, const void* x, const void* w, const int32_t* target,
                                    const float* lse, const float* dloss, const float* mean, void* dx, void* dw,
                                    void* ws, moe_stream_t stream) {
  const moe_status_t v = validate(cfg);
  if (v != MOE_OK) return v;
  if (!opt16(dx) || !opt16(dw) || (!dx && !dw)) return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 && (!ok16(x) || !ok16(w) || !ok16(target) || !ok16(lse) || !ok16(ws) || !opt16(dloss) || !opt16(mean) ||
                     (dloss != nullptr) == (mean != nullptr)))
    return MOE_ERR_INVALID_ARG;
  return status_of_launch(
      launch_head_loss_backward(*cfg, x, w, target, lse, dloss, mean, dx, dw, ws, word(ws), (cudaStream_t)stream));
}

moe_status_t moe_embed(const moe_embed_config_t* cfg, const void* table, const int32_t* token, void* out, void* ws,
                       moe_stream_t stream) {
  const moe_status_t v = validate(cfg);
  if (v != MOE_OK) return v;
  if (cfg->T == 0) return MOE_OK;
  if (!ok16(table) || !ok16(token) || !ok16(out) || !ok16(ws)) return MOE_ERR_INVALID_ARG;
  return status_of_launch(launch_embed(*cfg, table, token, out, word(ws), (cudaStream_t)stream));
}

moe_status_t moe_embed_workspace_size(const moe_embed_config_t* cfg, size_t* bytes) {
  const moe_status_t v = validate(cfg);
  if (v != MOE_OK) return v;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = embed_scratch(*cfg).total;
  return MOE_OK;
}

moe_status_t moe_embed_backward(const moe_embed_config_t* cfg, const int32_t* token, const void* dout, void* dtable,
                                int32_t accumulate, void* ws, moe_stream_t stream) {
  const moe_status_t v = validate(cfg);
  if (v != MOE_OK) return v;
  if ((accumulate != 0 && accumulate != 1) || !ok16(dtable)) return MOE_ERR_INVALID_ARG;
  if (cfg->T > 0 && (!ok16(token) || !ok16(dout) || !ok16(ws))) return MOE_ERR_INVALID_ARG;
  return status_of_launch(
      launch_embed_backward(*cfg, token, dout, dtable, accumulate, ws, word(ws), (cudaStream_t)stream));
}

moe_status_t moe_grad_clip_workspace_size(int32_t count, size_t* bytes) {
  if (count < 0 || !bytes) return MOE_ERR_INVALID_ARG;
  *bytes = grad_clip_ws_bytes(count);
  return MOE_OK;
}

moe_status_t moe_grad_norm(const moe_grad_t* grads, int32_t count, float* norm, void* ws, moe_stream_t stream) {
  return clip(grads, count, -1.0f, norm, ws, stream);
}

moe_status_t moe_grad_clip(const moe_grad_t* grads, int32_t count, float max_norm, float* norm, void* ws,
                           moe_stream_t stream) {
  if (!(max_norm > 0.0f) || !isfinite(max_norm)) return MOE_ERR_INVALID_ARG;
  return clip(grads, count, max_norm, norm, ws, stream);
}

}  // extern "C"
