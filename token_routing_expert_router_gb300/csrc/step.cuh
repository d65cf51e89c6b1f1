// Launchers of the operators on either side of the MoE layer in a training or serving step:
// block norms (norm.cu), vocabulary head loss (head_loss.cu), token embedding (embed.cu) and
// gradient clipping (grad_clip.cu). All stream-ordered, no host sync, no allocation.
#pragma once

#include "moe_internal.cuh"

namespace moe {

namespace tc {
int num_sms();  // of the current device (gemm_tc.cu)
}

// Words in the workspace head, which moe_workspace_init clears, away from the routing barrier's:
// each returns to what the next call expects, whatever call shared the workspace before.
constexpr size_t kClipState = 1024;   // grad_clip.cu's ticket and scale
constexpr size_t kHeadTicket = 1152;  // head_loss.cu's ticket

// Programmatic dependent launch inside a call: a kernel launched with launch_after may be set
// up while the one before it in the stream still runs, and calls after_previous() before it
// touches anything that kernel (or one before it) wrote or read; a kernel that is followed by
// such a launch calls let_next_begin() once. Worth 1 to 2 us per launch of a short chain.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_after(void (*kern)(P...), dim3 grid, dim3 block, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// ---- block norms
struct NormIn {
  const void *x, *y;                                  // [T, H] act; y may be NULL
  const float *w_post, *w_next, *gate, *token_gate;   // [H], [H], [H], [T]; each may be NULL
};
struct NormBwd {
  const void *r, *y;               // the forward's new residual and block output
  const float *w_post, *w_next, *gate, *token_gate;
  const void *dr, *dn;             // either may be NULL
  void *dx, *dy;                   // either may be NULL
  float *dw_post, *dw_next, *dgate, *dtoken_gate;  // each may be NULL
};
constexpr int kNormMaxH = 16384;
cudaError_t launch_block_norm(const moe_norm_config_t& c, const NormIn& in, void* r, void* n, cudaStream_t s);
size_t norm_part_bytes(const moe_norm_config_t& c);  // column partial sums of the backward
cudaError_t launch_block_norm_backward(const moe_norm_config_t& c, const NormBwd& b, float* part, cudaStream_t s);

// ---- token embedding
struct EmbedScratch {  // workspace offsets, after the status head
  size_t count, block_count, keys, stoken, spos, mpos, part, total;
};
constexpr int kEmbedMaxV = (1 << 21) - 1;  // a token and its place in a block of 2048 share 32 bits
EmbedScratch embed_scratch(const moe_embed_config_t& c);
cudaError_t launch_embed(const moe_embed_config_t& c, const void* table, const int32_t* token, void* out,
                         DeviceStatus* st, cudaStream_t s);
cudaError_t launch_embed_backward(const moe_embed_config_t& c, const int32_t* token, const void* dout, void* dtable,
                                  int accumulate, void* ws, DeviceStatus* st, cudaStream_t s);

// ---- gradient clipping
size_t grad_clip_ws_bytes(int32_t count);
// max_norm < 0: the norm alone
cudaError_t launch_grad_clip(const moe_grad_t* grads, int32_t count, float max_norm, float* norm, void* ws,
                             DeviceStatus* st, cudaStream_t s);

// ---- vocabulary head loss
struct HeadScratch {  // workspace offsets, after the status head
  size_t part, target_logit, plan, index, x, w, dlogits, dx, slices, total;
  int64_t piece;   // vocabulary rows whose logit gradients are held at once
  int ld;          // row length of dlogits
};
HeadScratch head_scratch(const moe_head_config_t& c);
cudaError_t launch_head_loss(const moe_head_config_t& c, const void* x, const void* w, const int32_t* target,
                             float* loss, float* lse, float* mean, void* ws, DeviceStatus* st, cudaStream_t s);
cudaError_t launch_head_loss_backward(const moe_head_config_t& c, const void* x, const void* w, const int32_t* target,
                                      const float* lse, const float* dloss, const float* mean, void* dx, void* dw,
                                      void* ws, DeviceStatus* st, cudaStream_t s);

}  // namespace moe
