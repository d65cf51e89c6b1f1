// Launchers of the operators on either side of the MoE layer in a training or serving step:
// block norms (norm.cu), rotary positions (rope.cu), attention (attn*.cu), vocabulary head loss
// (head_loss.cu), token embedding (embed.cu) and gradient clipping (grad_clip.cu). All stream-ordered, no host sync, no allocation.
#pragma once

#include "moe_internal.cuh"
#include "once.h"

namespace moe {

namespace tc {
int num_sms();  // of the current device (gemm_tc.cu)
}

// Words in the workspace head, which moe_workspace_init clears, away from the routing barrier's:
// each returns to what the next call expects, whatever call shared the workspace before.
constexpr size_t kClipState = 1024;   // grad_clip.cu's ticket and scale
constexpr size_t kHeadTicket = 1152;  // head_loss.cu's ticket
constexpr size_t kAttnTickets = 2048; // attention's tickets, up to 456
constexpr size_t kAttnQueue = 3968;   // attn_tc.cu's queue

// Programmatic dependent launch inside a call: a kernel launched with launch_after may be set
// up while the one before it in the stream still runs, and calls after_previous() before it
// touches anything that kernel (or one before it) wrote or read; a kernel that is followed by
// such a launch calls let_next_begin() once. Worth 1 to 2 us per launch of a short chain.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_after_smem(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
  return e != cudaSuccess ? e : cudaGetLastError();
}
template <typename... P, typename... A>
cudaError_t launch_after(void (*kern)(P...), dim3 grid, dim3 block, cudaStream_t s, A... args) {
  return launch_after_smem(kern, grid, block, 0, s, args...);
}

// A kernel's limit of dynamic shared memory, raised before its first launch.
template <typename K>
cudaError_t allow_smem(Once& once, K* kern, size_t smem) {
  return once([&] {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) cudaGetLastError();  // told here, not by the next launch's check as well
    return e;
  });
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

// ---- rotary positions
constexpr int kRopeMaxD = 4096;  // a token's cosines and sines take 16 KB of a block's shared memory
cudaError_t launch_rope_table(const moe_rope_freq_t& c, uint64_t* table, cudaStream_t s);
cudaError_t launch_rope(const moe_rope_config_t& c, const void* q, const void* k, const void* v, const int32_t* pos,
                        const int32_t* slot, const uint64_t* table, void* q_out, void* k_out, void* v_out,
                        DeviceStatus* st, cudaStream_t s);
cudaError_t launch_rope_backward(const moe_rope_config_t& c, const void* dq_out, const void* dk_out, const int32_t* pos,
                                 const uint64_t* table, void* dq, void* dk, cudaStream_t s);

// ---- attention
constexpr int kAttnMaxD = 128;
struct AttnSeqs {  // where the sequences' rows are: k_start and k_len NULL: keys beside their queries
  const int32_t *q_start, *k_start, *k_len;
};
struct AttnScratch {  // workspace offsets, after the status head
  size_t delta;                            // backward, on the FMA units
  size_t neg_lse, neg_delta, dq_plan, dkv_plan;  // backward, on the tensor cores
  size_t plan;                             // forward, tiles
  size_t first;                            // of either plan
  size_t stat;                             // forward, few rows over many keys
  size_t part;                             // parts of either
  size_t total;
};
AttnScratch attn_scratch(const moe_attn_config_t& c, bool backward);
cudaError_t launch_attn(const moe_attn_config_t& c, const void* q, const void* k, const void* v, const AttnSeqs& at,
                        void* o, float* lse, void* ws, DeviceStatus* st, cudaStream_t s);
cudaError_t launch_attn_backward(const moe_attn_config_t& c, const void* q, const void* k, const void* v,
                                 const AttnSeqs& at, const void* o, const float* lse, const void* d_o, void* dq, void* dk,
                                 void* dv, void* ws, DeviceStatus* st, cudaStream_t s);

}  // namespace moe
