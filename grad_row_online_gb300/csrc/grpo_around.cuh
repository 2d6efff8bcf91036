// grpo_around.cuh -- arguments and launches of the entry points around the
// loss: token log-probs and their gradient (grpo_token.cu), the gradient norm
// and clipping (grpo_clip.cu).
#pragma once

#include "grpo_internal.cuh"

namespace grpo {

// grpo_token_logps (grpo_token.cu)
struct TokenArgs {
  const void* logits;
  int64_t B, T, V, sb, st;  // row (b, t) at element b sb + t st
  const int64_t* actions;   // nullable (with logps)
  const uint8_t* mask;      // nullable
  float inv_t;              // s = 1 / temperature
  float s2;                 // s log2(e)
  float low;                // floor of the logits in the fast sweep; 0: none (set at launch)
  int k;
  float* logps;    // nullable
  float* entropy;  // nullable
  float* stats;    // nullable [2, B T]
  int64_t* top_ids;
  float* top_logps;
  WsHeader* hdr;   // nullable
};

// grpo_token_logps_grad (grpo_token.cu)
struct TokenGradArgs {
  const void* logits;
  int64_t B, T, V, sb, st;
  const int64_t* actions;
  const uint8_t* mask;      // nullable
  const float* stats;       // [2, B T]
  const float* entropy;     // nullable (with dent)
  const float* dlogp;       // nullable
  const float* dent;        // nullable
  float inv_t, s2;
  float low;                // as in TokenArgs
  void* grad;
  int64_t gsb, gst;
  int skip_masked;
  WsHeader* hdr;   // nullable
};

// grpo_clip_grad_norm (grpo_clip.cu): host arrays
struct ClipArgs {
  const void* const* tensors;
  void* const* outs;
  const int64_t* numels;
  const int32_t* dtypes;
  int64_t count;
  double max_norm, eps, scale;
  int norm_only;
  float* out2;
  double* partials;
};

cudaError_t launch_token_logps(const TokenArgs& a, grpo_dtype_t dt, cudaStream_t s);
cudaError_t launch_token_grad(const TokenGradArgs& a, grpo_dtype_t dt, cudaStream_t s);
size_t clip_partials(int64_t num_tensors);  // doubles of workspace
cudaError_t launch_clip(const ClipArgs& a, cudaStream_t s);

}  // namespace grpo
