// grpo_linear.cuh -- arguments and launches of the head's log-probs from
// hidden states and their gradient (grpo_linear.cu).
#pragma once

#include "grpo_internal.cuh"

namespace grpo {

struct LinearArgs {
  const void* hidden;  // row (b, t) at element b sb + t st
  const void* weight;  // [V, K], rows sv apart
  int64_t B, T, K, V, sb, st, sv;
  const int64_t* actions;  // nullable
  const uint8_t* mask;     // nullable
  float inv_t;             // s = 1 / temperature
  float s2;                // s log2(e)
  WsHeader* hdr;           // nullable
  char* ws;
  // grpo_linear_logps
  float* logps;    // nullable
  float* entropy;  // nullable
  float* stats;    // nullable [2, B T]
  // grpo_linear_logps_grad
  const float* in_stats;    // [2, B T]
  const float* in_entropy;  // nullable (with dent)
  const float* dlogp;       // nullable
  const float* dent;        // nullable
  void* dhidden;            // nullable; row (b, t) at b gsb + t gst
  int64_t gsb, gst;
  void* dweight;  // nullable; rows gsv apart, of type wdt
  int64_t gsv;
  const void* add;  // nullable; rows asv apart, of type wdt
  int64_t asv;
  grpo_dtype_t wdt;
  int skip_masked;
};

// bytes of workspace (0: sizes beyond the limits)
size_t linear_ws(const void* weight, grpo_dtype_t dt, int64_t N, int64_t K, int64_t V, int64_t sv,
                 bool backward);
cudaError_t launch_linear_logps(const LinearArgs& a, grpo_dtype_t dt, cudaStream_t s);
cudaError_t launch_linear_grad(const LinearArgs& a, grpo_dtype_t dt, cudaStream_t s);

}  // namespace grpo
