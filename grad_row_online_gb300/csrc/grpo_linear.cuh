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

// fp32 and a handful of tokens (grpo_linear_few.cu): products on the ordinary
// cores, the weight read once by each.
struct FewArgs {
  const void* hidden;
  int64_t T, sb, st;
  const int* idx;    // source row of a row; nullptr: itself
  const int* count;  // rows, on the device; nullptr: N
  int N, rows;       // rows: 1, 2, 4, 8 or 16, at least N
  int first;         // of a launch's rows
  const void* weight;
  int64_t V, K, sv;
  float s2;
  // logits with their online softmax
  const int64_t* actions;  // nullable
  float4* part;            // [CTAs][rpad] of (m, Z, D)
  float* xa;
  int rpad;
  // logits with their gradient
  const float4* coef;  // [rows] of (m, c0, c1, s dlogp)
  const int* target;
  float* d;            // [V][rows]
  // its products
  float* acc;          // [parts][rows][ldacc]; nullptr: dh is not wanted
  int64_t ldacc;
  void* dweight;       // nullptr: not wanted
  int64_t gsv;
  const void* add;
  int64_t asv;
};
int few_rows(grpo_dtype_t dt, int64_t N, int64_t K);  // 0: another form's case
int few_parts(int64_t V, int64_t K, int sms);         // of dh's sums
cudaError_t launch_few_stats(const FewArgs& a, int ctas, cudaStream_t s);
cudaError_t launch_few_grad(const FewArgs& a, int sms, cudaStream_t s);
cudaError_t launch_few_back(const FewArgs& a, int parts, cudaStream_t s);

// bytes of workspace (0: sizes beyond the limits)
size_t linear_ws(const void* weight, grpo_dtype_t dt, int64_t N, int64_t K, int64_t V, int64_t sv,
                 bool backward);
cudaError_t launch_linear_logps(const LinearArgs& a, grpo_dtype_t dt, cudaStream_t s);
cudaError_t launch_linear_grad(const LinearArgs& a, grpo_dtype_t dt, cudaStream_t s);

}  // namespace grpo
