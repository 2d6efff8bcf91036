// grpo_embed.cuh -- arguments and launches of the token embedding and its
// gradient (grpo_embed.cu).
#pragma once

#include "grpo_internal.cuh"

namespace grpo {

struct EmbedArgs {
  const void* weight;  // [V, K], rows sv apart
  int64_t V, K, sv, N, T;
  const int64_t* ids;
  const uint8_t* mask;  // nullable
  float scale;
  void* out;  // row n = b T + t at element b sb + t st
  int64_t sb, st;
  WsHeader* hdr;  // nullable
};

struct EmbedGradArgs {
  const void* grad;  // row n = b T + t at element b sb + t st
  int64_t V, K, sb, st, N, T;
  const int64_t* ids;
  const uint8_t* mask;  // nullable
  float scale;
  const void* add;  // nullable; [V, K], rows sa apart, of type odt
  int64_t sa;
  void* out;  // [V, K], rows so apart, of type odt
  int64_t so;
  grpo_dtype_t odt;
  WsHeader* hdr;  // nullable
  char* ws;
};

size_t embed_ws(int64_t N, int64_t K, int64_t V);
cudaError_t launch_embed(const EmbedArgs& a, grpo_dtype_t dt, cudaStream_t s);
cudaError_t launch_embed_grad(const EmbedGradArgs& a, grpo_dtype_t dt, cudaStream_t s);

}  // namespace grpo
