// grpo_embed.cu -- the embedding of tokens (grpo_embed_tokens) and its
// gradient by sorted tokens (grpo_embed_tokens_grad).
//
//   out_t = scale W[id_t]
//   dW_v  = add_v + scale sum_{t: id_t = v} g_t      (fp32, t ascending)
//
// The gradient sorts the tokens by id (stable, so equal ids keep their order),
// and adds the rows of each id in registers: no atomics on values, the same
// bits every time.
#include <algorithm>

#include "grpo_embed.cuh"

namespace grpo {
namespace {

// `n` (at most a 16-byte vector's) elements of a row as floats, zeros behind them
template <typename T>
__device__ __forceinline__ void load_vec(const T* p, int n, float* f) {
  constexpr int kVec = Storage<T>::kVec;
  if (n >= kVec && ((uintptr_t)p & 15) == 0) {
    Storage<T>::unpack(__ldg(reinterpret_cast<const uint4*>(p)), f);
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) f[i] = i < n ? Storage<T>::load1(p + i) : 0.f;
  }
}
// kVec floats, `n` of them inside, to a row of O
template <typename O, int kVec>
__device__ __forceinline__ void store_vec(O* p, int n, const float* f) {
  constexpr int kOut = Storage<O>::kVec;
  if (n >= kVec && kVec % kOut == 0 && ((uintptr_t)p & 15) == 0) {
#pragma unroll
    for (int i = 0; i < kVec; i += kOut)
      *reinterpret_cast<uint4*>(p + i) = Storage<O>::pack(f + i);
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (i < n) Storage<O>::store1(p + i, f[i]);
  }
}

// A thread takes a vector of a row, a CTA up to 256 of them.
template <typename T>
__global__ void __launch_bounds__(256) embed_kernel(const EmbedArgs a, int slices) {
  constexpr int kVec = Storage<T>::kVec;
  for (int64_t j = blockIdx.x; j < a.N * slices; j += gridDim.x) {
    const int64_t r = j / slices, k = ((j - r * slices) * 256 + threadIdx.x) * kVec;
    const bool on = !a.mask || a.mask[r];
    const int64_t id = on ? a.ids[r] : -1;
    const bool in = id >= 0 && id < a.V;
    if (on && !in && a.hdr && k == 0) atomicOr(&a.hdr->status, (unsigned)GRPO_ERR_ACTION_RANGE);
    if (k >= a.K) continue;
    const int n = (int)min((int64_t)kVec, a.K - k);
    float f[kVec];
    if (in) {
      load_vec((const T*)a.weight + id * a.sv + k, n, f);
#pragma unroll
      for (int i = 0; i < kVec; ++i) f[i] *= a.scale;
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i) f[i] = on ? __int_as_float(0x7FFFFFFF) : 0.f;
    }
    store_vec<T, kVec>((T*)a.out + r / a.T * a.sb + r % a.T * a.st + k, n, f);
  }
}

// ---------------------------------------------------------------- sort
// Stable sort of (id, token) by id, least significant digits first; tokens
// that take no part get the id V and end behind the others.  A CTA takes a
// chunk, each of its warps a part of that in order.
static constexpr int kSortThreads = 256, kSortWarps = kSortThreads / 32;
static constexpr int kMaxDigit = 9;

struct SortArgs {
  const int64_t* ids;  // first pass: nullptr afterwards
  const uint8_t* mask;
  int64_t V;
  const int2* in;
  int2* out;
  int* hist;  // [digits][chunks]
  unsigned char* taken;  // [V]: ids that occur
  unsigned* status;
  int N, chunk, chunks, shift, bits;
};

__device__ __forceinline__ int2 sort_key(const SortArgs& a, int i, bool first) {
  if (!a.ids) return a.in[i];
  int64_t id = a.V;
  if (!a.mask || a.mask[i]) {
    id = a.ids[i];
    if (id < 0 || id >= a.V) {
      id = a.V;
      if (first && a.status) atomicOr(a.status, (unsigned)GRPO_ERR_ACTION_RANGE);
    } else if (first) {
      a.taken[id] = 1;
    }
  }
  return make_int2((int)id, i);
}

// counts of a chunk's digits, of each warp's part of it
__device__ __forceinline__ void count_digits(const SortArgs& a, int (*s)[1 << kMaxDigit],
                                             bool first) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, digits = 1 << a.bits;
  for (int i = threadIdx.x; i < kSortWarps * digits; i += kSortThreads) s[i / digits][i % digits] = 0;
  __syncthreads();
  const int part = a.chunk / kSortWarps, from = blockIdx.x * a.chunk + warp * part;
  for (int i = from + lane; i < min(from + part, a.N); i += 32)
    atomicAdd(&s[warp][(sort_key(a, i, first).x >> a.shift) & (digits - 1)], 1);
  __syncthreads();
}

__global__ void __launch_bounds__(kSortThreads) count_kernel(const SortArgs a) {
  __shared__ int s[kSortWarps][1 << kMaxDigit];
  count_digits(a, s, true);
  for (int d = threadIdx.x; d < 1 << a.bits; d += kSortThreads) {
    int n = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) n += s[w][d];
    a.hist[d * a.chunks + blockIdx.x] = n;
  }
}

__global__ void __launch_bounds__(kSortThreads) place_kernel(const SortArgs a) {
  __shared__ int s[kSortWarps][1 << kMaxDigit];
  __shared__ int s_base[1 << kMaxDigit], s_before[1 << kMaxDigit], s_sum[kSortWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, digits = 1 << a.bits;
  count_digits(a, s, false);
  // a digit's place: all of smaller digits, its own of earlier chunks
  for (int d = warp; d < digits; d += kSortWarps) {
    int all = 0, before = 0;
    for (int c = lane; c < a.chunks; c += 32) {
      const int n = a.hist[d * a.chunks + c];
      all += n;
      before += c < (int)blockIdx.x ? n : 0;
    }
    all = __reduce_add_sync(~0u, all);
    before = __reduce_add_sync(~0u, before);
    if (lane == 0) s_base[d] = all, s_before[d] = before;
  }
  __syncthreads();
  // exclusive sums of the digits' totals: two digits a thread
  int v[2], sum = 0;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int d = threadIdx.x * 2 + j;
    v[j] = d < digits ? s_base[d] : 0;
    sum += v[j];
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(~0u, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) s_sum[warp] = inc;
  __syncthreads();
  int base = inc - sum;
  for (int w = 0; w < warp; ++w) base += s_sum[w];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int d = threadIdx.x * 2 + j;
    if (d < digits) s_base[d] = base;
    base += v[j];
  }
  __syncthreads();
  for (int d = threadIdx.x; d < digits; d += kSortThreads) {
    int at = s_base[d] + s_before[d];
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const int n = s[w][d];
      s[w][d] = at;
      at += n;
    }
  }
  __syncthreads();
  const int part = a.chunk / kSortWarps, from = blockIdx.x * a.chunk + warp * part;
  const int end = min(from + part, a.N);
  for (int i0 = from; i0 < end; i0 += 32) {
    const int i = i0 + lane;
    const bool in = i < end;
    const int2 key = in ? sort_key(a, i, false) : make_int2(0, 0);
    const int d = in ? (key.x >> a.shift) & (digits - 1) : -1;
    const unsigned same = __match_any_sync(~0u, d);
    const int rank = __popc(same & ((1u << lane) - 1u));
    int at = 0;
    if (in) at = s[warp][d];
    __syncwarp();
    if (in) {
      a.out[at + rank] = key;
      if (rank == 0) s[warp][d] = at + __popc(same);
    }
    __syncwarp();
  }
}

// ---------------------------------------------------------------- sums
// A CTA adds up a chunk of the sorted tokens, its threads a vector of columns
// each.  An id whose tokens lie in one chunk is done; the parts of one that
// goes on to other chunks are joined by join_kernel in the chunks' order.
static constexpr int kSumThreads = 128, kSumChunk = 32;

struct SumArgs {
  const void* grad;
  int64_t K, sb, st;
  int64_t V;
  int N, T;
  const int2* sorted;
  float scale;
  const void* add;
  int64_t sa;
  void* out;
  int64_t so;
  float* parts;  // [chunks][2][K]: of the id that came from before, of the id that goes on
  const unsigned char* taken;
};

template <typename T, typename O>
__device__ __forceinline__ void finish(const SumArgs& a, int64_t id, int64_t k, int n, float* f) {
  constexpr int kVec = Storage<T>::kVec;
  O* out = (O*)a.out + id * a.so + k;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    f[i] *= a.scale;
    if (a.add && i < n) f[i] += Storage<O>::load1((const O*)a.add + id * a.sa + k + i);
  }
  store_vec<O, kVec>(out, n, f);
}

template <typename T, typename O>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(const SumArgs a, int slices) {
  constexpr int kVec = Storage<T>::kVec;
  __shared__ int2 s_tok[kSumChunk + 2];
  const int c = blockIdx.x / slices, slice = blockIdx.x - c * slices;
  const int from = c * kSumChunk, n = min(kSumChunk, a.N - from);
  if (threadIdx.x < kSumChunk + 2) {
    const int i = from + (int)threadIdx.x - 1;
    s_tok[threadIdx.x] = i >= 0 && i < a.N ? a.sorted[i] : make_int2(-1, 0);
  }
  __syncthreads();
  const int64_t k = ((int64_t)slice * kSumThreads + threadIdx.x) * kVec;
  if (k >= a.K) return;
  const int cols = (int)min((int64_t)kVec, a.K - k);
  float f[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) f[i] = 0.f;
  int begin = 0;
  constexpr int kAhead = 8;
  for (int j0 = 0; j0 < n; j0 += kAhead) {
    float g[kAhead][kVec];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int2 t = s_tok[1 + min(j0 + u, n - 1)];
      if (t.x < a.V) load_vec((const T*)a.grad + t.y / a.T * a.sb + t.y % a.T * a.st + k, cols, g[u]);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = j0 + u;
      if (j >= n) break;
      const int id = s_tok[1 + j].x;
      if (id >= a.V) return;  // (the rest takes no part)
#pragma unroll
      for (int i = 0; i < kVec; ++i) f[i] += g[u][i];
      if (j + 1 < n && s_tok[2 + j].x == id) continue;
      const bool from_before = begin == 0 && s_tok[0].x == id;
      const bool goes_on = j + 1 == n && s_tok[2 + j].x == id;
      if (!from_before && !goes_on) {
        finish<T, O>(a, id, k, cols, f);
      } else {
        float* p = a.parts + ((int64_t)c * 2 + (from_before ? 0 : 1)) * a.K + k;
#pragma unroll
        for (int i = 0; i < kVec; ++i)
          if (i < cols) p[i] = f[i];
      }
#pragma unroll
      for (int i = 0; i < kVec; ++i) f[i] = 0.f;
      begin = j + 1;
    }
  }
}

template <typename T, typename O>
__global__ void __launch_bounds__(kSumThreads) join_kernel(const SumArgs a, int slices) {
  constexpr int kVec = Storage<T>::kVec;
  const int c = blockIdx.x / slices, slice = blockIdx.x - c * slices;
  const int next = (c + 1) * kSumChunk;
  if (next >= a.N) return;
  const int id = a.sorted[next - 1].x;
  // only where the id goes on and did not come from before
  if (id >= a.V || a.sorted[next].x != id) return;
  if (c > 0 && a.sorted[c * kSumChunk - 1].x == id) return;
  const int64_t k = ((int64_t)slice * kSumThreads + threadIdx.x) * kVec;
  if (k >= a.K) return;
  const int cols = (int)min((int64_t)kVec, a.K - k);
  float f[kVec];
  const float* p = a.parts + ((int64_t)c * 2 + 1) * a.K + k;
#pragma unroll
  for (int i = 0; i < kVec; ++i) f[i] = i < cols ? p[i] : 0.f;
  for (int d = c + 1;; ++d) {
    p = a.parts + (int64_t)d * 2 * a.K + k;
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (i < cols) f[i] += p[i];
    const int end = (d + 1) * kSumChunk;
    if (end >= a.N || a.sorted[end].x != id) break;
  }
  finish<T, O>(a, id, k, cols, f);
}

// Rows of ids that no token has: zero, or what is added to.
template <typename O>
__global__ void __launch_bounds__(256) absent_kernel(const SumArgs a) {
  constexpr int kVec = Storage<O>::kVec;
  for (int64_t v = blockIdx.x; v < a.V; v += gridDim.x) {
    if (a.taken[v]) continue;
    for (int64_t k = (int64_t)threadIdx.x * kVec; k < a.K; k += 256 * kVec) {
      const int n = (int)min((int64_t)kVec, a.K - k);
      float f[kVec];
#pragma unroll
      for (int i = 0; i < kVec; ++i) f[i] = 0.f;
      if (a.add) load_vec((const O*)a.add + v * a.sa + k, n, f);
      store_vec<O, kVec>((O*)a.out + v * a.so + k, n, f);
    }
  }
}

struct Layout {
  size_t keys[2], hist, taken, parts, total;
  int chunk, chunks, bits, passes, sums;
};

Layout layout(int64_t N, int64_t K, int64_t V) {
  Layout l{};
  int bits = 1;
  while (bits < 31 && (V >> bits) != 0) ++bits;  // ids 0 .. V
  l.passes = (bits + kMaxDigit - 1) / kMaxDigit;
  l.bits = (bits + l.passes - 1) / l.passes;
  // up to 256 chunks of at least 2,048 tokens
  l.chunk = (int)(std::max<int64_t>(2048, (N + 255) / 256) + 255) / 256 * 256;
  l.chunks = (int)((N + l.chunk - 1) / l.chunk);
  l.sums = (int)((N + kSumChunk - 1) / kSumChunk);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align256(bytes);
    return at;
  };
  l.taken = take((size_t)V);
  l.keys[0] = take((size_t)(8 * N));
  l.keys[1] = take((size_t)(8 * N));
  l.hist = take((size_t)(4ll << l.bits) * l.chunks);
  l.parts = take((size_t)(8 * l.sums * K));
  l.total = o;
  return l;
}

template <typename T, typename O>
cudaError_t sums(const SumArgs& a, const Layout& l, cudaStream_t s) {
  if (a.N > 0) {
    constexpr int kCols = kSumThreads * Storage<T>::kVec;
    const int slices = (int)((a.K + kCols - 1) / kCols);
    sum_kernel<T, O><<<(unsigned)(l.sums * slices), kSumThreads, 0, s>>>(a, slices);
    join_kernel<T, O><<<(unsigned)(l.sums * slices), kSumThreads, 0, s>>>(a, slices);
  }
  if (a.add != a.out) absent_kernel<O><<<(unsigned)std::min<int64_t>(a.V, 152 * 16), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t embed_ws(int64_t N, int64_t K, int64_t V) { return layout(N, K, V).total; }

cudaError_t launch_embed(const EmbedArgs& a, grpo_dtype_t dt, cudaStream_t s) {
  const int vec = dt == GRPO_F32 ? 4 : 8;
  const int slices = (int)((a.K + 256 * vec - 1) / (256 * vec));
  const unsigned grid = (unsigned)std::min<int64_t>(a.N * slices, 152 * 32);
  if (dt == GRPO_F32) embed_kernel<float><<<grid, 256, 0, s>>>(a, slices);
  else if (dt == GRPO_BF16) embed_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(a, slices);
  else embed_kernel<__half><<<grid, 256, 0, s>>>(a, slices);
  return cudaGetLastError();
}

cudaError_t launch_embed_grad(const EmbedGradArgs& a, grpo_dtype_t dt, cudaStream_t s) {
  const Layout l = layout(a.N, a.K, a.V);
  unsigned char* taken = (unsigned char*)(a.ws + l.taken);
  cudaError_t e = cudaMemsetAsync(taken, 0, (size_t)a.V, s);
  if (e != cudaSuccess) return e;
  int2* keys[2] = {(int2*)(a.ws + l.keys[0]), (int2*)(a.ws + l.keys[1])};
  SortArgs p{a.ids, a.mask, a.V, nullptr, nullptr, (int*)(a.ws + l.hist), taken,
             a.hdr ? &a.hdr->status : nullptr, (int)a.N, l.chunk, l.chunks, 0, l.bits};
  for (int i = 0; i < l.passes && a.N > 0; ++i) {
    p.out = keys[i & 1];
    p.shift = i * l.bits;
    count_kernel<<<l.chunks, kSortThreads, 0, s>>>(p);
    place_kernel<<<l.chunks, kSortThreads, 0, s>>>(p);
    p.ids = nullptr;
    p.in = p.out;
  }
  SumArgs g{a.grad, a.K, a.sb, a.st, a.V, (int)a.N, (int)std::max<int64_t>(a.T, 1), p.in, a.scale, a.add, a.sa, a.out, a.so,
            (float*)(a.ws + l.parts), taken};
  if (dt == GRPO_F32) return sums<float, float>(g, l, s);
  if (dt == GRPO_BF16)
    return a.odt == GRPO_F32 ? sums<__nv_bfloat16, float>(g, l, s)
                             : sums<__nv_bfloat16, __nv_bfloat16>(g, l, s);
  return a.odt == GRPO_F32 ? sums<__half, float>(g, l, s) : sums<__half, __half>(g, l, s);
}

}  // namespace grpo
