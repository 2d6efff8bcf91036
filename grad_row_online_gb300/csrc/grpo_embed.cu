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
#include "grpo_index.cuh"
#include "grpo_vec.cuh"

namespace grpo {
namespace {

__device__ __forceinline__ void launched_early() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A thread takes a vector of `kPer` rows one behind the other, a CTA up to 256
// vectors of them: the rows' loads are in flight together.  A memory-bound copy
// (a scale of 1 leaves a row's bits as they are): 65,536 tokens of 2,048 bf16
// in 61 us, 268 MB written and what of the weight is not in L2 read; 64 tokens
// 4 us, a launch.
template <typename T, int kPer>
__global__ void __launch_bounds__(256) embed_kernel(const EmbedArgs a, int slices) {
  constexpr int kVec = Storage<T>::kVec;
  launched_early();
  const unsigned part = blockIdx.x / (unsigned)slices;
  const int64_t first = (int64_t)part * kPer;
  const int64_t k = ((int64_t)(blockIdx.x - part * slices) * 256 + threadIdx.x) * kVec;
  const int n = (int)min((int64_t)kVec, a.K - k);
  if (n <= 0) return;
  // the first row's (b, t): the others follow it
  int64_t b = 0, t = first;
  if (a.T < a.N) {
    b = (unsigned)first / (unsigned)a.T;
    t = first - b * a.T;
  }
  int64_t id[kPer];  // -1: masked, -2: outside the vocabulary
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int64_t r = first + j;
    const bool on = r < a.N && (!a.mask || a.mask[r]);
    id[j] = on ? a.ids[r] : -1;
    if (on && (id[j] < 0 || id[j] >= a.V)) {
      id[j] = -2;
      if (a.hdr && k == 0) atomicOr(&a.hdr->status, (unsigned)GRPO_ERR_ACTION_RANGE);
    }
  }
  uint4 v[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    v[j] = id[j] >= 0 ? load_vec((const T*)a.weight + id[j] * a.sv + k, n) : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    if (first + j >= a.N) break;
    T* out = (T*)a.out + b * a.sb + t * a.st + k;
    if (a.scale == 1.f && id[j] != -2) {  // (as it lies: a copy)
      store_raw(out, n, v[j]);
    } else {
      float f[kVec];
      Storage<T>::unpack(v[j], f);
#pragma unroll
      for (int i = 0; i < kVec; ++i) f[i] = id[j] == -2 ? __int_as_float(0x7FFFFFFF) : f[i] * a.scale;
      store_vec<T, kVec>(out, n, f);
    }
    if (++t == a.T) t = 0, ++b;
  }
}

// ---------------------------------------------------------------- absent ids
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
  int slices, sums;  // of columns; CTAs that add up
};

// Rows of ids that no token has: zero, or what is added to.  A CTA takes eight
// of them, a thread a vector of four rows at a time.
static constexpr int kAbsentRows = 8, kSumThreads = 128;

template <typename O>
__device__ __forceinline__ void absent_rows(const SumArgs& a, int64_t first) {
  constexpr int kVec = Storage<O>::kVec;
  for (int64_t v0 = first; v0 < min(first + kAbsentRows, a.V); v0 += 4) {
    O* out[4];
    bool go[4];
    int64_t off[4];  // elements of the row's first 16-byte vector before the row
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      go[j] = v0 + j < a.V && !a.taken[v0 + j];
      out[j] = (O*)a.out + (v0 + j) * a.so;
      off[j] = ((uintptr_t)out[j] & 15) / sizeof(O);
    }
    for (int64_t q = (int64_t)threadIdx.x * kVec; q < a.K + kVec; q += kSumThreads * kVec) {
      uint4 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t k = q - off[j];
        x[j] = make_uint4(0, 0, 0, 0);
        if (a.add && go[j] && k >= 0 && k + kVec <= a.K) x[j] = load_vec((const O*)a.add + (v0 + j) * a.sa + k, kVec);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t k = q - off[j];
        if (!go[j]) continue;
        if (k >= 0 && k + kVec <= a.K) {
          __stcs(reinterpret_cast<uint4*>(out[j] + k), x[j]);  // (first to leave L2)
        } else {  // (a row's ends)
          for (int64_t i = max(k, (int64_t)0); i < min(k + kVec, a.K); ++i)
            Storage<O>::store1(out[j] + i, a.add ? Storage<O>::load1((const O*)a.add + (v0 + j) * a.sa + i) : 0.f);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- sort
// Stable sort of (id, token) by id, least significant digits first; tokens
// that take no part get the id V and end behind the others.  A CTA takes a
// chunk, each of its warps a part of that in order.  Digits of up to nine bits:
// two passes for 151,936 words, of two kernels each, 5 to 9 us a kernel,
// latency: counts, a scan over the chunks, then a warp's 32 tokens at a time.
// Up to 4,096 tokens one CTA does all passes in one kernel: the gradient of
// 1,000 tokens of 512 bf16 into 32,000 words takes 22.9 us, 24.9 with a kernel
// a pass.
static constexpr int kMaxDigit = 9;
static_assert(1 << kMaxDigit <= kSortThreads, "a thread has one digit");

struct SortArgs {
  const int64_t* ids;  // first pass: nullptr afterwards
  const uint8_t* mask;
  int64_t V;
  const int2* in;
  int2* out;
  int* hist;  // [chunks][digits]
  unsigned char* taken;  // [V]: ids that occur
  unsigned* status;
  int N, chunk, chunks, shift, bits;
};

// the id that a token is sorted by: V where it takes no part
__device__ __forceinline__ int sort_id(const SortArgs& a, bool on, int64_t id, bool first) {
  if (!on) return (int)a.V;
  if (id < 0 || id >= a.V) {
    if (first && a.status) atomicOr(a.status, (unsigned)GRPO_ERR_ACTION_RANGE);
    return (int)a.V;
  }
  if (first) a.taken[id] = 1;
  return (int)id;
}
// the (id, token) of four rounds of a warp from i on (what is behind `end`: id -1)
__device__ __forceinline__ void sort_keys(const SortArgs& a, int i, int end, bool first,
                                          int2 (&key)[4]) {
  if (!a.ids) {
#pragma unroll
    for (int j = 0; j < 4; ++j) key[j] = i + 32 * j < end ? a.in[i + 32 * j] : make_int2(-1, 0);
    return;
  }
  int64_t id[4];
  bool on[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bool in = i + 32 * j < end;
    id[j] = in ? a.ids[i + 32 * j] : 0;
    on[j] = in && (!a.mask || a.mask[i + 32 * j]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    key[j] = i + 32 * j < end ? make_int2(sort_id(a, on[j], id[j], first), i + 32 * j)
                              : make_int2(-1, 0);
}

// counts of a chunk's digits, of each warp's part of it
__device__ __forceinline__ void count_digits(const SortArgs& a, int (*s)[1 << kMaxDigit],
                                             bool first) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, digits = 1 << a.bits;
  for (int i = threadIdx.x; i < kSortWarps << kMaxDigit; i += kSortThreads) (&s[0][0])[i] = 0;
  const auto [from, end] = sort_part(a.chunk, (int)blockIdx.x, warp, a.N);
  int2 key[4];
  sort_keys(a, from + lane, end, first, key);
  __syncthreads();
  for (int i = from; i < end;) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (key[j].x >= 0) atomicAdd(&s[warp][(key[j].x >> a.shift) & (digits - 1)], 1);
    if ((i += 128) < end) sort_keys(a, i + lane, end, first, key);
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kSortThreads) count_kernel(const SortArgs a) {
  __shared__ int s[kSortWarps][1 << kMaxDigit];
  launched_early();
  count_digits(a, s, true);
  const int d = threadIdx.x, digits = 1 << a.bits;
  if (d >= digits) return;
  int n = 0;
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) n += s[w][d];
  a.hist[blockIdx.x * digits + d] = n;
}

// one pass over this CTA's chunk
__device__ __forceinline__ void place(const SortArgs& a, int (*s)[1 << kMaxDigit], int* s_sum,
                                      bool first) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, digits = 1 << a.bits;
  count_digits(a, s, first);
  // a digit's place: all of smaller digits, its own of earlier chunks, of earlier warps
  const int d = threadIdx.x;
  int all = 0, before = 0;
  if (d < digits) {
    if (a.chunks == 1) {
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) all += s[w][d];
    } else {
#pragma unroll 16
      for (int c = 0; c < a.chunks; ++c) {
        const int n = a.hist[c * digits + d];
        all += n;
        before += c < (int)blockIdx.x ? n : 0;
      }
    }
  }
  int inc = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(~0u, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) s_sum[warp] = inc;
  __syncthreads();
  int at = inc - all + before;
  for (int w = 0; w < warp; ++w) at += s_sum[w];
  if (d < digits) {
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const int n = s[w][d];
      s[w][d] = at;
      at += n;
    }
  }
  __syncthreads();
  const auto [from, end] = sort_part(a.chunk, (int)blockIdx.x, warp, a.N);
  for (int i = from; i < end; i += 128) {
    int2 key[4];
    sort_keys(a, i + lane, end, false, key);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool in = key[j].x >= 0;
      const int digit = in ? (key[j].x >> a.shift) & (digits - 1) : -1;
      const unsigned same = __match_any_sync(~0u, digit);
      const int rank = __popc(same & ((1u << lane) - 1u));
      int to = 0;
      if (in) to = s[warp][digit];
      __syncwarp();
      if (in) {
        a.out[to + rank] = key[j];
        if (rank == 0) s[warp][digit] = to + __popc(same);
      }
      __syncwarp();
    }
  }
}

__global__ void __launch_bounds__(kSortThreads) place_kernel(const SortArgs a) {
  __shared__ int s[kSortWarps][1 << kMaxDigit];
  __shared__ int s_sum[kSortWarps];
  launched_early();
  place(a, s, s_sum, false);
}

// a single chunk: all passes, by way of shared memory
__global__ void __launch_bounds__(kSortThreads) sort_kernel(SortArgs a, int passes) {
  __shared__ int s[kSortWarps][1 << kMaxDigit];
  __shared__ int s_sum[kSortWarps];
  extern __shared__ int2 s_keys[];
  launched_early();
  int2* out = a.out;
  for (int i = 0; i < passes; ++i) {
    a.out = i + 1 == passes ? out : s_keys + (i & 1) * a.chunk;
    place(a, s, s_sum, i == 0);
    __syncthreads();
    a.ids = nullptr;
    a.in = a.out;
    a.shift += a.bits;
  }
}

// ---------------------------------------------------------------- sums
// A CTA adds up a chunk of the sorted tokens, its threads a vector of columns
// each.  An id whose tokens lie in one chunk is done; the parts of one that
// goes on to other chunks are joined by join_kernel in the chunks' order.
// Behind those CTAs come the ones that fill the rows of absent ids.  Bound by
// memory: 38,881 tokens of 2,048 bf16 into 151,936 words, 754 MB, in 117 us
// (6.4 TB/s).  32 tokens a chunk: a frequent id's tokens are spread over as many
// CTAs as they fill chunks, and eight rows' loads are in flight a thread.
static constexpr int kSumChunk = 32;

// kVec elements of what is added to a row, as they lie: one or two vectors
template <typename T, typename O>
struct Addend {
  static constexpr int kVec = Storage<T>::kVec, kOut = Storage<O>::kVec;
  uint4 v[kVec / kOut];
  __device__ __forceinline__ void load(const SumArgs& a, int64_t id, int64_t k, int n) {
    const O* p = (const O*)a.add + id * a.sa + k;
#pragma unroll
    for (int i = 0; i < kVec / kOut; ++i)
      v[i] = n > i * kOut ? load_vec(p + i * kOut, n - i * kOut) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void plus(float* f) const {
#pragma unroll
    for (int i = 0; i < kVec / kOut; ++i) {
      float x[kOut];
      Storage<O>::unpack(v[i], x);
#pragma unroll
      for (int j = 0; j < kOut; ++j) f[i * kOut + j] += x[j];
    }
  }
};

template <typename T, typename O>
__device__ __forceinline__ void finish(const SumArgs& a, int64_t id, int64_t k, int n, float* f,
                                       const Addend<T, O>& add) {
  constexpr int kVec = Storage<T>::kVec;
#pragma unroll
  for (int i = 0; i < kVec; ++i) f[i] *= a.scale;
  if (a.add) add.plus(f);
  store_vec<O, kVec>((O*)a.out + id * a.so + k, n, f);
}

template <typename T, typename O, bool kAdd>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(const SumArgs a) {
  constexpr int kVec = Storage<T>::kVec;
  __shared__ int s_id[kSumChunk + 2];
  __shared__ const T* s_row[kSumChunk];
  launched_early();
  if ((int)blockIdx.x >= a.sums) {
    absent_rows<O>(a, (int64_t)(blockIdx.x - a.sums) * kAbsentRows);
    return;
  }
  const int c = blockIdx.x / a.slices, slice = blockIdx.x - c * a.slices;
  const int from = c * kSumChunk, n = min(kSumChunk, a.N - from);
  if (threadIdx.x < kSumChunk + 2) {
    const int j = (int)threadIdx.x - 1, i = from + j;
    const int2 x = i >= 0 && i < a.N ? a.sorted[i] : make_int2(-1, 0);
    s_id[threadIdx.x] = x.x;
    // (no row: id V, and what lies behind the chunk)
    if (j >= 0 && j < kSumChunk)
      s_row[j] = j < n && x.x < a.V ? (const T*)a.grad + x.y / a.T * a.sb + x.y % a.T * a.st : nullptr;
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
  static_assert(kSumChunk % kAhead == 0, "whole groups");
  for (int j0 = 0; j0 < n; j0 += kAhead) {
    uint4 g[kAhead];
    Addend<T, O> add[kAdd ? kAhead : 1];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const T* row = s_row[j0 + u];
      if (row) g[u] = load_vec(row + k, cols);
      // (an id's last token: what is added is on its way with the rows)
      if (kAdd && row && s_id[2 + j0 + u] != s_id[1 + j0 + u]) add[u].load(a, s_id[1 + j0 + u], k, cols);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = j0 + u;
      if (j >= n) break;
      const int id = s_id[1 + j];
      if (id >= a.V) return;  // (the rest takes no part)
      float h[kVec];
      Storage<T>::unpack(g[u], h);
#pragma unroll
      for (int i = 0; i < kVec; ++i) f[i] += h[i];
      if (j + 1 < n && s_id[2 + j] == id) continue;
      const bool from_before = begin == 0 && s_id[0] == id;
      const bool goes_on = j + 1 == n && s_id[2 + j] == id;
      if (!from_before && !goes_on) {
        finish<T, O>(a, id, k, cols, f, add[kAdd ? u : 0]);
      } else {
        store_vec<float, kVec>(a.parts + ((int64_t)c * 2 + (from_before ? 0 : 1)) * a.K + k, cols, f);
      }
#pragma unroll
      for (int i = 0; i < kVec; ++i) f[i] = 0.f;
      begin = j + 1;
    }
  }
}

// Ids that go on from one chunk to others, each joined from the chunk c where
// it begins: of parts 0 (chunk c's) .. n - 1.
//
// Most have two parts or three: a warp looks at a chunk for one that begins
// there, a lane has a vector of columns.  Ids of more than kLong parts are left
// to the first CTAs, which look for them at kLongChunks chunks each; their four
// warps take a quarter of the parts.  Latency: 10 us for 38,881 tokens of 2,048
// bf16, the most frequent id's; 17 with a CTA for every chunk and 256 columns,
// of which most had little to do and waited for a place.
static constexpr int kLong = 16, kLongChunks = 64;

// the id that begins in chunk c, or before it in the array, and goes on; -1: none
__device__ __forceinline__ int goes_on(const SumArgs& a, int64_t c) {
  const int64_t next = (c + 1) * kSumChunk;
  if (next >= a.N) return -1;
  const int id = a.sorted[next - 1].x, after = a.sorted[next].x;
  const int before = c > 0 ? a.sorted[next - kSumChunk - 1].x : -1;
  return id >= a.V || after != id || before == id ? -1 : id;
}
// whether it ends in chunk c
__device__ __forceinline__ bool ends_in(const SumArgs& a, int id, int64_t c) {
  const int64_t i = (c + 1) * kSumChunk;
  return i >= a.N || a.sorted[i].x != id;
}

template <int kVec>
__device__ __forceinline__ void add_parts(const SumArgs& a, int64_t c, int64_t from, int64_t to, int64_t k,
                                          int cols, float (&f)[kVec]) {
  if (cols == kVec && (a.K & 3) == 0) {
#pragma unroll 4
    for (int64_t d = from; d < to; ++d) {
      const float* q = a.parts + ((c + d) * 2 + (d == 0)) * a.K + k;
#pragma unroll
      for (int i = 0; i < kVec; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(q + i);
        f[i] += v.x, f[i + 1] += v.y, f[i + 2] += v.z, f[i + 3] += v.w;
      }
    }
  } else {
#pragma unroll 4
    for (int64_t d = from; d < to; ++d) {
      const float* q = a.parts + ((c + d) * 2 + (d == 0)) * a.K + k;
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (i < cols) f[i] += q[i];
    }
  }
}

template <typename T, typename O>
__global__ void __launch_bounds__(kSumThreads) join_kernel(const SumArgs a, int slices, int longs) {
  constexpr int kVec = Storage<T>::kVec, kWarps = kSumThreads / 32;
  __shared__ int s_end;
  __shared__ unsigned s_long[kLongChunks / 32];
  __shared__ float s_sum[kWarps][32][kVec];
  launched_early();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float f[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) f[i] = 0.f;
  Addend<T, O> add;
  if ((int)blockIdx.x >= longs) {
    const int64_t u = ((int64_t)blockIdx.x - longs) * kWarps + warp, c = u / slices;
    const int id = goes_on(a, c);
    if (id < 0) return;
    const unsigned ends = __ballot_sync(~0u, lane >= kLong || ends_in(a, id, c + 1 + lane));
    const int parts = __ffs(ends) + 1;
    const int64_t k = ((u - c * slices) * 32 + lane) * kVec;
    const int cols = (int)min((int64_t)kVec, a.K - k);
    if (parts > kLong + 1 || cols <= 0) return;
    if (a.add) add.load(a, id, k, cols);
    add_parts(a, c, 0, parts, k, cols, f);
    finish<T, O>(a, id, k, cols, f, add);
    return;
  }
  const int group = blockIdx.x / slices;
  const int64_t k = ((int64_t)(blockIdx.x - group * slices) * 32 + lane) * kVec;
  const int cols = (int)max((int64_t)0, min((int64_t)kVec, a.K - k));
  if (warp < kLongChunks / 32) {
    const int64_t c = (int64_t)group * kLongChunks + threadIdx.x;
    const int id = goes_on(a, c);
    const unsigned found = __ballot_sync(~0u, id >= 0 && !ends_in(a, id, c + kLong));
    if (lane == 0) s_long[warp] = found;
  }
  __syncthreads();
  for (int w = 0; w < kLongChunks / 32; ++w) {
    for (unsigned left = s_long[w]; left; left &= left - 1) {
      const int64_t c = (int64_t)group * kLongChunks + w * 32 + __ffs(left) - 1;
      const int id = a.sorted[(c + 1) * kSumChunk].x;
      int64_t last = c + 1 + kLong;
      for (;; last += kSumThreads) {
        if (threadIdx.x == 0) s_end = kSumThreads;
        __syncthreads();
        if (ends_in(a, id, last + threadIdx.x)) atomicMin(&s_end, (int)threadIdx.x);
        __syncthreads();
        const int end = s_end;
        __syncthreads();
        if (end < kSumThreads) {
          last += end;
          break;
        }
      }
      const int64_t parts = last - c + 1;
#pragma unroll
      for (int i = 0; i < kVec; ++i) f[i] = 0.f;
      add_parts(a, c, parts * warp / kWarps, parts * (warp + 1) / kWarps, k, cols, f);
#pragma unroll
      for (int i = 0; i < kVec; ++i) s_sum[warp][lane][i] = f[i];
      __syncthreads();
      if (warp != 0 || cols == 0) continue;
#pragma unroll
      for (int v = 1; v < kWarps; ++v)
#pragma unroll
        for (int i = 0; i < kVec; ++i) f[i] += s_sum[v][lane][i];
      if (a.add) add.load(a, id, k, cols);
      finish<T, O>(a, id, k, cols, f, add);
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
  l.chunk = (int)sort_chunk(N);
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

// A launch that may be set up while the one before it ends (its threads wait
// for that before they touch memory).
template <typename... Args>
cudaError_t launch(void (*k)(Args...), int64_t grid, unsigned block, int smem, cudaStream_t s,
                   const Args&... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)grid);
  c.blockDim = dim3(block);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, k, args...);
}

template <typename T, typename O>
cudaError_t sorted_sums(SortArgs p, SumArgs a, const Layout& l, char* ws, cudaStream_t s) {
  constexpr int kCols = kSumThreads * Storage<T>::kVec, kJoin = 32 * Storage<T>::kVec;
  a.slices = (int)((a.K + kCols - 1) / kCols);
  a.sums = l.sums * a.slices;
  cudaError_t e = cudaSuccess;
  if (l.chunks == 1) {
    p.out = (int2*)(ws + l.keys[0]);
    const int smem = (int)sizeof(int2) * l.chunk * std::min(l.passes - 1, 2);
    // (the limit is the function's, in all threads: never less than any call needs)
    constexpr int kMost = (int)sizeof(int2) * kSortOne * 2;
    if ((e = cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost)) != cudaSuccess ||
        (e = launch(sort_kernel, 1, kSortThreads, smem, s, p, l.passes)) != cudaSuccess)
      return e;
    p.in = p.out;
  }
  for (int i = 0; i < l.passes && l.chunks > 1; ++i) {
    p.out = (int2*)(ws + l.keys[i & 1]);
    p.shift = i * l.bits;
    if ((e = launch(count_kernel, l.chunks, kSortThreads, 0, s, p)) != cudaSuccess ||
        (e = launch(place_kernel, l.chunks, kSortThreads, 0, s, p)) != cudaSuccess)
      return e;
    p.ids = nullptr;
    p.in = p.out;
  }
  a.sorted = p.in;
  // (in place, absent ids' rows stay)
  const int absent = a.add == a.out ? 0 : (int)((a.V + kAbsentRows - 1) / kAbsentRows);
  if (a.sums + absent == 0) return cudaSuccess;
  auto* k = a.add ? sum_kernel<T, O, true> : sum_kernel<T, O, false>;
  e = launch(k, (int64_t)a.sums + absent, kSumThreads, 0, s, a);
  if (e != cudaSuccess || l.sums < 2) return e;
  const int joins = (int)((a.K + kJoin - 1) / kJoin);
  // (an id of more than kLong + 1 parts takes as many chunks)
  const int longs = l.sums > kLong + 1 ? (l.sums + kLongChunks - 1) / kLongChunks * joins : 0;
  const int64_t shorts = ((int64_t)l.sums * joins + kSumThreads / 32 - 1) / (kSumThreads / 32);
  return launch(join_kernel<T, O>, longs + shorts, kSumThreads, 0, s, a, joins, longs);
}

template <typename T>
cudaError_t embed(EmbedArgs a, cudaStream_t s) {
  constexpr int kCols = 256 * Storage<T>::kVec;
  const int slices = (int)((a.K + kCols - 1) / kCols);
  if (a.sb == a.T * a.st) a.T = a.N;  // rows evenly apart
  // Rows together where there are enough of them: 2,048 bf16 a row, one a thread
  // and four take 3.8 and 4.4 us for 1,024 tokens, 5.4 and 5.3 for 2,048, 15.1 and
  // 12.4 for 8,192, 104 and 78 for 65,536; 1,021 fp32, 5.5 and 7.6 for 2,048, 8.9
  // and 9.1 for 4,096.
  constexpr int64_t kMany = 2432;
  if (a.N * slices >= kMany) return launch(embed_kernel<T, 4>, (a.N + 3) / 4 * slices, 256, 0, s, a, slices);
  return launch(embed_kernel<T, 1>, a.N * slices, 256, 0, s, a, slices);
}

}  // namespace

size_t embed_ws(int64_t N, int64_t K, int64_t V) { return layout(N, K, V).total; }

cudaError_t launch_embed(const EmbedArgs& a, grpo_dtype_t dt, cudaStream_t s) {
  return dt == GRPO_F32    ? embed<float>(a, s)
         : dt == GRPO_BF16 ? embed<__nv_bfloat16>(a, s)
                           : embed<__half>(a, s);
}

cudaError_t launch_embed_grad(const EmbedGradArgs& a, grpo_dtype_t dt, cudaStream_t s) {
  const Layout l = layout(a.N, a.K, a.V);
  unsigned char* taken = (unsigned char*)(a.ws + l.taken);
  cudaError_t e = cudaMemsetAsync(taken, 0, (size_t)a.V, s);
  if (e != cudaSuccess) return e;
  const SortArgs p{a.ids, a.mask, a.V, nullptr, nullptr, (int*)(a.ws + l.hist), taken,
                   a.hdr ? &a.hdr->status : nullptr, (int)a.N, l.chunk, l.chunks, 0, l.bits};
  const SumArgs g{a.grad, a.K, a.sb, a.st, a.V, (int)a.N, (int)std::max<int64_t>(a.T, 1), nullptr,
                  a.scale, a.add, a.sa, a.out, a.so, (float*)(a.ws + l.parts), taken, 0, 0};
  if (dt == GRPO_F32) return sorted_sums<float, float>(p, g, l, a.ws, s);
  if (dt == GRPO_BF16)
    return a.odt == GRPO_F32 ? sorted_sums<__nv_bfloat16, float>(p, g, l, a.ws, s)
                             : sorted_sums<__nv_bfloat16, __nv_bfloat16>(p, g, l, a.ws, s);
  return a.odt == GRPO_F32 ? sorted_sums<__half, float>(p, g, l, a.ws, s)
                           : sorted_sums<__half, __half>(p, g, l, a.ws, s);
}

}  // namespace grpo
