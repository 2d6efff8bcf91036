// grpo_clip.cu -- the global norm of many gradient tensors, and clipping.
//
//   norm = scale sqrt(sum g^2),  c = scale min(1, max_norm / (norm + eps)),
//   out = c g
//
// The tensors' pointers and sizes go to the kernels as launch parameters (a
// table of up to 32 KB): nothing is copied to the device and nothing is kept
// from one call for the next.
//
//   clip_norm_kernel   every CTA sums the squares of its chunks into one
//                      double of the workspace
//   clip_scale_kernel  every CTA adds all those doubles in one fixed order,
//                      which gives it c, and scales its chunks
// Both read at memory speed: a chunk is cut from one tensor, its elements
// taken as 16-byte vectors where the tensor's alignment allows.
#include "grpo_internal.cuh"

namespace grpo {

static constexpr int kClipThreads = 256;
static constexpr int kClipCtasPerSm = 4;
static constexpr int kClipMaxGrid = 1024;
// elements of a chunk: 64 a thread, which one fp32 sum of squares covers
static constexpr int64_t kClipChunk = 64 * kClipThreads;

struct ClipEntry {
  const void* in;
  void* out;
  unsigned long long n;  // elements, and the type in the two top bits
  unsigned chunk0;       // the entry's first chunk among the table's
  unsigned pad_;
};
template <int kCap>
struct ClipTable {
  int count;
  unsigned chunks;
  ClipEntry e[kCap];
};
// Two table sizes: a launch costs what its parameters take to copy.
static constexpr int kClipFew = 64;
static constexpr int kClipMany = 1000;
static_assert(sizeof(ClipTable<kClipMany>) + 64 <= 32764, "kernel parameters end at 32,764 bytes");

// The entry that holds chunk c, at or after entry i.
template <int kCap>
__device__ __forceinline__ int find_entry(const ClipTable<kCap>& t, unsigned c, int i) {
  int lo = i, hi = t.count;  // e[lo].chunk0 <= c < e[hi].chunk0
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (t.e[mid].chunk0 <= c) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <typename T>
struct ClipChunk {
  const T* in;
  T* out;
  int n, head, nvec, t0;
  __device__ ClipChunk(const ClipEntry& e, unsigned c) {
    const int64_t at = (int64_t)(c - e.chunk0) * kClipChunk;
    const int64_t size = (int64_t)(e.n & ((1ull << 62) - 1));
    in = (const T*)e.in + at;
    out = (T*)e.out + at;
    n = (int)(size - at < kClipChunk ? size - at : kClipChunk);
    head = (int)(((16 - ((uintptr_t)in & 15)) & 15) / sizeof(T));
    if (head > n) head = n;
    nvec = (n - head) / Storage<T>::kVec;
    t0 = head + nvec * Storage<T>::kVec;
  }
};

__device__ __forceinline__ float clip_load(const float* p) { return *p; }
__device__ __forceinline__ float clip_load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float clip_load(const __half* p) { return __half2float(*p); }

// This thread's part of a chunk's sum of squares.  The fp32 sum is taken
// where it lies well inside the range (or the elements are all zero); a sum
// that overflowed, or so small that squares were lost below the range, is
// formed again in double.
template <typename T>
__device__ double chunk_squares(const ClipChunk<T>& k) {
  constexpr int VEC = Storage<T>::kVec;
  constexpr int kVecs = (int)(kClipChunk / kClipThreads) / VEC;  // vectors a thread at most
  const int tid = threadIdx.x;
  const uint4* vec = reinterpret_cast<const uint4*>(k.in + k.head);
  float s = 0.f;
  unsigned any = 0;
  const bool edge = tid < k.head + (k.n - k.t0);
  const int ev = tid < k.head ? tid : k.t0 + tid - k.head;
  if (edge) {
    const float x = clip_load(k.in + ev);
    any = x != 0.f;
    s = x * x;
  }
#pragma unroll 4
  for (int i = 0; i < kVecs; ++i) {
    const int j = tid + i * kClipThreads;
    if (j >= k.nvec) break;
    const uint4 v = vec[j];
    float x[VEC];
    Storage<T>::unpack(v, x);
    any |= v.x | v.y | v.z | v.w;
#pragma unroll
    for (int e = 0; e < VEC; ++e) s = fmaf(x[e], x[e], s);
  }
  if (s > 0x1p-100f && s < 0x1p126f) return (double)s;
  if (any == 0u) return 0.0;
  double d = 0.0;
  if (edge) {
    const double x = clip_load(k.in + ev);
    d = x * x;
  }
  for (int j = tid; j < k.nvec; j += kClipThreads)
    for (int e = 0; e < VEC; ++e) {
      const double x = clip_load(k.in + k.head + j * VEC + e);
      d += x * x;
    }
  return d;
}

// Sum over the CTA in a fixed order; the result in every thread.
__device__ __forceinline__ double cta_sum(double v, double* sm) {
  v = warp_sum(v);
  __syncthreads();
  if (threadIdx.x % 32 == 0) sm[threadIdx.x / 32] = v;
  __syncthreads();
  double t = sm[0];
#pragma unroll
  for (int i = 1; i < kClipThreads / 32; ++i) t += sm[i];
  return t;
}

template <int kCap>
__global__ void __launch_bounds__(kClipThreads)
clip_norm_kernel(const __grid_constant__ ClipTable<kCap> t, double* partials) {
  __shared__ double sm[kClipThreads / 32];
  double sum = 0.0;
  int i = 0;
  for (unsigned c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    i = find_entry(t, c, i);
    const ClipEntry& e = t.e[i];
    switch (e.n >> 62) {
      case GRPO_F32: sum += chunk_squares(ClipChunk<float>(e, c)); break;
      case GRPO_BF16: sum += chunk_squares(ClipChunk<__nv_bfloat16>(e, c)); break;
      default: sum += chunk_squares(ClipChunk<__half>(e, c)); break;
    }
  }
  sum = cta_sum(sum, sm);
  if (threadIdx.x == 0) partials[blockIdx.x] = sum;
}

struct ClipScale {
  const double* partials;
  int count;
  double max_norm, eps, scale;
  float* out2;
  int first;  // this launch writes out2
};

// norm and c from the partial sums, the same in every thread of every CTA.
__device__ __forceinline__ float clip_factor(const ClipScale& k, double* sm) {
  double sum = 0.0;
  for (int i = threadIdx.x; i < k.count; i += kClipThreads) sum += k.partials[i];
  const double norm = k.scale * sqrt(cta_sum(sum, sm));
  double c = 1.0;
  if (!(k.max_norm >= norm + k.eps)) c = k.max_norm / (norm + k.eps);
  float f = (float)(c * k.scale);
  if (!(norm < INFINITY)) f = NAN;  // NaN too
  if (k.first && blockIdx.x == 0 && threadIdx.x == 0) {
    k.out2[0] = (float)norm;
    k.out2[1] = f;
  }
  return f;
}

template <typename T>
__device__ __forceinline__ void scale_chunk(const ClipChunk<T>& k, float f) {
  constexpr int VEC = Storage<T>::kVec;
  constexpr int kVecs = (int)(kClipChunk / kClipThreads) / VEC;
  const int tid = threadIdx.x;
  if (f == 1.f && k.in == k.out) return;
  if (tid < k.head + (k.n - k.t0)) {
    const int v = tid < k.head ? tid : k.t0 + tid - k.head;
    Storage<T>::store1(k.out + v, clip_load(k.in + v) * f);
  }
  const uint4* vec = reinterpret_cast<const uint4*>(k.in + k.head);
  const bool together = (((uintptr_t)k.in ^ (uintptr_t)k.out) & 15) == 0;
#pragma unroll 4
  for (int i = 0; i < kVecs; ++i) {
    const int j = tid + i * kClipThreads;
    if (j >= k.nvec) break;
    float x[VEC];
    Storage<T>::unpack(vec[j], x);
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] *= f;
    if (together) {
      reinterpret_cast<uint4*>(k.out + k.head)[j] = Storage<T>::pack(x);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) Storage<T>::store1(k.out + k.head + j * VEC + e, x[e]);
    }
  }
}

template <int kCap>
__global__ void __launch_bounds__(kClipThreads)
clip_scale_kernel(const __grid_constant__ ClipTable<kCap> t, const ClipScale k) {
  __shared__ double sm[kClipThreads / 32];
  const float f = clip_factor(k, sm);
  if (f != f) return;
  int i = 0;
  for (unsigned c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    i = find_entry(t, c, i);
    const ClipEntry& e = t.e[i];
    switch (e.n >> 62) {
      case GRPO_F32: scale_chunk(ClipChunk<float>(e, c), f); break;
      case GRPO_BF16: scale_chunk(ClipChunk<__nv_bfloat16>(e, c), f); break;
      default: scale_chunk(ClipChunk<__half>(e, c), f); break;
    }
  }
}

size_t clip_partials(int64_t num_tensors) {
  // a table's launch leaves at most kClipMaxGrid sums
  const int64_t tables = (num_tensors + kClipMany - 1) / kClipMany;
  return (size_t)(tables > 0 ? tables : 1) * kClipMaxGrid;
}

// Fills a table from tensor *i on; returns its chunks and moves *i past it.
template <int kCap>
static void fill_table(const ClipArgs& a, int64_t* i, ClipTable<kCap>* t) {
  t->count = 0;
  t->chunks = 0;
  for (; *i < a.count && t->count < kCap; ++*i) {
    const int64_t n = a.numels[*i];
    if (n == 0) continue;
    ClipEntry& e = t->e[t->count++];
    e.in = a.tensors[*i];
    e.out = a.outs ? a.outs[*i] : const_cast<void*>(a.tensors[*i]);
    e.n = (unsigned long long)n | (unsigned long long)a.dtypes[*i] << 62;
    e.chunk0 = t->chunks;
    t->chunks += (unsigned)((n + kClipChunk - 1) / kClipChunk);
  }
}

template <int kCap>
static cudaError_t launch_clip_t(const ClipArgs& a, int sms, cudaStream_t s) {
  const unsigned most = (unsigned)(sms * kClipCtasPerSm < kClipMaxGrid ? sms * kClipCtasPerSm
                                                                       : kClipMaxGrid);
  ClipTable<kCap> t;
  ClipScale k{a.partials, 0, a.max_norm, a.eps, a.scale, a.out2, 1};
  int64_t i = 0;
  do {
    fill_table(a, &i, &t);
    const unsigned grid = t.chunks < most ? (t.chunks ? t.chunks : 1) : most;
    clip_norm_kernel<kCap><<<grid, kClipThreads, 0, s>>>(t, a.partials + k.count);
    k.count += (int)grid;
  } while (i < a.count);
  i = 0;
  do {
    if (a.norm_only) {
      t.count = 0;
      t.chunks = 0;
      i = a.count;
    } else {
      fill_table(a, &i, &t);
    }
    const unsigned grid = t.chunks < most ? (t.chunks ? t.chunks : 1) : most;
    clip_scale_kernel<kCap><<<grid, kClipThreads, 0, s>>>(t, k);
    k.first = 0;
  } while (i < a.count);
  return cudaGetLastError();
}

cudaError_t launch_clip(const ClipArgs& a, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  return a.count <= kClipFew ? launch_clip_t<kClipFew>(a, sms, s)
                             : launch_clip_t<kClipMany>(a, sms, s);
}

}  // namespace grpo
