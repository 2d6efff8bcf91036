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
// A chunk is cut from one tensor, its elements taken as 16-byte vectors where
// the tensor's alignment allows.
//
// Bound by memory: the tensors are read once for the norm and, where they are
// larger than L2, again to be scaled.  291 bf16 tensors of 3.6 GB: norm 507 us
// (7.0 TB/s), both 1556 us for 10.7 GB (6.8 TB/s, the rate of a copy); 111
// packed tensors of mixed types, 0.45 GB: 84 and 228 us.  Unclipped in place
// 506 us: the second kernel returns.  Small sets cost latency: one tensor of 1000
// elements 4.5 us, 21 of 7.5 MB in all 10 us.
#include "grpo_around.cuh"

namespace grpo {

static constexpr int kClipThreads = 256;
// CTAs an SM and vectors a thread in flight in each kernel.  Norm of 3.6 GB,
// us: 4 CTAs x 8 vectors 508, 5 x 8 498 (but 89 instead of 84 on 0.45 GB), 4 x 4
// 559, 6 x 4 511, 8 x 4 622.  Scaling: a grid of 6 CTAs an SM x 4, chosen with
// pieces of two chunks on both sets; 32 CTAs an SM cost 70 us where nothing is
// clipped.  Its registers (71; 51 with the smaller chunks) let 3 (4) of the 6
// be resident, so the grid runs as two waves, and each forms the norm again.
static constexpr int kNormCtasPerSm = 4, kNormAhead = 8;
static constexpr int kScaleCtasPerSm = 6, kScaleAhead = 4;
static constexpr int kClipMaxGrid = 2048;
// A chunk holds kPer elements a thread, whose squares one fp32 sum covers: 64,
// or 16 up to kSmallTotal elements, where chunks of 64 leave SMs idle (us at 16
// / 64: one tensor of 100,000 5.7 / 10.4, 200 of them 41 / 52, 400 80 / 91;
// 113 M elements 242 / 230).
static constexpr int64_t kSmallTotal = 64 << 20;
static constexpr unsigned kPiece = 2;  // chunks a CTA takes at a time
template <int kPer>
__host__ __device__ constexpr int64_t clip_chunk() { return (int64_t)kPer * kClipThreads; }

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

// A CTA takes pieces of kPiece consecutive chunks; the entry of a piece's
// first chunk is searched for (each probe of the table is a constant-cache
// miss when it is long), the others follow it.

// The last entry whose chunk0 is at most c.
template <int kCap>
__device__ __forceinline__ int find_entry(const ClipTable<kCap>& t, unsigned c) {
  int lo = 0, hi = t.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (t.e[mid].chunk0 <= c) lo = mid;
    else hi = mid;
  }
  return lo;
}

// fn(entry, chunk) for each chunk of piece p.
template <int kCap, typename F>
__device__ __forceinline__ void each_chunk(const ClipTable<kCap>& t, unsigned p, F fn) {
  unsigned c = p * kPiece;
  const unsigned end = min(c + kPiece, t.chunks);
  int i = find_entry(t, c);
  unsigned next = i + 1 < t.count ? t.e[i + 1].chunk0 : t.chunks;
  for (; c < end; ++c) {
    if (c >= next) {
      ++i;
      next = i + 1 < t.count ? t.e[i + 1].chunk0 : t.chunks;
    }
    fn(t.e[i], c);
  }
}

template <typename T, int kPer>
struct ClipChunk {
  const T* in;
  T* out;
  int n, head, nvec, t0;
  __device__ ClipChunk(const ClipEntry& e, unsigned c) {
    // chunks are cut at 16-byte boundaries of the input: all but a tensor's
    // first and last are whole vectors
    const int64_t skew = ((uintptr_t)e.in & 15) / sizeof(T);
    const int64_t size = (int64_t)(e.n & ((1ull << 62) - 1));
    const int64_t end = (int64_t)(c - e.chunk0 + 1) * clip_chunk<kPer>() - skew;
    const int64_t at = c == e.chunk0 ? 0 : end - clip_chunk<kPer>();
    in = (const T*)e.in + at;
    out = (T*)e.out + at;
    n = (int)((size < end ? size : end) - at);
    head = (int)(((16 - ((uintptr_t)in & 15)) & 15) / sizeof(T));
    if (head > n) head = n;
    nvec = (n - head) / Storage<T>::kVec;
    t0 = head + nvec * Storage<T>::kVec;
  }
};

__device__ __forceinline__ float clip_load(const float* p) { return *p; }
__device__ __forceinline__ float clip_load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float clip_load(const __half* p) { return __half2float(*p); }

// The gradients of a chunk; not kept in L1.
__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// A thread's sum of squares: a float pair (fp32 operations: double ones run at
// a 64th of their rate on this GPU) and, for what lies outside its range, a
// double.
struct ClipSum {
  float hi = 0.f, lo = 0.f;
  double wide = 0.0;
  int used = 0;  // whether wide holds anything
};

// This thread's part of a chunk's sum of squares.  The fp32 sum is taken
// where it lies well inside the range (or the elements are all zero); a sum
// that overflowed, or so small that squares were lost below the range, is
// formed again in double.
template <typename T, int kPer>
__device__ __forceinline__ void add_squares(const ClipChunk<T, kPer>& k, ClipSum& sum) {
  constexpr int VEC = Storage<T>::kVec;
  constexpr int kVecs = kPer / VEC;  // vectors a thread at most
  constexpr int kAhead = kNormAhead < kVecs ? kNormAhead : kVecs;
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
  auto take = [&](const uint4& v) {
    float x[VEC];
    Storage<T>::unpack(v, x);
    any |= v.x | v.y | v.z | v.w;
#pragma unroll
    for (int e = 0; e < VEC; ++e) s = fmaf(x[e], x[e], s);
  };
  // the loads of kAhead vectors in flight together
  if (k.nvec == kVecs * kClipThreads) {
#pragma unroll
    for (int i = 0; i < kVecs; i += kAhead) {
      uint4 v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) v[u] = ld_stream(vec + tid + (i + u) * kClipThreads);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) take(v[u]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVecs; i += kAhead) {
      uint4 v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int j = tid + (i + u) * kClipThreads;
        v[u] = j < k.nvec ? ld_stream(vec + j) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) take(v[u]);
    }
  }
  if (s > 0x1p-100f && s < 0x1p100f) {
    const FF t = two_sum(sum.hi, s);
    sum.hi = t.hi;
    sum.lo = __fadd_rn(sum.lo, t.lo);
    return;
  }
  if (any == 0u) return;
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
  sum.wide += d;
  sum.used = 1;
}

struct ClipSmem {
  FF pair[kClipThreads / 32];
  double wide[kClipThreads / 32];
  float factor;
};

// The CTA's sum in a fixed order, in thread 0.
__device__ __forceinline__ double cta_squares(const ClipSum& v, ClipSmem& sm) {
  constexpr int kWarps = kClipThreads / 32;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const FF w = warp_sum_ff2(FF{v.hi, v.lo});
  if (lane == 0) sm.pair[warp] = w;
  const bool wide = __syncthreads_or(v.used);
  if (wide) {  // rare
    const double d = warp_sum(v.wide);
    if (lane == 0) sm.wide[warp] = d;
    __syncthreads();
  }
  double t = 0.0;
  if (threadIdx.x == 0) {
    FF f = sm.pair[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) f = ff_add(f, sm.pair[i]);
    t = (double)f.hi + (double)f.lo;
    if (wide)
      for (int i = 0; i < kWarps; ++i) t += sm.wide[i];
  }
  return t;
}

template <int kCap, int kPer>
__global__ void __launch_bounds__(kClipThreads)
clip_norm_kernel(const __grid_constant__ ClipTable<kCap> t, double* partials) {
  __shared__ ClipSmem sm;
  // the scaling CTAs may take their places beside these, and wait
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  ClipSum sum;
  const unsigned pieces = (t.chunks + kPiece - 1) / kPiece;
  for (unsigned p = blockIdx.x; p < pieces; p += gridDim.x)
    each_chunk(t, p, [&](const ClipEntry& e, unsigned c) {
      switch (e.n >> 62) {
        case GRPO_F32: add_squares(ClipChunk<float, kPer>(e, c), sum); break;
        case GRPO_BF16: add_squares(ClipChunk<__nv_bfloat16, kPer>(e, c), sum); break;
        default: add_squares(ClipChunk<__half, kPer>(e, c), sum); break;
      }
    });
  const double total = cta_squares(sum, sm);
  if (threadIdx.x == 0) partials[blockIdx.x] = total;
}

struct ClipScale {
  const double* partials;
  int count;
  double max_norm, eps, scale;
  float* out2;
  int first;     // this launch writes out2
  int in_place;  // no tensor has an output of its own
  int norm_only; // nothing is written
};

// norm and c from the partial sums, the same in every CTA; by one warp of it,
// because the double operations of eight would take microseconds.
__device__ __forceinline__ float clip_factor(const ClipScale& k, ClipSmem& sm) {
  const int lane = threadIdx.x;
  if (lane < 32) {
    double sum = 0.0;
#pragma unroll 8
    for (int i = lane; i < k.count; i += 32) sum += k.partials[i];
    sum = warp_sum(sum);
    const double norm = k.scale * sqrt(sum);
    double c = 1.0;
    if (!(k.max_norm >= norm + k.eps)) c = k.max_norm / (norm + k.eps);
    float f = (float)(c * k.scale);
    // (NaN too.)  Finite in fp64 but not as the fp32 number that the caller
    // sees: nothing may be written, and only a call that writes nothing gets c
    if (!(norm < INFINITY) || (!k.norm_only && !((float)norm < INFINITY))) f = NAN;
    if (lane == 0) {
      sm.factor = f;
      if (k.first && blockIdx.x == 0) {
        k.out2[0] = (float)norm;
        k.out2[1] = f;
      }
    }
  }
  __syncthreads();
  return sm.factor;
}

template <typename T, int kPer>
__device__ __forceinline__ void scale_chunk(const ClipChunk<T, kPer>& k, float f) {
  constexpr int VEC = Storage<T>::kVec;
  constexpr int kVecs = kPer / VEC;
  constexpr int kAhead = kScaleAhead < kVecs ? kScaleAhead : kVecs;
  const int tid = threadIdx.x;
  if (f == 1.f && k.in == k.out) return;
  if (tid < k.head + (k.n - k.t0)) {
    const int v = tid < k.head ? tid : k.t0 + tid - k.head;
    Storage<T>::store1(k.out + v, clip_load(k.in + v) * f);
  }
  const uint4* vec = reinterpret_cast<const uint4*>(k.in + k.head);
  const bool together = (((uintptr_t)k.in ^ (uintptr_t)k.out) & 15) == 0;
  const uint64_t pol = l2_evict_first();
  auto put = [&](int j, const uint4& v) {
    float x[VEC];
    Storage<T>::unpack(v, x);
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] *= f;
    if (together) {
      // first to leave L2: what is still to be read stays
      st_hint(reinterpret_cast<uint4*>(k.out + k.head) + j, Storage<T>::pack(x), pol);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) Storage<T>::store1(k.out + k.head + j * VEC + e, x[e]);
    }
  };
#pragma unroll
  for (int i = 0; i < kVecs; i += kAhead) {
    uint4 v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = tid + (i + u) * kClipThreads;
      if (j < k.nvec) v[u] = ld_stream(vec + j);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int j = tid + (i + u) * kClipThreads;
      if (j < k.nvec) put(j, v[u]);
    }
  }
}

template <int kCap, int kPer>
__global__ void __launch_bounds__(kClipThreads)
clip_scale_kernel(const __grid_constant__ ClipTable<kCap> t, const ClipScale k) {
  __shared__ ClipSmem sm;
  // launched while the norm's last CTAs run; their sums are complete from here
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const float f = clip_factor(k, sm);
  if (f != f || (f == 1.f && k.in_place)) return;
  // from the end: what the norm read last is in L2 still (the first wave's
  // pieces: the second one starts from the end again)
  const unsigned pieces = (t.chunks + kPiece - 1) / kPiece;
  for (unsigned q = blockIdx.x; q < pieces; q += gridDim.x)
    each_chunk(t, pieces - 1 - q, [&](const ClipEntry& e, unsigned c) {
      switch (e.n >> 62) {
        case GRPO_F32: scale_chunk(ClipChunk<float, kPer>(e, c), f); break;
        case GRPO_BF16: scale_chunk(ClipChunk<__nv_bfloat16, kPer>(e, c), f); break;
        default: scale_chunk(ClipChunk<__half, kPer>(e, c), f); break;
      }
    });
}

size_t clip_partials(int64_t num_tensors) {
  // a table's launch leaves at most kClipMaxGrid sums
  const int64_t tables = (num_tensors + kClipMany - 1) / kClipMany;
  return (size_t)(tables > 0 ? tables : 1) * kClipMaxGrid;
}

// Fills a table from tensor *i on; returns its chunks and moves *i past it.
template <int kCap, int kPer>
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
    const int64_t skew = ((uintptr_t)e.in & 15) / (a.dtypes[*i] == GRPO_F32 ? 4 : 2);
    t->chunks += (unsigned)((n + skew + clip_chunk<kPer>() - 1) / clip_chunk<kPer>());
  }
}

template <int kCap, int kPer>
static cudaError_t launch_clip_t(const ClipArgs& a, int sms, cudaStream_t s) {
  const unsigned most = (unsigned)min(sms * kNormCtasPerSm, kClipMaxGrid);
  const unsigned most_scale = (unsigned)(sms * kScaleCtasPerSm);
  ClipTable<kCap> t;
  ClipScale k{a.partials, 0, a.max_norm, a.eps, a.scale, a.out2, 1, a.outs == nullptr,
              a.norm_only};
  int64_t i = 0;
  do {
    fill_table<kCap, kPer>(a, &i, &t);
    const unsigned pieces = (t.chunks + kPiece - 1) / kPiece;
    const unsigned grid = max(1u, min(pieces, most));
    clip_norm_kernel<kCap, kPer><<<grid, kClipThreads, 0, s>>>(t, a.partials + k.count);
    k.count += (int)grid;
  } while (i < a.count);
  i = 0;
  do {
    if (a.norm_only) {
      t.count = 0;
      t.chunks = 0;
      i = a.count;
    } else {
      fill_table<kCap, kPer>(a, &i, &t);
    }
    const unsigned pieces = (t.chunks + kPiece - 1) / kPiece;
    const unsigned grid = max(1u, min(pieces, most_scale));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kClipThreads);
    cfg.stream = s;
    // the first one may be dispatched while the norm kernel ends (it waits
    // for it); a later one follows it in full
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = k.first ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, clip_scale_kernel<kCap, kPer>, t, k);
    if (e != cudaSuccess) return e;
    k.first = 0;
  } while (i < a.count);
  return cudaGetLastError();
}

cudaError_t launch_clip(const ClipArgs& a, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  int64_t total = 0;
  for (int64_t i = 0; i < a.count; ++i) total += a.numels[i];
  const bool few = a.count <= kClipFew;
  if (total <= kSmallTotal)
    return few ? launch_clip_t<kClipFew, 16>(a, sms, s) : launch_clip_t<kClipMany, 16>(a, sms, s);
  return few ? launch_clip_t<kClipFew, 64>(a, sms, s) : launch_clip_t<kClipMany, 64>(a, sms, s);
}

}  // namespace grpo
