// grpo_token.cu -- log-probs of given tokens with entropy and top
// alternatives, and their gradient with respect to the logits.
//
// A row x of V logits, s = 1 / temperature, s2 = s log2(e):
//   m = max_v x_v,  u_v = s2 (x_v - m),  Z = sum 2^u_v,  D = sum 2^u_v u_v
//   logp = s (x_a - m) - ln Z,   H = ln Z - ln2 D / Z
// Z and D are formed online in one pass over the row: each thread holds the
// maximum of the logits it has seen and the two sums relative to it, and
// rescales both when the maximum moves (from m to m', d = s2 (m - m'):
// Z' = 2^d Z, D' = 2^d (D + d Z)).  u is a subtraction and a multiplication,
// not one fused multiply-add with a rounded s2 m: x - m is exact near the
// maximum and cannot overflow to +inf, so rows of the type's lowest value
// come out uniform.
//
//   token_logps_kernel  one CTA per row
//   token_grad_kernel   one CTA per row and chunk of the row
#include <type_traits>

#include "grpo_rows_common.cuh"

namespace grpo {

constexpr float kLn2f = 0.693147180559945309f;
// 2^u is 0 in fp32 (subnormals flushed) below this; u enters products with
// 2^u clamped to it, so that 0 x -inf does not turn a row into NaN.
constexpr float kLowU = -200.f;

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// Maximum and sums of the logits a thread (a warp, a CTA) has seen.
// NaN logits never become the maximum; they make Z NaN.
struct Stat {
  float m, Z, D;
};

template <bool kEnt>
__device__ __forceinline__ Stat merge(const Stat& a, const Stat& b, float s2) {
  Stat r;
  r.m = fmaxf(a.m, b.m);
  // -inf - -inf: both are empty (or hold -inf alone); the sums are 0 or NaN
  const float da = a.m == r.m ? 0.f : fmaxf((a.m - r.m) * s2, kLowU);
  const float db = b.m == r.m ? 0.f : fmaxf((b.m - r.m) * s2, kLowU);
  const float fa = ex2_fast(da), fb = ex2_fast(db);
  r.Z = a.Z * fa + b.Z * fb;
  if (kEnt) r.D = (a.D + da * a.Z) * fa + (b.D + db * b.Z) * fb;
  return r;
}

template <bool kEnt, int N>
__device__ __forceinline__ void add_logits(Stat& st, const float* x, float s2) {
  // the reference is 0 while nothing finite was seen: 2^(s2 (-inf)) = 0
  const float ref = st.m == -INFINITY ? 0.f : st.m;
  float e[N], d[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float u = (x[j] - ref) * s2;
    e[j] = ex2_fast(u);
    if (kEnt) d[j] = e[j] * fmaxf(u, kLowU);
  }
#pragma unroll
  for (int w = 1; w < N; w *= 2)
#pragma unroll
    for (int j = 0; j + w < N; j += 2 * w) {
      e[j] += e[j + w];
      if (kEnt) d[j] += d[j + w];
    }
  st.Z += e[0];
  if (kEnt) st.D += d[0];
}

// Raises the running maximum to vmax.
template <bool kEnt>
__device__ __forceinline__ void raise(Stat& st, float vmax, float s2) {
  const float d = fmaxf((st.m - vmax) * s2, kLowU);  // st.m = -inf: the sums are 0 or NaN
  const float f = ex2_fast(d);
  if (kEnt) st.D = (st.D + d * st.Z) * f;
  st.Z *= f;
  st.m = vmax;
}

// A logit and its index as one number that orders by value, then by lowest
// index.  0 is below every logit.
__device__ __forceinline__ unsigned order_of(float x) {
  const unsigned b = __float_as_uint(x + 0.f);  // -0 counts as 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float order_value(unsigned o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ unsigned long long key_of(float x, unsigned v) {
  return ((unsigned long long)order_of(x) << 32) | (0xFFFFFFFFu - v);
}

// Top-k.  A thread's slice is the 16-byte vectors tid, tid + kThreads, ... of
// the row.  The sweep leaves every thread's maximum; the k-th largest of them
// is a lower bound tau of the k-th largest logit, because k distinct logits
// reach it, and only slices whose maximum reaches tau can hold one of the top
// k.  So only those slices -- k of them, and those that tie -- are read
// again (from L2), and their logits at or above tau collected; each collected
// key's rank among them is its place in the answer.  The sweep itself pays
// nothing for the alternatives.
template <int kThreads, int kVec>
struct TopSmem {
  // a batch of kBatch vectors a thread may pass the bound whole
  static constexpr int kBatch = 2;
  static constexpr int kCompactAt = 2 * kThreads;
  static constexpr int kCap = kCompactAt + kThreads * kVec * kBatch;
  unsigned long long key[kCap];
  unsigned long long best[GRPO_MAX_TOP_K];
  unsigned ord[kThreads];        // each thread's maximum
  unsigned short sel[kThreads];  // slices to read again, in index order
  int nsel, n;
  unsigned tau;
};

// The k largest of sm.key[0 .. n) into best[0 .. k), largest first (keys are
// distinct).  Called by the whole CTA; ends with a barrier.
template <int kThreads, int kVec>
__device__ void rank_keys(TopSmem<kThreads, kVec>& sm, int n, int k) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const unsigned long long mine = sm.key[i];
    int above = 0;
    for (int j = 0; j < n; ++j) above += sm.key[j] > mine;
    if (above < k) sm.best[above] = mine;
  }
  __syncthreads();
}

template <typename T, int kThreads>
__device__ void top_alternatives(const T* row, const Geom<T>& g, float mine, int k,
                                 TopSmem<kThreads, Storage<T>::kVec>& sm) {
  constexpr int VEC = Storage<T>::kVec;
  using Smem = TopSmem<kThreads, VEC>;
  const int tid = threadIdx.x;
  const bool has = tid < g.nvec;
  sm.ord[tid] = has ? order_of(mine) : 0u;
  if (tid == 0) sm.n = 0;
  __syncthreads();
  if (tid < 32) {
    // tau: the largest bound, of 20 leading bits, that k maxima reach
    unsigned o[kThreads / 32];
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) o[i] = sm.ord[tid + 32 * i];
    unsigned t = 0;
    for (int b = 31; b >= 12; --b) {
      const unsigned c = t | (1u << b);
      int cnt = 0;
#pragma unroll
      for (int i = 0; i < kThreads / 32; ++i) cnt += o[i] >= c;
      if (__reduce_add_sync(0xFFFFFFFFu, cnt) >= k) t = c;
    }
    // the slices that reach it, in index order
    int at = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
      const bool in = o[i] >= t && o[i] != 0u;
      const unsigned b = __ballot_sync(0xFFFFFFFFu, in);
      if (in) sm.sel[at + __popc(b & ((1u << tid) - 1u))] = (unsigned short)(tid + 32 * i);
      at += __popc(b);
    }
    if (tid == 0) {
      sm.nsel = at;
      sm.tau = t;
    }
  }
  __syncthreads();
  unsigned long long bound = (unsigned long long)sm.tau << 32;
  const int nsel = sm.nsel;
  auto push = [&](float x, int64_t v) {
    const unsigned long long key = key_of(x, (unsigned)v);
    if (key >= bound) sm.key[atomicAdd(&sm.n, 1)] = key;
  };
  // row ends outside the vectors (fewer than kVec on either side)
  if (tid < g.head) push(Storage<T>::load1(row + tid), tid);
  if (tid < g.tail) push(Storage<T>::load1(row + g.t0 + tid), g.t0 + tid);
  // vectors in index order: j steps over the slices' length, i over the slices
  const unsigned total = (unsigned)nsel * (unsigned)((g.nvec + kThreads - 1) / kThreads);
  const uint4* vec = reinterpret_cast<const uint4*>(row + g.head);
  for (unsigned q0 = 0; q0 < total; q0 += Smem::kBatch * kThreads) {
    uint4 v[Smem::kBatch];
    int64_t at[Smem::kBatch];
#pragma unroll
    for (int u = 0; u < Smem::kBatch; ++u) {
      const unsigned q = q0 + tid + u * kThreads;
      at[u] = g.nvec;
      if (q < total) at[u] = sm.sel[q % nsel] + (q / nsel) * kThreads;
      if (at[u] < g.nvec) v[u] = __ldg(vec + at[u]);
    }
#pragma unroll
    for (int u = 0; u < Smem::kBatch; ++u) {
      if (at[u] >= g.nvec) continue;
      float x[VEC];
      Storage<T>::unpack(v[u], x);
#pragma unroll
      for (int e = 0; e < VEC; ++e) push(x[e], g.head + at[u] * VEC + e);
    }
    __syncthreads();
    // many ties: keep the k best so far, which raises the bound
    const int n = sm.n;
    if (n > Smem::kCompactAt) {
      rank_keys(sm, n, k);
      if (tid < k) sm.key[tid] = sm.best[tid];
      if (tid == 0) sm.n = k;
      bound = sm.best[k - 1];
      // the k-th key itself is held already
      bound += 1;
    }
    __syncthreads();
  }
  __syncthreads();
  rank_keys(sm, sm.n, k);
}

// One CTA per row: a sweep with kUnroll 16-byte loads a thread in flight, a
// tree over the threads, one thread's finish, then the alternatives.
template <typename T, int kThreads, bool kEnt, bool kTop>
__global__ void __launch_bounds__(kThreads)
token_logps_kernel(const TokenArgs a) {
  constexpr int VEC = Storage<T>::kVec;
  constexpr int kWarps = kThreads / 32;
  __shared__ Stat warp_stat[kWarps];
  __shared__ Stat total;
  __shared__ typename std::conditional<kTop, TopSmem<kThreads, VEC>, int>::type top;
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x, rows = a.B * a.T;
  if (a.mask && !a.mask[r]) {
    if (tid == 0) {
      if (a.logps) a.logps[r] = 0.f;
      if (a.entropy) a.entropy[r] = 0.f;
      if (a.stats) {
        a.stats[r] = 0.f;
        a.stats[rows + r] = 1.f;
      }
    }
    if (kTop && tid < a.k) {
      a.top_ids[r * a.k + tid] = -1;
      a.top_logps[r * a.k + tid] = 0.f;
    }
    return;
  }
  const T* row = (const T*)a.logits + (r / a.T) * a.sb + (r % a.T) * a.st;
  const Geom<T> g(row, a.V);
  const float s2 = a.s2;
  Stat st{-INFINITY, 0.f, 0.f};
  const uint4* vec = reinterpret_cast<const uint4*>(row + g.head);
  auto take = [&](const uint4& v) {
    float x[VEC];
    Storage<T>::unpack(v, x);
    float vmax = x[0];
#pragma unroll
    for (int e = 1; e < VEC; ++e) vmax = fmaxf(vmax, x[e]);
    if (vmax > st.m) raise<kEnt>(st, vmax, s2);
    add_logits<kEnt, VEC>(st, x, s2);
  };
  int64_t j = tid;
  for (; j + (kUnroll - 1) * kThreads < g.nvec; j += kUnroll * kThreads) {
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) v[u] = __ldg(vec + j + u * kThreads);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) take(v[u]);
  }
  for (; j < g.nvec; j += kThreads) take(__ldg(vec + j));
  const float mine = st.m;  // the maximum of this thread's slice
  if (tid < g.head + g.tail) {
    const float x = Storage<T>::load1(row + (tid < g.head ? tid : g.t0 + tid - g.head));
    if (x > st.m) raise<kEnt>(st, x, s2);
    add_logits<kEnt, 1>(st, &x, s2);
  }

#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Stat other;
    other.m = __shfl_xor_sync(0xFFFFFFFFu, st.m, o);
    other.Z = __shfl_xor_sync(0xFFFFFFFFu, st.Z, o);
    other.D = kEnt ? __shfl_xor_sync(0xFFFFFFFFu, st.D, o) : 0.f;
    st = merge<kEnt>(st, other, s2);
  }
  if (tid % 32 == 0) warp_stat[tid / 32] = st;
  __syncthreads();
  if (tid == 0) {
    Stat w = warp_stat[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) w = merge<kEnt>(w, warp_stat[i], s2);
    if (w.m == -INFINITY) w.Z = NAN;  // no finite logit: no distribution
    total = w;
    const float lnZ = logf(w.Z);
    if (a.logps) {
      const int64_t act = a.actions[r];
      float lp = NAN;
      if (act >= 0 && act < a.V)
        lp = (Storage<T>::load1(row + act) - w.m) * a.inv_t - lnZ;
      else if (a.hdr)
        atomicOr(&a.hdr->status, (unsigned)GRPO_ERR_ACTION_RANGE);
      a.logps[r] = lp;
    }
    if (kEnt) a.entropy[r] = lnZ - kLn2f * (w.D / w.Z);
    if (a.stats) {
      a.stats[r] = w.m;
      a.stats[rows + r] = w.Z;
    }
  }
  if constexpr (kTop) {
    __syncthreads();
    const Stat w = total;
    if (!(w.Z <= 3.4e38f)) {  // NaN or +inf
      if (tid < a.k) {
        a.top_ids[r * a.k + tid] = -1;
        a.top_logps[r * a.k + tid] = NAN;
      }
      return;
    }
    top_alternatives<T, kThreads>(row, g, mine, a.k, top);
    if (tid < a.k) {
      const unsigned long long key = top.best[tid];
      const float x = order_value((unsigned)(key >> 32));
      a.top_ids[r * a.k + tid] = (int64_t)(0xFFFFFFFFu - (unsigned)key);
      a.top_logps[r * a.k + tid] = (x - w.m) * a.inv_t - logf(w.Z);
    }
  }
}

// Rows of at most this many bytes go to one warp, longer ones to 256 threads.
static constexpr int64_t kWarpRowBytes = 4096;

template <typename T, int kThreads>
static cudaError_t launch_logps_t(const TokenArgs& a, cudaStream_t s) {
  const unsigned grid = (unsigned)(a.B * a.T);
  if (a.k > 0) {
    if (a.entropy) token_logps_kernel<T, kThreads, true, true><<<grid, kThreads, 0, s>>>(a);
    else token_logps_kernel<T, kThreads, false, true><<<grid, kThreads, 0, s>>>(a);
  } else {
    if (a.entropy) token_logps_kernel<T, kThreads, true, false><<<grid, kThreads, 0, s>>>(a);
    else token_logps_kernel<T, kThreads, false, false><<<grid, kThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

template <typename T>
static cudaError_t launch_logps_d(const TokenArgs& a, cudaStream_t s) {
  return a.V * (int64_t)sizeof(T) <= kWarpRowBytes ? launch_logps_t<T, 32>(a, s)
                                                   : launch_logps_t<T, 256>(a, s);
}

cudaError_t launch_token_logps(const TokenArgs& a, grpo_dtype_t dt, cudaStream_t s) {
  switch (dt) {
    case GRPO_F32: return launch_logps_d<float>(a, s);
    case GRPO_BF16: return launch_logps_d<__nv_bfloat16>(a, s);
    default: return launch_logps_d<__half>(a, s);
  }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
// With u = s2 (x_v - m):  dL/dx_v = s dlogp 1[v = a] - 2^u (c0 + c1 u),
//   c0 = s (dlogp + dH (H - ln Z)) / Z,   c1 = s dH ln2 / Z
// (log p_v = ln2 u - ln Z).  m and Z are the forward pass' own, so 2^u / Z
// carries no rounding of a logsumexp.
struct GradRow {
  float m, c0, c1, ga;  // ga: added at the action
  int64_t act;
};

__device__ __forceinline__ float token_grad(float x, const GradRow& q, float s2) {
  const float u = (x - q.m) * s2;
  return -ex2_fast(u) * (q.c0 + q.c1 * fmaxf(u, kLowU));
}

static constexpr int kGradThreads = 256;

// A CTA works on chunks of one row, kGradVecs 16-byte vectors a thread each;
// the row's unaligned ends go to its first CTA.  Plain loads, not the
// read-only path: in place, the row is written by this kernel.
static constexpr int kGradVecs = 4;

__device__ __forceinline__ float load_plain(const float* p) { return *p; }
__device__ __forceinline__ float load_plain(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load_plain(const __half* p) { return __half2float(*p); }

template <typename T>
__global__ void __launch_bounds__(kGradThreads)
token_grad_kernel(const TokenGradArgs a, unsigned chunks, unsigned ctas) {
  constexpr int VEC = Storage<T>::kVec;
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x / ctas, rows = a.B * a.T;
  const unsigned first = blockIdx.x % ctas;
  const bool on = !a.mask || a.mask[r];
  if (!on && a.skip_masked) return;
  T* grow = (T*)a.grad + (r / a.T) * a.gsb + (r % a.T) * a.gst;
  const T* row = (const T*)a.logits + (r / a.T) * a.sb + (r % a.T) * a.st;
  const float w = on && a.dlogp ? a.dlogp[r] : 0.f;
  const float h = on && a.dent ? a.dent[r] : 0.f;
  const bool zero = w == 0.f && h == 0.f;
  GradRow q{0.f, 0.f, 0.f, 0.f, -1};
  if (!zero) {
    const float Z = a.stats[rows + r];
    q.m = a.stats[r];
    float c0 = w;
    if (h != 0.f) c0 += h * (a.entropy[r] - logf(Z));
    q.c0 = a.inv_t * c0 / Z;
    q.c1 = a.inv_t * kLn2f * h / Z;
    if (w != 0.f) {
      q.act = a.actions[r];
      q.ga = a.inv_t * w;
      if (q.act < 0 || q.act >= a.V) {
        q.c0 = NAN;
        if (a.hdr && first == 0 && tid == 0)
          atomicOr(&a.hdr->status, (unsigned)GRPO_ERR_ACTION_RANGE);
      }
    }
  }
  const Geom<T> g(grow, a.V);  // by the gradient's alignment: the stores are whole
  if (first == 0 && tid < g.head + g.tail) {
    const int64_t v = tid < g.head ? tid : g.t0 + tid - g.head;
    float d = 0.f;
    if (!zero) d = token_grad(load_plain(row + v), q, a.s2) + (v == q.act ? q.ga : 0.f);
    Storage<T>::store1(grow + v, d);
  }
  const bool together = (((uintptr_t)grow ^ (uintptr_t)row) & 15) == 0;
  uint4* out = reinterpret_cast<uint4*>(grow + g.head);
  const T* in = row + g.head;
  const int64_t act = q.act - g.head;  // among the vectors' elements
  for (unsigned chunk = first; chunk < chunks; chunk += ctas) {
    const int64_t j0 = (int64_t)chunk * (kGradVecs * kGradThreads) + tid;
    if (zero) {
#pragma unroll
      for (int k = 0; k < kGradVecs; ++k)
        if (j0 + k * kGradThreads < g.nvec) out[j0 + k * kGradThreads] = make_uint4(0u, 0u, 0u, 0u);
      continue;
    }
    uint4 v[kGradVecs];
#pragma unroll
    for (int k = 0; k < kGradVecs; ++k) {
      const int64_t j = j0 + k * kGradThreads;
      if (j >= g.nvec) continue;
      if (together) {
        v[k] = *(reinterpret_cast<const uint4*>(in) + j);
      } else {
        T t[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) t[e] = in[j * VEC + e];
        v[k] = *reinterpret_cast<const uint4*>(t);
      }
    }
#pragma unroll
    for (int k = 0; k < kGradVecs; ++k) {
      const int64_t j = j0 + k * kGradThreads;
      if (j >= g.nvec) continue;
      float x[VEC];
      Storage<T>::unpack(v[k], x);
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[e] = token_grad(x[e], q, a.s2);
      const uint64_t at = (uint64_t)(act - j * VEC);
      if (at < VEC) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[e] += at == e ? q.ga : 0.f;
      }
      out[j] = Storage<T>::pack(x);
    }
  }
}

template <typename T>
static cudaError_t launch_grad_t(const TokenGradArgs& a, cudaStream_t s) {
  const int64_t per = (int64_t)kGradThreads * kGradVecs * Storage<T>::kVec;
  const int64_t chunks = (a.V + per - 1) / per, rows = a.B * a.T;
  // one CTA per chunk, fewer where the grid would pass 2^31 - 1 CTAs
  const int64_t most = 0x7FFFFFFF / rows, ctas = chunks < most ? chunks : most;
  token_grad_kernel<T><<<(unsigned)(rows * ctas), kGradThreads, 0, s>>>(a, (unsigned)chunks,
                                                                        (unsigned)ctas);
  return cudaGetLastError();
}

cudaError_t launch_token_grad(const TokenGradArgs& a, grpo_dtype_t dt, cudaStream_t s) {
  switch (dt) {
    case GRPO_F32: return launch_grad_t<float>(a, s);
    case GRPO_BF16: return launch_grad_t<__nv_bfloat16>(a, s);
    default: return launch_grad_t<__half>(a, s);
  }
}

}  // namespace grpo
