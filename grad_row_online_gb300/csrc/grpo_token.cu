// grpo_token.cu -- log-probs of given tokens with entropy and top
// alternatives, and their gradient with respect to the logits.
//
// A row x of V logits, s = 1 / temperature, s2 = s log2(e):
//   m = max_v x_v,  u_v = s2 (x_v - m),  Z = sum 2^u_v,  D = sum 2^u_v u_v
//   logp = s (x_a - m) - ln Z,   H = ln Z - ln2 D / Z
// Z and D are formed online in one pass over the row: each thread holds the
// maximum of the logits it has seen and the two sums relative to it, and
// rescales both when the maximum moves (from m to m', d = s2 (m - m'):
// Z' = 2^d Z, D' = 2^d (D + d Z)).
//
//   token_logps_kernel  one CTA, or a cluster of CTAs, per row
//   token_grad_kernel   one CTA per row and chunk of the row
#include <cooperative_groups.h>

#include <type_traits>

#include "grpo_rows_common.cuh"

namespace grpo {

namespace cg = cooperative_groups;

constexpr float kLn2f = 0.693147180559945309f;
// 2^u is 0 in fp32 (subnormals flushed) below this; where u may be -inf it
// enters products with 2^u clamped to this, so that 0 x -inf is not a NaN.
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
  r.D = kEnt ? (a.D + da * a.Z) * fa + (b.D + db * b.Z) * fb : 0.f;
  return r;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// Logits as they are stored, two to a 32-bit word for the 16-bit types:
// maxima and the lower clamp act on words.  floor_word: a lower bound in
// every place of a word; at_least keeps NaN, larger drops it.
template <typename T> struct Words;
template <> struct Words<float> {
  static constexpr int kPairs = 2;  // pairs of logits in 16 bytes
  __device__ static uint32_t floor_word(float low) { return __float_as_uint(low); }
  __device__ static uint32_t at_least(uint32_t w, uint32_t low) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(w)), "f"(__uint_as_float(low)));
    return __float_as_uint(r);
  }
  __device__ static uint32_t larger(uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }
  __device__ static float value(uint32_t w) { return __uint_as_float(w); }  // of a maximum
};
template <> struct Words<__nv_bfloat16> {
  static constexpr int kPairs = 4;
  __device__ static uint32_t floor_word(float low) {
    return Storage<__nv_bfloat16>::pack2(low, low);
  }
  __device__ static uint32_t at_least(uint32_t w, uint32_t low) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(low));
    return r;
  }
  __device__ static uint32_t larger(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  __device__ static float value(uint32_t w) {
    return fmaxf(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
};
template <> struct Words<__half> {
  static constexpr int kPairs = 4;
  __device__ static uint32_t floor_word(float low) { return Storage<__half>::pack2(low, low); }
  __device__ static uint32_t at_least(uint32_t w, uint32_t low) {
    uint32_t r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(low));
    return r;
  }
  __device__ static uint32_t larger(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  __device__ static float value(uint32_t w) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return fmaxf(f.x, f.y);
  }
};

// The sweep's accumulator.  At memory speed an SM has to take 12 bf16 logits
// a cycle, and issues 4 warp instructions a cycle: about ten to a logit.  So
// exponents are one fused multiply-add, x s2 - mL with mL = fl(m s2) -- the
// rounding of mL is the same in every term and taken out at the end -- and
// products and sums run as pairs.  That holds where |m| s2 stays below
// kFastRange; -inf and the types' lowest values are raised to a floor `low`
// whose exponential is 0 all the same, so no exponent is infinite.  A row (a
// cluster's part of one) whose maximum leaves the range is swept again by
// sweep_any, which subtracts the maximum first.
constexpr float kFastRange = 4096.f;

template <typename T, bool kEnt>
struct Fast {
  static constexpr int kPairs = Words<T>::kPairs;
  float m, mL;
  float2 Z, D;
  __device__ void init(float low, float s2) {
    m = low;
    mL = low * s2;
    Z = D = make_float2(0.f, 0.f);
  }
  __device__ __forceinline__ void raise(float vmax, float s2) {
    const float nL = __fmul_rn(vmax, s2);
    const float d = mL - nL, f = ex2_fast(d);
    const float2 f2 = make_float2(f, f);
    if (kEnt) D = mul2(fma2(make_float2(d < kLowU ? kLowU : d, d < kLowU ? kLowU : d), Z, D), f2);
    Z = mul2(Z, f2);
    m = vmax;
    mL = nL;
  }
  // N 16-byte vectors
  template <int N>
  __device__ __forceinline__ void take(uint4 (&v)[N], uint32_t low, float s2) {
    uint32_t top = 0;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      uint32_t* w = &v[n].x;
      if (kEnt) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = Words<T>::at_least(w[i], low);
      }
      const uint32_t t = Words<T>::larger(Words<T>::larger(w[0], w[1]),
                                          Words<T>::larger(w[2], w[3]));
      top = n == 0 ? t : Words<T>::larger(top, t);
    }
    const float vmax = Words<T>::value(top);
    if (vmax > m) raise(vmax, s2);
    const float2 sc = make_float2(s2, s2), off = make_float2(-mL, -mL);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float x[2 * kPairs];
      Storage<T>::unpack(v[n], x);
      float2 e[kPairs], d;
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const float2 u = fma2(make_float2(x[2 * i], x[2 * i + 1]), sc, off);
        e[i] = make_float2(ex2_fast(u.x), ex2_fast(u.y));
        if (kEnt) d = i == 0 ? mul2(e[i], u) : fma2(e[i], u, d);
      }
#pragma unroll
      for (int w = 1; w < kPairs; w *= 2)
#pragma unroll
        for (int i = 0; i + w < kPairs; i += 2 * w) e[i] = add2(e[i], e[i + w]);
      Z = add2(Z, e[0]);
      if (kEnt) D = add2(D, d);
    }
  }
  __device__ __forceinline__ void take1(float x, float low, float s2) {
    if (x < low) x = low;
    if (x > m) raise(x, s2);
    const float u = __fmaf_rn(x, s2, -mL), e = ex2_fast(u);
    Z.x += e;
    if (kEnt) D.x = __fmaf_rn(e, u, D.x);
  }
  // relative to m itself: the exponents were too small by r = m s2 - mL
  __device__ Stat stat(float s2) const {
    const float r = __fmaf_rn(m, s2, -mL), f = ex2_fast(-r);
    Stat st;
    st.m = m;
    st.Z = (Z.x + Z.y) * f;
    st.D = kEnt ? (D.x + D.y - r * (Z.x + Z.y)) * f : 0.f;
    return st;
  }
};

// A part of a row: scalars [0, head) and [t0, t0 + tail), vectors [v0, v1).
struct Part {
  int head, tail;
  int64_t t0, v0, v1;
};

// The sweep for any values: x - m is formed first, exactly near the maximum
// and without overflow to +inf, so that rows of the type's lowest value come
// out uniform.  Out of line: few rows come here.
template <typename T, int kThreads, bool kEnt>
__device__ __noinline__ Stat sweep_any(const T* row, const uint4* vec, Part p, float s2,
                                       float* mine) {
  constexpr int VEC = Storage<T>::kVec;
  Stat st{-INFINITY, 0.f, 0.f};
  auto one = [&](float x) {
    if (x > st.m) {
      const float d = fmaxf((st.m - x) * s2, kLowU), f = ex2_fast(d);  // from -inf: sums 0 or NaN
      st.D = (st.D + d * st.Z) * f;
      st.Z *= f;
      st.m = x;
    }
    // the reference is 0 while nothing finite was seen: 2^(s2 (-inf)) = 0
    const float u = (x - (st.m == -INFINITY ? 0.f : st.m)) * s2, e = ex2_fast(u);
    st.Z += e;
    if (kEnt) st.D += e * fmaxf(u, kLowU);
  };
  // sums of a few vectors apart, so that no long chain of additions forms
  Stat all{-INFINITY, 0.f, 0.f};
  for (int64_t j = p.v0 + threadIdx.x; j < p.v1; j += kThreads) {
    float x[VEC];
    Storage<T>::unpack(__ldg(vec + j), x);
    st = Stat{-INFINITY, 0.f, 0.f};
    for (int e = 0; e < VEC; ++e) one(x[e]);
    all = merge<kEnt>(all, st, s2);
  }
  *mine = all.m;
  if ((int)threadIdx.x < p.head + p.tail) {
    const int i = threadIdx.x;
    st = Stat{-INFINITY, 0.f, 0.f};
    one(Storage<T>::load1(row + (i < p.head ? i : p.t0 + i - p.head)));
    all = merge<kEnt>(all, st, s2);
  }
  return all;
}

template <typename T, int kThreads, bool kEnt>
__device__ __forceinline__ Stat sweep_fast(const T* row, const uint4* vec, const Part& p, float low,
                                           float s2, float* mine) {
  Fast<T, kEnt> f;
  f.init(low, s2);
  const uint32_t low_word = Words<T>::floor_word(low);
  int64_t j = p.v0 + threadIdx.x;
  for (; j + (kUnroll - 1) * kThreads < p.v1; j += kUnroll * kThreads) {
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) v[u] = __ldg(vec + j + u * kThreads);
    f.take(v, low_word, s2);
  }
  for (; j < p.v1; j += kThreads) {
    uint4 v[1] = {__ldg(vec + j)};
    f.take(v, low_word, s2);
  }
  *mine = f.m > low ? f.m : -INFINITY;
  if ((int)threadIdx.x < p.head + p.tail) {
    const int i = threadIdx.x;
    f.take1(Storage<T>::load1(row + (i < p.head ? i : p.t0 + i - p.head)), low, s2);
  }
  return f.stat(s2);
}

// The CTA's Stat from its threads', the same in every thread.  Ends with a
// barrier.
template <int kThreads, bool kEnt>
__device__ __forceinline__ Stat cta_stat(Stat st, float s2, Stat* sm) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Stat other;
    other.m = __shfl_xor_sync(0xFFFFFFFFu, st.m, o);
    other.Z = __shfl_xor_sync(0xFFFFFFFFu, st.Z, o);
    other.D = kEnt ? __shfl_xor_sync(0xFFFFFFFFu, st.D, o) : 0.f;
    st = merge<kEnt>(st, other, s2);
  }
  constexpr int kWarps = kThreads / 32;
  if (kWarps == 1) return st;
  __syncthreads();
  if (threadIdx.x % 32 == 0) sm[threadIdx.x / 32] = st;
  __syncthreads();
  const int lane = threadIdx.x % 32;
  st = lane < kWarps ? sm[lane] : Stat{-INFINITY, 0.f, 0.f};
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1) {
    Stat other;
    other.m = __shfl_xor_sync(0xFFFFFFFFu, st.m, o);
    other.Z = __shfl_xor_sync(0xFFFFFFFFu, st.Z, o);
    other.D = kEnt ? __shfl_xor_sync(0xFFFFFFFFu, st.D, o) : 0.f;
    st = merge<kEnt>(st, other, s2);
  }
  st.m = __shfl_sync(0xFFFFFFFFu, st.m, 0);
  st.Z = __shfl_sync(0xFFFFFFFFu, st.Z, 0);
  st.D = __shfl_sync(0xFFFFFFFFu, st.D, 0);
  return st;
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
  static constexpr int kBatch = 1;
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
__device__ void top_alternatives(const T* row, const uint4* vec, const Part& p, int head,
                                 float mine, int k,
                                 TopSmem<kThreads, Storage<T>::kVec>& sm) {
  constexpr int VEC = Storage<T>::kVec;
  using Smem = TopSmem<kThreads, VEC>;
  const int tid = threadIdx.x;
  const bool has = p.v0 + tid < p.v1;
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
  if (tid < p.head) push(Storage<T>::load1(row + tid), tid);
  if (tid < p.tail) push(Storage<T>::load1(row + p.t0 + tid), p.t0 + tid);
  // vectors in index order: j steps over the slices' length, i over the slices
  const unsigned total = (unsigned)nsel * (unsigned)((p.v1 - p.v0 + kThreads - 1) / kThreads);
  for (unsigned q0 = 0; q0 < total; q0 += Smem::kBatch * kThreads) {
    uint4 v[Smem::kBatch];
    int64_t at[Smem::kBatch];
#pragma unroll
    for (int u = 0; u < Smem::kBatch; ++u) {
      const unsigned q = q0 + tid + u * kThreads;
      at[u] = p.v1;
      if (q < total) at[u] = p.v0 + sm.sel[q % nsel] + (q / nsel) * kThreads;
      if (at[u] < p.v1) v[u] = __ldg(vec + at[u]);
    }
#pragma unroll
    for (int u = 0; u < Smem::kBatch; ++u) {
      if (at[u] >= p.v1) continue;
      float x[VEC];
      Storage<T>::unpack(v[u], x);
#pragma unroll
      for (int e = 0; e < VEC; ++e) push(x[e], head + at[u] * VEC + e);
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

// A row's results, by one thread; `act` is its action.
template <typename T, bool kEnt>
__device__ __forceinline__ void finish_row(const TokenArgs& a, int64_t r, const T* row, Stat w) {
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
    a.stats[a.B * a.T + r] = w.Z;
  }
}

// What the CTAs of a cluster leave in its first CTA's shared memory.
static constexpr int kMaxCluster = 8;
struct Parts {
  Stat st[kMaxCluster];
  int n[kMaxCluster];  // keys held
  unsigned long long key[kMaxCluster * GRPO_MAX_TOP_K];
};

// One CTA per row, or with kSplit a cluster of CTAs, each of which takes a
// contiguous part of the row's vectors: a sweep with kUnroll 16-byte loads a
// thread in flight, a tree over the threads, the part's alternatives, and in
// a cluster the parts joined by its first CTA.
template <typename T, int kThreads, bool kEnt, bool kTop, bool kSplit>
__global__ void __launch_bounds__(kThreads)
token_logps_kernel(const TokenArgs a) {
  constexpr int VEC = Storage<T>::kVec;
  __shared__ Stat warp_stat[kThreads / 32];
  __shared__ typename std::conditional<kTop, TopSmem<kThreads, VEC>, int>::type top;
  __shared__ typename std::conditional<kSplit, Parts, int>::type parts;
  const int tid = threadIdx.x;
  unsigned rank = 0, ctas = 1;
  if constexpr (kSplit) {
    rank = cg::this_cluster().block_rank();
    ctas = cg::this_cluster().num_blocks();
  }
  const int64_t r = blockIdx.x / ctas, rows = a.B * a.T;
  if (a.mask && !a.mask[r]) {  // the whole cluster
    if (rank != 0) return;
    if (tid == 0) {
      if (a.logps) a.logps[r] = 0.f;
      if (kEnt) a.entropy[r] = 0.f;
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
  const uint4* vec = reinterpret_cast<const uint4*>(row + g.head);
  Part p{g.head, g.tail, g.t0, 0, g.nvec};
  if constexpr (kSplit) {
    const int64_t per = (g.nvec + ctas - 1) / ctas;
    p.v0 = min((int64_t)rank * per, g.nvec);
    p.v1 = min(p.v0 + per, g.nvec);
    if (rank != 0) p.head = p.tail = 0;
  }
  const float s2 = a.s2;
  float mine;
  Stat st;
  bool fast = a.low < 0.f;
  if (fast) {
    st = cta_stat<kThreads, kEnt>(
        sweep_fast<T, kThreads, kEnt>(row, vec, p, a.low, s2, &mine), s2, warp_stat);
    fast = fabsf(st.m) * s2 <= kFastRange && st.m > 0.5f * a.low;
  }
  if (!fast)
    st = cta_stat<kThreads, kEnt>(sweep_any<T, kThreads, kEnt>(row, vec, p, s2, &mine), s2,
                                  warp_stat);
  if constexpr (kSplit) {
    // every CTA of the cluster runs before its shared memory is written
    cg::cluster_group cluster = cg::this_cluster();
    if constexpr (kTop) {
      // a part may hold fewer than k logits
      top_alternatives<T, kThreads>(row, vec, p, g.head, mine, a.k, top);
    }
    cluster.sync();
    Parts* first = cluster.map_shared_rank(&parts, 0);
    if (tid == 0) first->st[rank] = st;
    if constexpr (kTop) {
      const int n = min(a.k, top.n);
      if (tid == 0) first->n[rank] = n;
      if (tid < n) first->key[rank * GRPO_MAX_TOP_K + tid] = top.best[tid];
    }
    cluster.sync();
    if (rank != 0) return;
    st = parts.st[0];
    for (unsigned i = 1; i < ctas; ++i) st = merge<kEnt>(st, parts.st[i], s2);
  }
  if (st.m == -INFINITY) st.Z = NAN;  // no finite logit: no distribution
  if (tid == 0) finish_row<T, kEnt>(a, r, row, st);
  if constexpr (kTop) {
    if (!(st.Z <= 3.4e38f)) {  // NaN or +inf
      if (tid < a.k) {
        a.top_ids[r * a.k + tid] = -1;
        a.top_logps[r * a.k + tid] = NAN;
      }
      return;
    }
    auto put = [&](int i, unsigned long long key) {
      const float x = order_value((unsigned)(key >> 32));
      a.top_ids[r * a.k + i] = (int64_t)(0xFFFFFFFFu - (unsigned)key);
      a.top_logps[r * a.k + i] = (x - st.m) * a.inv_t - logf(st.Z);
    };
    if constexpr (kSplit) {
      // the rank of each part's keys among all of them
      const int part = tid / GRPO_MAX_TOP_K, i = tid % GRPO_MAX_TOP_K;
      static_assert(kThreads >= kMaxCluster * GRPO_MAX_TOP_K, "a thread for each key");
      if (part < (int)ctas && i < parts.n[part]) {
        const unsigned long long key = parts.key[tid];
        int above = 0;
        for (int q = 0; q < (int)ctas; ++q)
          for (int n = 0; n < parts.n[q]; ++n) above += parts.key[q * GRPO_MAX_TOP_K + n] > key;
        if (above < a.k) put(above, key);
      }
    } else {
      top_alternatives<T, kThreads>(row, vec, p, g.head, mine, a.k, top);
      if (tid < a.k) put(tid, top.best[tid]);
    }
  }
}

// Rows of at most this many bytes go to one warp, longer ones to 256 threads.
static constexpr int64_t kWarpRowBytes = 4096;
// A cluster's CTA gets at least this much of a row.
static constexpr int64_t kPartBytes = 8192;

template <typename T, int kThreads, bool kSplit>
static cudaError_t launch_logps_t(const TokenArgs& a, unsigned ctas, cudaStream_t s) {
  void (*fn)(const TokenArgs) =
      a.k > 0 ? (a.entropy ? token_logps_kernel<T, kThreads, true, true, kSplit>
                           : token_logps_kernel<T, kThreads, false, true, kSplit>)
              : (a.entropy ? token_logps_kernel<T, kThreads, true, false, kSplit>
                           : token_logps_kernel<T, kThreads, false, false, kSplit>);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.B * a.T) * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  if (kSplit) {
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, fn, a);
}

template <typename T>
static cudaError_t launch_logps_d(TokenArgs a, cudaStream_t s) {
  // The floor of the fast sweep (see Fast): 2^(s2 (low - m)) is 0 for every
  // maximum m > low / 2, and s2 |low| is below 2^30, so that the rounding of
  // a thread's mL is below 2^6.  0: not for this temperature.
  if (std::is_same<T, __half>::value)
    a.low = a.s2 >= 0.01f && a.s2 <= 1e4f ? -65504.f : 0.f;
  else
    a.low = a.s2 >= 1e-30f && a.s2 <= 1e30f ? -16384.f / a.s2 : 0.f;
  if (std::is_same<T, __nv_bfloat16>::value) a.low = __bfloat162float(__float2bfloat16(a.low));
  const int64_t bytes = a.V * (int64_t)sizeof(T), rows = a.B * a.T;
  if (bytes <= kWarpRowBytes) return launch_logps_t<T, 32, false>(a, 1, s);
  // few rows: a cluster for each, while the CTAs all run at once
  unsigned ctas = 1;
  while (ctas < kMaxCluster && rows * (2 * ctas) <= 152 * 4 && bytes / (2 * ctas) >= kPartBytes)
    ctas *= 2;
  return ctas == 1 ? launch_logps_t<T, 256, false>(a, 1, s)
                   : launch_logps_t<T, 256, true>(a, ctas, s);
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
