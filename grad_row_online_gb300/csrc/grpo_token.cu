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
//   token_logps_kernel  a warp, one CTA, or a cluster of CTAs per row
//   token_grad_kernel   a warp per row, or one CTA per row and up to 64 KB of it
//
// Both are bound by memory: 2 or 4 bytes a logit read once, against about five
// issued instructions a bf16 logit of the ten that memory speed leaves room
// for; the gradient also writes as much.  Sums are fp32: a thread adds its
// share of a row (1/32 of rows of up to 24 KB, else 1/128 or 1/256) one 16-byte
// vector's sum at a time, n of them, then a tree follows, so Z is off by at most
// n + 20 roundings of 2^-24 beside those of its terms.  n is 74 for 151936 bf16
// logits, at most 48 for shorter rows, and grows with longer ones (V / 2048,
// fp32 V / 1024).
#include <cooperative_groups.h>

#include <type_traits>

#include "grpo_around.cuh"
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

// A row's kThreads threads: a whole CTA, or one warp of a CTA of
// kWarpRows rows.
static constexpr int kWarpRows = 8;
template <int kThreads>
__device__ __forceinline__ int row_tid() {
  return kThreads == 32 ? (int)threadIdx.x % 32 : (int)threadIdx.x;
}
template <int kThreads>
__device__ __forceinline__ void row_sync() {
  if (kThreads == 32) __syncwarp();
  else __syncthreads();
}
template <int kThreads>
__host__ __device__ constexpr int rows_per_cta() { return kThreads == 32 ? kWarpRows : 1; }

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
  float cur;  // the largest logit since it was last cleared
  __device__ void init(float low, float s2) {
    m = cur = low;
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
    cur = fmaxf(cur, vmax);
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

// 16-byte loads a thread of the sweep has in flight, and the CTAs an SM that
// leaves registers for (us for 2048 rows of 304 KB at 256 threads: 6 CTAs x 4
// loads 107, 5 x 5 100.5, 5 x 6 100.6, 4 x 8 101.4, 5 x 8 134; ragged 64 x 1024
// rows of 64 KB at 128 threads: 11 x 4 342, 12 x 3 354, 10 x 5 353, 9 x 6 359).
template <int kThreads>
__host__ __device__ constexpr int in_flight() { return kThreads == 256 ? 5 : 4; }
template <int kThreads, bool kSplit>
__host__ __device__ constexpr int ctas_per_sm() {
  return kThreads == 32 ? 6 : kThreads == 128 ? 11 : kThreads == 256 && !kSplit ? 5 : 4;
}

// A thread's share of a part, its slice: the vectors v0 + tid, v0 + tid +
// kThreads, ...; one of them is a round.  For the alternatives the sweep leaves
// the maximum of every slice's segments of `rounds` rounds (kMaxSegs of them at
// most, whole groups of loads in flight).
static constexpr int kMaxSegs = 8;
template <int kThreads>
struct Segments {
  int rounds, count;
  __device__ explicit Segments(const Part& p) {
    const int all = (int)((p.v1 - p.v0 + kThreads - 1) / kThreads);
    constexpr int U = in_flight<kThreads>();
    rounds = (all + kMaxSegs * U - 1) / (kMaxSegs * U) * U;
    count = all > 0 ? (all + rounds - 1) / rounds : 0;
  }
  __device__ int64_t end(const Part& p, int seg) const {
    const int64_t e = p.v0 + (int64_t)(seg + 1) * rounds * kThreads;
    return e < p.v1 ? e : p.v1;
  }
};

// The sweep for any values: x - m is formed first, exactly near the maximum
// and without overflow to +inf, so that rows of the type's lowest value come
// out uniform.  Out of line: at ordinary temperatures few rows come here.  They
// are those whose maximum passes 2839 temperatures (kFastRange / log2 e), and
// cost a second, slower sweep: with maxima near 40, 8,192 rows of 32768 bf16
// logits take 87 us (99 with 8 alternatives) at temperatures of 0.02 and above
// and 282 us at 0.01.
template <typename T, int kThreads, bool kEnt>
__device__ __noinline__ Stat sweep_any(const T* row, const uint4* vec, Part p, float s2,
                                       float* seg_max, float* slice_max) {
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
  const Segments<kThreads> segs(p);
  const int tid = row_tid<kThreads>();
  int64_t j = p.v0 + tid;
  for (int seg = 0; seg < segs.count; ++seg) {
    float cur = -INFINITY;
    for (; j < segs.end(p, seg); j += kThreads) {
      float x[VEC];
      Storage<T>::unpack(__ldg(vec + j), x);
      st = Stat{-INFINITY, 0.f, 0.f};
      for (int e = 0; e < VEC; ++e) one(x[e]);
      cur = fmaxf(cur, st.m);
      all = merge<kEnt>(all, st, s2);
    }
    if (seg_max) seg_max[seg * kThreads + tid] = cur;
  }
  *slice_max = all.m;
  if (tid < p.head + p.tail) {
    st = Stat{-INFINITY, 0.f, 0.f};
    one(Storage<T>::load1(row + (tid < p.head ? tid : p.t0 + tid - p.head)));
    all = merge<kEnt>(all, st, s2);
  }
  return all;
}

// A logits vector, read once: not kept in L1.
__device__ __forceinline__ uint4 ld_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <typename T, int kThreads, bool kEnt, bool kTop>
__device__ __forceinline__ Stat sweep_fast(const T* row, const uint4* vec, const Part& p, float low,
                                           float s2, float* seg_max, float* slice_max) {
  Fast<T, kEnt> f;
  f.init(low, s2);
  const uint32_t low_word = Words<T>::floor_word(low);
  const int tid = row_tid<kThreads>();
  int64_t j = p.v0 + tid;
  // one form for whole groups and the last one, which the floor fills up: the
  // code is fetched cold in every launch
  auto run = [&](int64_t end) {
    constexpr int U = in_flight<kThreads>();
    for (; j < end; j += U * kThreads) {
      const int left = (int)(end - j);
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        v[u] = u * kThreads < left ? ld_once(vec + j + u * kThreads)
                                   : make_uint4(low_word, low_word, low_word, low_word);
      f.take(v, low_word, s2);
    }
  };
  if (kTop) {
    const Segments<kThreads> segs(p);
    for (int seg = 0; seg < segs.count; ++seg) {
      f.cur = low;
      run(segs.end(p, seg));
      seg_max[seg * kThreads + tid] = f.cur > low ? f.cur : -INFINITY;
    }
  } else {
    run(p.v1);
  }
  *slice_max = f.m > low ? f.m : -INFINITY;
  if (tid < p.head + p.tail)
    f.take1(Storage<T>::load1(row + (tid < p.head ? tid : p.t0 + tid - p.head)), low, s2);
  return f.stat(s2);
}

// A tree over kLanes lanes; every lane gets lane 0's result (the lanes'
// roundings may differ: a row has one value).
template <bool kEnt, int kLanes>
__device__ __forceinline__ Stat warp_stat_of(Stat st, float s2) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) {
    Stat other;
    other.m = __shfl_xor_sync(0xFFFFFFFFu, st.m, o);
    other.Z = __shfl_xor_sync(0xFFFFFFFFu, st.Z, o);
    other.D = kEnt ? __shfl_xor_sync(0xFFFFFFFFu, st.D, o) : 0.f;
    st = merge<kEnt>(st, other, s2);
  }
  st.m = __shfl_sync(0xFFFFFFFFu, st.m, 0);
  st.Z = __shfl_sync(0xFFFFFFFFu, st.Z, 0);
  st.D = kEnt ? __shfl_sync(0xFFFFFFFFu, st.D, 0) : 0.f;
  return st;
}

// The row's Stat from its threads', the same in every thread.  What threads
// wrote to shared memory before is visible after it.  kAgain: sm was used
// before.
template <int kThreads, bool kEnt, bool kAgain>
__device__ __forceinline__ Stat cta_stat(Stat st, float s2, Stat* sm) {
  st = warp_stat_of<kEnt, 32>(st, s2);
  constexpr int kWarps = kThreads / 32;
  if (kWarps == 1) {
    row_sync<kThreads>();
    return st;
  }
  if (kAgain) row_sync<kThreads>();
  if (threadIdx.x % 32 == 0) sm[threadIdx.x / 32] = st;
  row_sync<kThreads>();
  const int lane = threadIdx.x % 32;
  st = lane < kWarps ? sm[lane] : Stat{-INFINITY, 0.f, 0.f};
  return warp_stat_of<kEnt, kWarps>(st, s2);
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

// Top-k.  The k-th largest of the slices' maxima is a lower bound tau of the
// k-th largest logit, because k distinct logits reach it; and only segments
// whose maximum reaches tau can hold one of the top k.  So only those segments
// -- little more than k of them -- are read again (from L2), and their logits at
// or above tau collected; each collected key's rank among them is its place in
// the answer.  The sweep itself pays one maximum in four vectors for the
// alternatives.
template <int kThreads, int kVec>
struct TopSmem {
  static constexpr int kBatch = 4;  // vectors a thread in flight
  static constexpr int kCap = 4 * kThreads;
  static constexpr int kCompactAt = 2 * kThreads;
  float seg_max[kMaxSegs * kThreads];
  unsigned long long key[kCap];
  unsigned long long best[GRPO_MAX_TOP_K];
  unsigned ord[kThreads];                   // each slice's maximum
  uint4 group[16];                          // maxima of 64 (32) groups of slices
  unsigned short sel[kMaxSegs * kThreads];  // segments to read again: seg kThreads + tid
  int nsel, n;
  unsigned tau;
};

// put(place, key) for the k largest of sm.key[0 .. n), place 0 the largest
// (keys are distinct), each by some thread of the row.
template <int kThreads, int kVec, typename F>
__device__ __forceinline__ void rank_keys(const TopSmem<kThreads, kVec>& sm, int n, int k, F put) {
  for (int i = row_tid<kThreads>(); i < n; i += kThreads) {
    const unsigned long long mine = sm.key[i];
    int above = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) above += sm.key[j] > mine;
    if (above < k) put(above, mine);
  }
}

// What the alternatives start from, by every thread after its sweep: its
// slice's maximum, and the keys of the row's ends, which lie in no slice (fewer
// than kVec on either side: they are ranked whatever their size).
template <typename T, int kThreads>
__device__ __forceinline__ void top_begin(const T* row, const Part& p, float slice_max,
                                          TopSmem<kThreads, Storage<T>::kVec>& sm) {
  const int tid = row_tid<kThreads>();
  // an empty slice is below every logit
  sm.ord[tid] = p.v0 + tid < p.v1 ? order_of(slice_max) : 0u;
  if (tid < p.head + p.tail) {
    const int64_t v = tid < p.head ? tid : p.t0 + tid - p.head;
    sm.key[tid] = key_of(Storage<T>::load1(row + v), (unsigned)v);
  }
  if (tid == 0) {
    sm.nsel = 0;
    sm.n = p.head + p.tail;
  }
}

// put(place, key) for the alternatives, after top_begin and a barrier; returns
// how many there are (k, or all of a short part).
template <typename T, int kThreads, typename F>
__device__ int top_alternatives(const uint4* vec, const Part& p, int head, int k,
                                TopSmem<kThreads, Storage<T>::kVec>& sm, F put) {
  constexpr int VEC = Storage<T>::kVec;
  using Smem = TopSmem<kThreads, VEC>;
  const int tid = row_tid<kThreads>();
  const Segments<kThreads> segs(p);
  const unsigned mine = sm.ord[tid];
  if (tid < 32) {
    // tau: the k-th largest maximum of (at most) 64 groups of slices -- a lower
    // bound than the slices' own, at the price of a few segments more: the
    // smallest that fewer than k exceed
    constexpr int kGroups = kThreads >= 64 ? 2 : 1;  // a lane
    unsigned* group = &sm.group[0].x;
    unsigned o[kGroups];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) o[i] = 0u;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i)
      o[i % kGroups] = max(o[i % kGroups], sm.ord[tid + 32 * i]);
#pragma unroll
    for (int i = 0; i < kGroups; ++i) group[tid + 32 * i] = o[i];
    __syncwarp();
    int above[kGroups] = {};
#pragma unroll
    for (int j = 0; j < 8 * kGroups; ++j) {
      const uint4 w = sm.group[j];
#pragma unroll
      for (int i = 0; i < kGroups; ++i)
        above[i] += (w.x > o[i]) + (w.y > o[i]) + (w.z > o[i]) + (w.w > o[i]);
    }
    unsigned t = above[0] < k ? o[0] : 0xFFFFFFFFu;
    if (kGroups == 2) t = min(t, above[kGroups - 1] < k ? o[kGroups - 1] : 0xFFFFFFFFu);
    t = __reduce_min_sync(0xFFFFFFFFu, t);
    if (tid == 0) sm.tau = t;
  }
  row_sync<kThreads>();
  const unsigned tau = sm.tau;
  if (mine >= tau && mine != 0u) {
    unsigned reach = 0;
#pragma unroll
    for (int i = 0; i < kMaxSegs; ++i)
      if (i < segs.count && order_of(sm.seg_max[i * kThreads + tid]) >= tau) reach |= 1u << i;
    int to = atomicAdd(&sm.nsel, __popc(reach));
    for (; reach != 0; reach &= reach - 1)
      sm.sel[to++] = (unsigned short)((__ffs(reach) - 1) * kThreads + tid);
  }
  unsigned long long bound = (unsigned long long)tau << 32;
  row_sync<kThreads>();
  const unsigned nsel = (unsigned)sm.nsel, total = nsel * (unsigned)segs.rounds;
  const unsigned nvec = (unsigned)(p.v1 - p.v0);
  const float per_sel = 1.f / (float)nsel;
  int n = p.head + p.tail;  // keys held, the same in every thread
  // keeps the k best keys so far, which raises the bound; at least k are held
  auto compact = [&]() {
    rank_keys(sm, n, k, [&](int i, unsigned long long key) { sm.best[i] = key; });
    row_sync<kThreads>();
    if (tid < k) sm.key[tid] = sm.best[tid];
    if (tid == 0) sm.n = k;
    n = k;
    bound = sm.best[k - 1] + 1;  // the k-th itself is held
    row_sync<kThreads>();
  };
  for (unsigned q0 = 0; q0 < total; q0 += Smem::kBatch * kThreads) {
    uint4 v[Smem::kBatch];
    unsigned at[Smem::kBatch];  // vector of the part
    const int held = n;
#pragma unroll
    for (int u = 0; u < Smem::kBatch; ++u) {
      const unsigned q = q0 + tid + u * kThreads;
      at[u] = nvec;
      if (q < total) {
        // q / nsel, off by one at most where q is below 2^22
        unsigned d = q < 1u << 22 ? (unsigned)((float)q * per_sel) : q / nsel;
        int rest = (int)(q - d * nsel);
        if (rest < 0) --d, rest += (int)nsel;
        if (rest >= (int)nsel) ++d, rest -= (int)nsel;
        const unsigned seg = sm.sel[rest];
        at[u] = (seg / kThreads * segs.rounds + d) * kThreads + seg % kThreads;
        if (at[u] < nvec) v[u] = __ldg(vec + p.v0 + at[u]);
      }
    }
    // the keys of a vector that pass, with one reservation
    auto push_vec = [&](const uint4& w, unsigned i) {
      float x[VEC];
      Storage<T>::unpack(w, x);
      const unsigned e0 = (unsigned)(head + (p.v0 + i) * VEC);
      unsigned pass = 0;
#pragma unroll
      for (int e = 0; e < VEC; ++e) pass |= (key_of(x[e], e0 + e) >= bound ? 1u : 0u) << e;
      if (pass == 0) return;
      int to = atomicAdd(&sm.n, __popc(pass));
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (pass >> e & 1u) {
          if (to < Smem::kCap) sm.key[to] = key_of(x[e], e0 + e);
          ++to;
        }
    };
    if (q0 > 0) row_sync<kThreads>();  // every thread has read the last batch's sm.n
#pragma unroll
    for (int u = 0; u < Smem::kBatch; ++u)
      if (at[u] < nvec) push_vec(v[u], at[u]);
    row_sync<kThreads>();
    n = sm.n;
    if (n > Smem::kCap) {
      // ties: again, in steps that fit, from the keys that were held before
      row_sync<kThreads>();
      if (tid == 0) sm.n = held;
      row_sync<kThreads>();
      constexpr int kStep = (Smem::kCap - Smem::kCompactAt) / VEC;  // threads a step
#pragma unroll 1
      for (int u = 0; u < Smem::kBatch; ++u)
#pragma unroll 1
        for (int t0 = 0; t0 < kThreads; t0 += kStep) {
          if (tid >= t0 && tid < t0 + kStep) {
            const unsigned i = u == 0 ? at[0] : u == 1 ? at[1] : u == 2 ? at[2] : at[3];
            if (i < nvec) push_vec(__ldg(vec + p.v0 + i), i);
          }
          row_sync<kThreads>();
          n = sm.n;
          row_sync<kThreads>();
          if (n > Smem::kCompactAt) compact();
        }
    } else if (n > Smem::kCompactAt) {
      compact();
    }
  }
  rank_keys(sm, n, k, put);
  return min(n, k);
}

// A row's results, by one thread; xa is its action's logit (NaN for an id out
// of range).
template <bool kEnt>
__device__ __forceinline__ void finish_row(const TokenArgs& a, int64_t r, float xa, Stat w,
                                           float lnZ) {
  if (a.logps) a.logps[r] = (xa - w.m) * a.inv_t - lnZ;
  if (kEnt) a.entropy[r] = lnZ - kLn2f * (w.D / w.Z);
  if (a.stats) {
    a.stats[r] = w.m;
    a.stats[a.B * a.T + r] = w.Z;
  }
}

// The outputs of a masked row, by the first threads of a warp or more.
template <bool kEnt, bool kTop>
__device__ __forceinline__ void masked_row(const TokenArgs& a, int64_t r, int lane) {
  if (lane == 0) {
    if (a.logps) a.logps[r] = 0.f;
    if (kEnt) a.entropy[r] = 0.f;
    if (a.stats) {
      a.stats[r] = 0.f;
      a.stats[a.B * a.T + r] = 1.f;
    }
  }
  if (kTop && lane < a.k) {
    a.top_ids[r * a.k + lane] = -1;
    a.top_logps[r * a.k + lane] = 0.f;
  }
}

// Alternative i of row r.
__device__ __forceinline__ void put_top(const TokenArgs& a, int64_t r, int i,
                                        unsigned long long key, float m, float lnZ) {
  const float x = order_value((unsigned)(key >> 32));
  a.top_ids[r * a.k + i] = (int64_t)(0xFFFFFFFFu - (unsigned)key);
  a.top_logps[r * a.k + i] = (x - m) * a.inv_t - lnZ;
}

// Whether row r has a distribution; if not, its alternatives are marked so.
__device__ __forceinline__ bool has_top(const TokenArgs& a, int64_t r, int tid, const Stat& st) {
  if (st.Z <= 3.4e38f) return true;  // not NaN, not +inf
  if (tid < a.k) {
    a.top_ids[r * a.k + tid] = -1;
    a.top_logps[r * a.k + tid] = NAN;
  }
  return false;
}

// What the CTAs of a cluster leave in its first CTA's shared memory.
static constexpr int kMaxCluster = 8;
struct Parts {
  Stat st[kMaxCluster];
  unsigned long long key[kMaxCluster][GRPO_MAX_TOP_K];  // largest first, 0 where there is none
};

// One CTA per row, or with kSplit a cluster of CTAs, each of which takes a
// contiguous part of the row's vectors: a sweep, a tree over the threads, the
// part's alternatives, and in a cluster the parts joined by its first CTA.
// Many independent CTAs an SM keep memory busy over the ends of rows: 36,836 of
// 65,536 rows of 32768 bf16 logits take 340 us (7.1 TB/s; 44 % of the ALU pipe,
// 36 % of the exponential unit, 58 % of issue), 4,601 of 8,192 rows of 151936
// with 8 alternatives 224 us (6.2 TB/s), 4,337 rows of 128256 fp32 303 us (7.3
// TB/s).  Few rows are a chain of latencies: one of 32768 with 5 alternatives
// 5.6 us, 64 of 151936 with 20 9.7 us.  (A persistent form -- a producer warp
// streaming rows through a ring of bulk copies -- measured 387 us and 322 us on
// the first two when they took 368 and 265: its three CTAs an SM hide a row's
// end worse.)
template <typename T, int kThreads, bool kEnt, bool kTop, bool kSplit>
__global__ void __launch_bounds__(kThreads* rows_per_cta<kThreads>(),
                                  ctas_per_sm<kThreads, kSplit>())
token_logps_kernel(const TokenArgs a) {
  constexpr int VEC = Storage<T>::kVec, kRows = rows_per_cta<kThreads>();
  __shared__ Stat warp_stat[kThreads / 32];
  __shared__ typename std::conditional<kTop, TopSmem<kThreads, VEC>, int>::type tops[kRows];
  __shared__ typename std::conditional<kSplit, Parts, int>::type parts;
  const int tid = row_tid<kThreads>(), mine = kRows == 1 ? 0 : (int)threadIdx.x / 32;
  auto& top = tops[mine];
  unsigned rank = 0, ctas = 1;
  if constexpr (kSplit) {
    rank = cg::this_cluster().block_rank();
    ctas = cg::this_cluster().num_blocks();
  }
  const int64_t r = kRows == 1 ? blockIdx.x / ctas : (int64_t)blockIdx.x * kRows + mine;
  if (kRows > 1 && r >= a.B * a.T) return;
  // asked for beside the mask; its logit is asked for before the sweep, or in a
  // cluster, where the wait for the id would delay the sweep, after it
  const bool scores = tid == 0 && rank == 0 && a.logps;
  const int64_t act = scores ? a.actions[r] : -1;
  if (a.mask && !a.mask[r]) {  // the whole cluster
    if (rank == 0) masked_row<kEnt, kTop>(a, r, tid);
    return;
  }
  if constexpr (kSplit) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  unsigned b = (unsigned)r, t = 0;
  if (a.T > 1) {
    b = (unsigned)r / (unsigned)a.T;
    t = (unsigned)r - b * (unsigned)a.T;
  }
  const T* row = (const T*)a.logits + b * a.sb + t * a.st;
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
  float* seg_max = nullptr;
  if constexpr (kTop) seg_max = top.seg_max;
  Stat st;
  float slice_max, xa = NAN;
  auto ask = [&]() {
    if (!scores) return;
    if (act >= 0 && act < a.V)
      xa = Storage<T>::load1(row + act);
    else if (a.hdr)
      atomicOr(&a.hdr->status, (unsigned)GRPO_ERR_ACTION_RANGE);
  };
  if (!kSplit) ask();
  bool fast = a.low < 0.f;
  if (fast) {
    st = sweep_fast<T, kThreads, kEnt, kTop>(row, vec, p, a.low, s2, seg_max, &slice_max);
    if (kSplit) ask();
    if constexpr (kTop) top_begin<T, kThreads>(row, p, slice_max, top);
    st = cta_stat<kThreads, kEnt, false>(st, s2, warp_stat);
    fast = fabsf(st.m) * s2 <= kFastRange && st.m > 0.5f * a.low;
  }
  if (!fast) {
    st = sweep_any<T, kThreads, kEnt>(row, vec, p, s2, seg_max, &slice_max);
    if (kSplit) ask();
    if constexpr (kTop) top_begin<T, kThreads>(row, p, slice_max, top);
    st = cta_stat<kThreads, kEnt, true>(st, s2, warp_stat);
  }
  if constexpr (kSplit) {
    cg::cluster_group cluster = cg::this_cluster();
    int held = 0;
    if constexpr (kTop) {
      // a part may hold fewer than k logits
      held = top_alternatives<T, kThreads>(
          vec, p, g.head, a.k, top, [&](int i, unsigned long long key) { top.best[i] = key; });
      // parts that are not there hold nothing
      if (tid / GRPO_MAX_TOP_K >= (int)ctas)
        parts.key[tid / GRPO_MAX_TOP_K][tid % GRPO_MAX_TOP_K] = 0ull;
      row_sync<kThreads>();  // best is complete
    }
    // (arrived at the start) every CTA of the cluster runs before its shared
    // memory is written
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    Parts* first = cluster.map_shared_rank(&parts, 0);
    if (tid == 0) first->st[rank] = st;
    if constexpr (kTop) {
      if (tid < GRPO_MAX_TOP_K) first->key[rank][tid] = tid < held ? top.best[tid] : 0ull;
    }
    cluster.sync();
    if (rank != 0) return;
    const unsigned lane = tid % 32;
    st = lane < ctas ? parts.st[lane] : Stat{-INFINITY, 0.f, 0.f};
    st = warp_stat_of<kEnt, kMaxCluster>(st, s2);
  }
  if (st.m == -INFINITY) st.Z = NAN;  // no finite logit: no distribution
  const float lnZ = logf(st.Z);
  if (tid == 0) finish_row<kEnt>(a, r, xa, st, lnZ);
  if constexpr (kTop) {
    if (!has_top(a, r, tid, st)) return;
    auto put = [&](int i, unsigned long long key) { put_top(a, r, i, key, st.m, lnZ); };
    if constexpr (kSplit) {
      // a key's place: how many keys of each part lie above it, by bisection
      // of the parts' ordered lists, all parts at once
      const int part = tid / GRPO_MAX_TOP_K, i = tid % GRPO_MAX_TOP_K;
      static_assert(kThreads >= kMaxCluster * GRPO_MAX_TOP_K, "a thread for each key");
      const unsigned long long key = parts.key[part][i];
      if (key != 0ull) {
        int above[kMaxCluster];
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q) above[q] = 0;
#pragma unroll 1
        for (int step = GRPO_MAX_TOP_K / 2; step > 0; step /= 2)
#pragma unroll
          for (int q = 0; q < kMaxCluster; ++q)
            above[q] += parts.key[q][above[q] + step - 1] > key ? step : 0;
        int place = 0;
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q)
          place += above[q] + (parts.key[q][above[q]] > key);
        if (place < a.k) put(place, key);
      }
    } else {
      top_alternatives<T, kThreads>(vec, p, g.head, a.k, top, put);
    }
  }
}

// Which threads a row gets.  A warp: up to kWarpRowBytes, and up to
// kManyWarpRowBytes where there are kManyRows of them.  us by a warp / 128
// threads, for bf16 rows that are not in L2 (alone, with 8 alternatives, and the
// gradient, whose other side is 256 threads):
//           1,000 rows                      2,000 rows
//    8 KB    8.3/6.2  12.4/10.3  8.3/8.3     8.6/9.3  14.3/15.2  10.2/10.6
//   16 KB   12.0/8.3  16.5/12.3 12.2/8.6    12.5/12.3 18.6/18.4  15.2/12.5
//   24 KB   14.4/10.2 20.5/12.5 16.5/12.4   16.3/14.5 24.2/21.4  22.7/22.5
//           5,000 rows                      20,000 rows
//    8 KB   12.4/14.5 22.6/28.3 18.4/22.3   33.3/45.3 59.8/92.5  56.5/86.2
//   16 KB   19.6/20.5 30.8/33.4 36.9/32.8   57.7/63.5 91.0/111   107/114
//   24 KB   26.5/26.7 39.1/38.8 52.8/46.5   81.8/82.7 124/131    157/165
// (the two constants are a compromise: 8 KB rows cross over below 2,000 of them,
// 24 KB rows between 5,000 and 20,000.)  128 threads below kLongRowBytes, 256
// from there on and for few rows: more and smaller CTAs hide the ends of short
// rows better, and on long rows too few CTAs are left at the end.  us by 128 / 256
// threads, alone and with 8 alternatives:
//           2,000 rows            8,192 rows
//   32 KB   18.3/19.0 24.6/28.7   49.4/59.7 67.5/94.4
//   64 KB   29.5/30.3 35.4/39.1   86.4/96.2 101/130
//   72 KB   32.5/30.8 38.8/39.3   96.1/99.3 115/132
//   80 KB   35.1/32.1 41.2/39.7    106/105  124/134
//  128 KB   52.5/47.7 57.9/56.1    161/163  179/192
// (with alternatives and many rows 128 threads stay ahead beyond 72 KB; the rule
// follows the sweep alone.)
static constexpr int64_t kWarpRowBytes = 4096, kManyWarpRowBytes = 24 * 1024, kManyRows = 2000;
static constexpr int64_t kLongRowBytes = 72 * 1024;
static bool to_warps(int64_t bytes, int64_t rows) {
  return bytes <= (rows >= kManyRows ? kManyWarpRowBytes : kWarpRowBytes);
}
// A cluster's CTA gets at least this much of a row (40 rows of 64 KB: 4 parts
// 3.7 us, 8 parts 4.6 us; 152 rows: 2 parts 4.3, 4 parts 6.8).
static constexpr int64_t kPartBytes = 16384;
// Rows that are worth halving where they are two an SM (304 rows of 304 KB: 16.4
// us in halves, 21.0 whole).
static constexpr int64_t kHalvedRowBytes = 128 * 1024;
static constexpr int64_t kSms = 152;  // of a GB300

template <typename T, int kThreads, bool kSplit>
static cudaError_t launch_logps_t(const TokenArgs& a, unsigned ctas, cudaStream_t s) {
  void (*fn)(const TokenArgs) =
      a.k > 0 ? (a.entropy ? token_logps_kernel<T, kThreads, true, true, kSplit>
                           : token_logps_kernel<T, kThreads, false, true, kSplit>)
              : (a.entropy ? token_logps_kernel<T, kThreads, true, false, kSplit>
                           : token_logps_kernel<T, kThreads, false, false, kSplit>);
  cudaLaunchConfig_t cfg{};
  constexpr int kRows = rows_per_cta<kThreads>();
  cfg.gridDim = dim3((unsigned)((a.B * a.T + kRows - 1) / kRows) * ctas);
  cfg.blockDim = dim3(kThreads * kRows);
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

// The floor of the fast arithmetic (see Fast): 2^(s2 (low - m)) is 0 for every
// maximum m > low / 2, and s2 |low| is below 2^30, so that the rounding of a
// thread's mL is below 2^6.  0: not for this temperature.
template <typename T>
static float floor_of(float s2) {
  if (std::is_same<T, __half>::value) return s2 >= 0.01f && s2 <= 1e4f ? -65504.f : 0.f;
  const float low = s2 >= 1e-30f && s2 <= 1e30f ? -16384.f / s2 : 0.f;
  return std::is_same<T, float>::value ? low : __bfloat162float(__float2bfloat16(low));
}

template <typename T>
static cudaError_t launch_logps_d(TokenArgs a, cudaStream_t s) {
  a.low = floor_of<T>(a.s2);
  const int64_t bytes = a.V * (int64_t)sizeof(T), rows = a.B * a.T;
  if (to_warps(bytes, rows)) return launch_logps_t<T, 32, false>(a, 1, s);
  // few rows: a cluster for each, while its CTAs are at most two an SM (four
  // for two halves of a long row)
  unsigned ctas = 1;
  while (ctas < kMaxCluster && rows * (2 * ctas) <= 2 * kSms && bytes / (2 * ctas) >= kPartBytes)
    ctas *= 2;
  if (ctas == 1 && rows <= 2 * kSms && bytes >= kHalvedRowBytes) ctas = 2;
  if (ctas > 1) return launch_logps_t<T, 256, true>(a, ctas, s);
  return rows > 2 * kSms && bytes < kLongRowBytes ? launch_logps_t<T, 128, false>(a, 1, s)
                                                 : launch_logps_t<T, 256, false>(a, 1, s);
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
// carries no rounding of a logsumexp.  Where |m| s2 stays below kFastRange, u
// is one fused multiply-add, x s2 - mL with mL = fl(m s2); what mL rounds off,
// r = m s2 - mL, goes into the coefficients (2^u = 2^(u' - r), u = u' - r).
struct GradRow {
  float off;      // -mL, or -m
  float c0, c1;   // negated: the gradient is 2^u (c0 + c1 u)
  float ga;       // added at the action
  uint32_t low;   // floor of the logits, as a word (fused)
  bool fused;
};

// The gradient of two logits; fused: the logits are no lower than the floor
// (Fast), so u is finite.
template <bool kEnt, bool kFused>
__device__ __forceinline__ float2 token_grad2(float2 x, const GradRow& q, float s2) {
  const float2 sc = make_float2(s2, s2), off = make_float2(q.off, q.off);
  float2 u = kFused ? fma2(x, sc, off) : mul2(add2(x, off), sc);
  const float2 e = make_float2(ex2_fast(u.x), ex2_fast(u.y));
  if (!kEnt) return mul2(e, make_float2(q.c0, q.c0));
  if (!kFused) u = make_float2(fmaxf(u.x, kLowU), fmaxf(u.y, kLowU));
  return mul2(e, fma2(u, make_float2(q.c1, q.c1), make_float2(q.c0, q.c0)));
}

// A CTA takes steps of kGradVecs 16-byte vectors a thread along one row, its
// loads of a step in flight together.  Plain loads, not the read-only path:
// in place, the row is written by this kernel.
static constexpr int kGradVecs = 4;

__device__ __forceinline__ float load_plain(const float* p) { return *p; }
__device__ __forceinline__ float load_plain(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load_plain(const __half* p) { return __half2float(*p); }

// One step: this thread's vectors j0, j0 + kThreads, ...; kWhole: all of
// them inside the row.
template <typename T, int kThreads, bool kEnt, bool kFused, bool kWhole>
__device__ __forceinline__ void grad_step(const T* in, T* out, int64_t j0, int64_t nvec,
                                          int64_t act, const GradRow& q, float s2,
                                          bool together) {
  constexpr int VEC = Storage<T>::kVec;
  uint4 v[kGradVecs];
#pragma unroll
  for (int k = 0; k < kGradVecs; ++k) {
    const int64_t j = j0 + k * kThreads;
    if (!kWhole && j >= nvec) continue;
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
    const int64_t j = j0 + k * kThreads;
    if (!kWhole && j >= nvec) continue;
    float x[VEC];
    if (kEnt && kFused) {
      uint32_t* words = &v[k].x;
#pragma unroll
      for (int i = 0; i < 4; ++i) words[i] = Words<T>::at_least(words[i], q.low);
    }
    Storage<T>::unpack(v[k], x);
#pragma unroll
    for (int e = 0; e < VEC; e += 2) {
      const float2 d = token_grad2<kEnt, kFused>(make_float2(x[e], x[e + 1]), q, s2);
      x[e] = d.x;
      x[e + 1] = d.y;
    }
    const uint64_t at = (uint64_t)(act - j * VEC);
    if (at < VEC) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[e] += at == e ? q.ga : 0.f;
    }
    reinterpret_cast<uint4*>(out)[j] = Storage<T>::pack(x);
  }
}

template <typename T, int kThreads, bool kEnt, bool kFused>
__device__ __forceinline__ void grad_steps(const T* in, T* out, int64_t step0, int64_t steps,
                                           int64_t nvec, int64_t act, const GradRow& q, float s2,
                                           bool together) {
  for (int64_t i = step0; i < steps; ++i) {
    const int64_t j0 = i * (kGradVecs * kThreads) + row_tid<kThreads>();
    if ((i + 1) * (kGradVecs * kThreads) <= nvec)
      grad_step<T, kThreads, kEnt, kFused, true>(in, out, j0, nvec, act, q, s2, together);
    else
      grad_step<T, kThreads, kEnt, kFused, false>(in, out, j0, nvec, act, q, s2, together);
  }
}

// CTA c of a row takes its steps [c per, (c + 1) per); the row's unaligned
// ends go to its first CTA.  Bound by memory: 64 x 512 rows of 32768 bf16 logits
// (18,404 active) with an entropy term 498 us, 6.7 TB/s; 16 x 256 rows of
// 128256 fp32 434 us, 6.9 TB/s: the rate of a copy.  Four steps a CTA against
// one: 182 and 213 us on 8,192 rows of 32768; more CTAs an SM with fewer
// registers (6 x 4 vectors, 8 x 2) 234 and 202 us.  Short rows go to warps (see
// to_warps).
template <typename T, int kThreads, bool kEnt>
__global__ void __launch_bounds__(kThreads* rows_per_cta<kThreads>(), 4)
token_grad_kernel(const TokenGradArgs a, unsigned ctas, unsigned per) {
  constexpr int kRows = rows_per_cta<kThreads>();
  const int tid = row_tid<kThreads>();
  const int64_t rows = a.B * a.T;
  const int64_t r = kRows == 1 ? blockIdx.x / ctas
                               : (int64_t)blockIdx.x * kRows + threadIdx.x / 32;
  const unsigned cta = kRows == 1 ? blockIdx.x % ctas : 0;
  if (kRows > 1 && r >= rows) return;
  // the row's scalars, all asked for at once
  const bool on = !a.mask || a.mask[r];
  float w = a.dlogp ? a.dlogp[r] : 0.f;
  float h = kEnt ? a.dent[r] : 0.f;
  const float H = kEnt ? a.entropy[r] : 0.f;
  const float m = a.stats[r], Z = a.stats[rows + r];
  const int64_t id = a.dlogp ? a.actions[r] : 0;
  if (!on && a.skip_masked) return;
  const unsigned b = (unsigned)r / (unsigned)a.T, t = (unsigned)r % (unsigned)a.T;
  T* grow = (T*)a.grad + b * a.gsb + t * a.gst;
  const T* row = (const T*)a.logits + b * a.sb + t * a.st;
  const Geom<T> g(grow, a.V);  // by the gradient's alignment: the stores are whole
  uint4* out = reinterpret_cast<uint4*>(grow + g.head);
  const int64_t steps = min((int64_t)(cta + 1) * per,
                            (g.nvec + kGradVecs * kThreads - 1) / (kGradVecs * kThreads));
  const int ev = tid < g.head ? tid : (int)g.t0 + tid - g.head;  // this thread's end element
  const bool edge = cta == 0 && tid < g.head + g.tail;
  if (!on || (w == 0.f && h == 0.f)) {
    if (edge) Storage<T>::store1(grow + ev, 0.f);
    for (int64_t i = (int64_t)cta * per; i < steps; ++i)
#pragma unroll
      for (int k = 0; k < kGradVecs; ++k) {
        const int64_t j = (i * kGradVecs + k) * kThreads + tid;
        if (j < g.nvec) out[j] = make_uint4(0u, 0u, 0u, 0u);
      }
    return;
  }
  GradRow q;
  const float mL = m * a.s2;
  q.fused = a.low < 0.f && fabsf(mL) <= kFastRange && m > 0.5f * a.low;
  q.low = Words<T>::floor_word(a.low);
  q.off = q.fused ? -mL : -m;
  const float rest = q.fused ? __fmaf_rn(m, a.s2, -mL) : 0.f;
  const float f = -a.inv_t * ex2_fast(-rest) / Z;
  q.c1 = f * kLn2f * h;
  q.c0 = (kEnt && h != 0.f) ? f * (w + h * (H - logf(Z))) - q.c1 * rest : f * w;
  q.ga = a.inv_t * w;
  int64_t act = -1;
  if (w != 0.f) {
    act = id;
    if (id < 0 || id >= a.V) {
      q.c0 = NAN;
      if (a.hdr && cta == 0 && tid == 0) atomicOr(&a.hdr->status, (unsigned)GRPO_ERR_ACTION_RANGE);
    }
  }
  if (edge) {
    float x = load_plain(row + ev);
    if (q.fused && x < a.low) x = a.low;
    const float2 x2 = make_float2(x, x);
    float d = q.fused ? token_grad2<kEnt, true>(x2, q, a.s2).x
                      : token_grad2<kEnt, false>(x2, q, a.s2).x;
    if (ev == act) d += q.ga;
    Storage<T>::store1(grow + ev, d);
  }
  const bool together = (((uintptr_t)grow ^ (uintptr_t)row) & 15) == 0;
  const T* in = row + g.head;
  T* o = grow + g.head;
  act -= g.head;  // among the vectors' elements
  if (q.fused)
    grad_steps<T, kThreads, kEnt, true>(in, o, (int64_t)cta * per, steps, g.nvec, act, q, a.s2, together);
  else
    grad_steps<T, kThreads, kEnt, false>(in, o, (int64_t)cta * per, steps, g.nvec, act, q, a.s2, together);
}

template <typename T, int kThreads>
static cudaError_t launch_grad_t(const TokenGradArgs& a, cudaStream_t s) {
  const int64_t step = (int64_t)kThreads * kGradVecs * Storage<T>::kVec;
  const int64_t steps = (a.V + step - 1) / step, rows = a.B * a.T;
  constexpr int kRows = rows_per_cta<kThreads>();
  // steps a CTA: all of a warp's row; up to 4, one where the rows alone are too
  // few to fill the GPU several times over, and enough to keep the grid below
  // 2^31 CTAs
  int64_t per = kRows > 1 ? steps : 1;
  while (per < 4 && per < steps && rows * ((steps + 2 * per - 1) / (2 * per)) >= kSms * 32) per *= 2;
  while (rows * ((steps + per - 1) / per) > 0x7FFFFFFF) per *= 2;
  const int64_t ctas = (steps + per - 1) / per;
  const unsigned grid = (unsigned)(kRows > 1 ? (rows + kRows - 1) / kRows : rows * ctas);
  auto fn = a.dent ? token_grad_kernel<T, kThreads, true> : token_grad_kernel<T, kThreads, false>;
  fn<<<grid, kThreads * kRows, 0, s>>>(a, (unsigned)ctas, (unsigned)per);
  return cudaGetLastError();
}

template <typename T>
static cudaError_t launch_grad_d(TokenGradArgs a, cudaStream_t s) {
  a.low = floor_of<T>(a.s2);
  const int64_t bytes = a.V * (int64_t)sizeof(T);
  return to_warps(bytes, a.B * a.T) ? launch_grad_t<T, 32>(a, s) : launch_grad_t<T, 256>(a, s);
}

cudaError_t launch_token_grad(const TokenGradArgs& a, grpo_dtype_t dt, cudaStream_t s) {
  switch (dt) {
    case GRPO_F32: return launch_grad_d<float>(a, s);
    case GRPO_BF16: return launch_grad_d<__nv_bfloat16>(a, s);
    default: return launch_grad_d<__half>(a, s);
  }
}

}  // namespace grpo
