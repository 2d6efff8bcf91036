// grpo_linear.cu -- log-probs of given tokens from hidden states and the
// head's weight (grpo_linear_logps) and their gradient to both
// (grpo_linear_logps_grad), without the logits in memory.
//
//   x_v = sum_k h_k W_vk,  m = max_v x_v,  Z = sum_v exp(s (x_v - m))
//   logp = s (x_a - m) - log Z,   H = log Z - sum_v e_v log e_v / Z
//   d_v  = s (dlogp (1[v = a] - p_v) - dH p_v (log p_v + H))
//   dh   = d W,   dW = d^T h
//
// One kernel does the four products on the tensor cores: the logits with
// their online softmax (kStats), the logits again with their gradient
// (kGrad), and the two products of that gradient, in one launch (kBack).  The
// gradient of the logits exists for a piece of the vocabulary at a time.
// Every kernel here may be set up while the one before it ends, and waits for
// that before it touches memory.
#include <cuda.h>

#include <algorithm>
#include <type_traits>

#include "grpo_index.cuh"
#include "grpo_linear.cuh"
#include "grpo_tensor.cuh"

namespace grpo {
namespace {

using namespace tc;

enum Epi { kStats, kGrad, kBack };

static constexpr int kThreads = 384;  // warps: loads, products, tensor memory, (idle), 8 of results
static constexpr int kBlk = 64;       // elements of the reduction a stage holds: 128 bytes a row
static constexpr int kRows = 128;     // rows of a CTA's tile (lanes of tensor memory)
static constexpr int kPad = 256;      // packed rows are padded to the rows of a pair's tile
static constexpr int kMaxStages = 12;
static constexpr int kSmem = 227 * 1024 - 320;  // of a CTA's, beside the barriers
// kParts: registers a thread of the first four warps and of the others, of 168 at the launch
static constexpr int kFewRegs = 56, kManyRegs = 224;
static_assert(4 * kFewRegs + 8 * kManyRegs <= 12 * 168, "what the launch gives");
static constexpr int kTurn = 33;          // words of a row in the results' 16 x 32 turn

struct Product {
  CUtensorMap a, b;
  const int* count;  // packed rows, on the device; nullptr: rows
  int rows;
  int v0, vp;     // the piece of the vocabulary
  int K;          // width
  int bn, nt;     // columns of a tile, tiles of columns
  int kb;         // blocks of the reduction where it is not over the rows
  int on;         // kBack: this product is wanted
  int least;      // kBack, dW: what a tile takes at least, for its results, in blocks
  int splits;     // kBack, dh: parts of the reduction
  int pairs;      // products of planes: 1, 2 (of A's two), or 6 of three planes each
  int a_rows;     // rows of A that are loaded (kCg 1; the others' results are not used)
  int sums;       // kParts: blocks that one accumulator sums up
  int kc;         // kSets: of accumulators that a logit's reduction is cut into, in order
  int slot, bufs; // columns of a set; tiles that are in flight, 1 or 2
  int want_entropy; // kStats: D is wanted; kGrad: c1 is not 0
  int run;        // kStats: one record of a CTA's tiles, which are of the same rows
  int stages, mb; // tiles of rows that are taken together
  uint32_t fmt;
  float s, s2;
  // rows
  const int* idx;        // source row of a packed row; nullptr: itself
  const int64_t* actions;
  // kStats
  float4* part;          // [nt][rpad] of (m, Z, D)
  float* xa;             // [rpad]
  int rpad;
  // kGrad
  const float4* coef;    // [rpad] of (m, c0, c1, s dlogp)
  const int* target;     // [rpad]
  __nv_bfloat16* d;      // [planes][rpad][ldd]
  int planes;
  int64_t ldd;
  const unsigned* bound; // f16: largest |d|, as bits; nullptr: no scaling
  // kBack.  dh: fp32 sums, or results
  float* acc;            // [splits][rpad][ldacc]
  int64_t ldacc;
  int acc_old, acc_new;  // sums are there, are left there
  void* out;
  int64_t T, osb, ost;   // rows of the results
  int odt;
  const void* add;       // dW
  int64_t asv;
  unsigned* status;
};

struct Tile {
  int m0, n0, k0, k1, split;
  bool weight;  // kBack: of dW
};

struct Stats {
  float m, Z, D;
};

// Products of planes, the small ones first: x = x0 + x1 + x2 in bf16, and what
// is left out is below 2^-26 of |x| |w|.
__device__ __constant__ signed char kPairs[6][2] = {{0, 2}, {2, 0}, {1, 1}, {0, 1}, {1, 0}, {0, 0}};

// the planes of product p of a block
__device__ __forceinline__ int2 planes_of(int pairs, int p) {
  return pairs == 6 ? make_int2(kPairs[p][0], kPairs[p][1]) : make_int2(pairs - 1 - p, 0);
}

// 2^e with the largest |d| times it in [2^14, 2^15): fp16 has no range of its
// own to spare, and 2^-28 of the largest value is still a normal number.
__device__ __forceinline__ float range_scale(unsigned bits) {
  const int e = (int)(bits >> 23) - 127;
  if (bits == 0 || e > 126) return 1.f;
  return __int_as_float((min(14 - e, 126) + 127) << 23);
}

__device__ __forceinline__ void launched_early() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename T>
__device__ __forceinline__ float load1(const T* p) { return Storage<T>::load1(p); }

// Two fp32 operations in one instruction: a warp of results has less to issue
// beside the thread that feeds the tensor cores.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mov.b64 c, {%6, %7};\n fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mul.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// the largest / smallest of 32, NaN left out
__device__ __forceinline__ float max32(const float (&v)[32]) {
  float m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = max3(v[i], v[i + 4], v[i + 8]);
#pragma unroll
  for (int i = 12; i < 28; i += 8)
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = max3(m[j], v[i + j], v[i + j + 4]);
#pragma unroll
  for (int j = 0; j < 4; ++j) m[j] = fmaxf(m[j], v[28 + j]);
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}
__device__ __forceinline__ float min32(const float (&v)[32]) {
  float m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = min3(v[i], v[i + 4], v[i + 8]);
#pragma unroll
  for (int i = 12; i < 28; i += 8)
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = min3(m[j], v[i + j], v[i + j + 4]);
#pragma unroll
  for (int j = 0; j < 4; ++j) m[j] = fminf(m[j], v[28 + j]);
  return fminf(fminf(m[0], m[1]), fminf(m[2], m[3]));
}

__device__ __forceinline__ void store32(void* p, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x),
               "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

__device__ __forceinline__ void store_if(uintptr_t p, unsigned v, bool yes) {
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n @p st.global.b32 [%0], %1;\n}" ::"l"(p),
               "r"(v), "r"((unsigned)yes)
               : "memory");
}

// 32 results of a row, times `scale` plus `add`'s, in 16- or 32-byte stores.
template <typename T>
__device__ __forceinline__ void store_row(T* out, const T* add, const float (&v)[32], float scale) {
  constexpr int kVec = Storage<T>::kVec;
#pragma unroll
  for (int i = 0; i < 32; i += 2 * kVec) {
    float f[2 * kVec];
#pragma unroll
    for (int j = 0; j < 2 * kVec; ++j) f[j] = v[i + j] * scale;
    if (add) {
#pragma unroll
      for (int j = 0; j < 2 * kVec; ++j) f[j] += load1(add + i + j);
    }
    const uint4 a = Storage<T>::pack(f), b = Storage<T>::pack(f + kVec);
    if (((uintptr_t)out & 31) == 0) {
      store32(out + i, a, b);
    } else {
      *reinterpret_cast<uint4*>(out + i) = a;
      *reinterpret_cast<uint4*>(out + i + kVec) = b;
    }
  }
}

// Where the rows of a warp's results start, in elements (-1: no row), and half
// of the results on their turn.
struct alignas(16) Turn {
  int64_t at[32], add_at[32];
  float v[16 * kTurn];  // (or 32 x 16 words)
};

// A warp's 32 x 32 results, a row a lane, column `c` of the row on, `n` columns
// of them inside.  Rows that 16-byte stores cannot take (or the last columns)
// are turned, so that a store of the warp covers adjacent elements of one row:
// a lane's own row would be 32 stores of single elements in 32 places each.
template <typename T>
__device__ __forceinline__ void store_tile(T* out, const T* add, int c, const float (&v)[32], int n,
                                           float scale, Turn& turn) {
  const int lane = threadIdx.x & 31;
  const int64_t at = turn.at[lane];
  const bool whole = at < 0 || ((uintptr_t)(out + at + c) & 15) == 0;
  if (n >= 32 && __all_sync(~0u, whole)) {
    if (at >= 0) store_row(out + at + c, add ? add + turn.add_at[lane] + c : nullptr, v, scale);
    return;
  }
  if constexpr (sizeof(T) == 2) {
    if (!add && n >= 32) {
      // pairs of elements in words, two rows a store; a row that starts in the
      // middle of a word has its pairs put together anew
      unsigned* words = reinterpret_cast<unsigned*>(turn.v);
      auto shuffle = [](int r) { return (r & 6) << 1; };  // (for the banks)
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 32; i += 8) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = v[i + j] * scale;
        const uint4 w = Storage<T>::pack(f);
        *reinterpret_cast<uint4*>(words + lane * 16 + ((i / 2) ^ shuffle(lane))) = w;
      }
      __syncwarp();
      const int l = lane & 15, half = lane >> 4;
      const uintptr_t base = (uintptr_t)(out + c);
#pragma unroll 4
      for (int r0 = 0; r0 < 32; r0 += 2) {
        const int r = r0 + half;
        const int64_t row = turn.at[r];
        const unsigned w = words[r * 16 + (l ^ shuffle(r))], before = words[r * 16 + ((l - (l > 0)) ^ shuffle(r))];
        const uintptr_t to = base + (uintptr_t)(row * 2);
        const unsigned odd = (unsigned)to & 2u;
        store_if(to + 4u * l - odd, __funnelshift_l(before, w, odd * 8u), row >= 0 && l >= (int)(odd >> 1));
      }
      // the ends of a shifted row: its first element and its last
      if (at >= 0 && ((uintptr_t)(out + at + c) & 2)) {
        Storage<T>::store1(out + at + c, v[0] * scale);
        Storage<T>::store1(out + at + c + 31, v[31] * scale);
      }
      __syncwarp();
      return;
    }
  }
#pragma unroll
  for (int h = 0; h < 32; h += 16) {
    __syncwarp();
    if (lane >= h && lane < h + 16) {
#pragma unroll
      for (int i = 0; i < 32; ++i) turn.v[(lane - h) * kTurn + i] = v[i] * scale;
    }
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 16; q += 8) {  // (eight rows' reads in flight together)
      int64_t to[8];
      float x[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        to[r] = lane < n ? turn.at[h + q + r] : -1;
        x[r] = turn.v[(q + r) * kTurn + lane];
      }
      if (add) {
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (to[r] >= 0) x[r] += load1(add + turn.add_at[h + q + r] + c + lane);
      }
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (to[r] >= 0) Storage<T>::store1(out + to[r] + c + lane, x[r]);
    }
  }
  __syncwarp();
}

// `n` records into one: their largest maximum first, then one scaled sum.
template <int n>
__device__ __forceinline__ float4 join(const float4 (&x)[n], float s2) {
  float m = x[0].x;
#pragma unroll
  for (int i = 1; i < n; ++i) m = fmaxf(m, x[i].x);
  float4 y = make_float4(m, 0.f, 0.f, 0.f);
  // (nothing above -inf in any: Z is 0 in all, or NaN)
  const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
  for (int i = 0; i < n; ++i) {
    const float u = fmaxf((x[i].x - ref) * s2, -1000.f), k = exp2f(u);
    y.y += x[i].y * k;
    y.z += k * fmaf(x[i].y, u, x[i].z);
  }
  return y;
}

// The record of a row from the two warps that have its columns (at < 0: none).
__device__ __forceinline__ void record(const Product& g, const Stats& st, Stats* pair, int side,
                                       int64_t at) {
  const int row = threadIdx.x & 127;
  float4 x[2] = {make_float4(st.m, st.Z, st.D, 0.f)};
  asm volatile("bar.sync 1, 256;" ::: "memory");  // (the record before has been read)
  if (side == 1) pair[row] = Stats{x[0].x, x[0].y, x[0].z};
  asm volatile("bar.sync 1, 256;" ::: "memory");
  if (side == 1) return;
  x[1] = make_float4(pair[row].m, pair[row].Z, pair[row].D, 0.f);
  if (at >= 0) g.part[at] = join(x, g.s2);
}

// What a thread needs of its row, read while the tile's products run.
struct RowData {
  int64_t id;  // the token, -1: none
  float4 q;    // kGrad: the coefficients
};
template <int kEpi>
__device__ __forceinline__ RowData row_data(const Product& g, const Tile& t, int rank, int count) {
  RowData x{-1, make_float4(0.f, 0.f, 0.f, 0.f)};
  const int r = t.m0 + rank * kRows + (threadIdx.x & 127);
  if (r >= count) return x;
  if (kEpi == kStats && g.actions) x.id = g.actions[g.idx ? g.idx[r] : r];
  if (kEpi == kGrad) x.id = g.target[r], x.q = g.coef[r];
  return x;
}

// ---- results of a tile: a thread has one row; two warps share 32 rows and take
// blocks of 32 columns in turn, from tensor memory at `tm` or (kParts) added
// up in `acc`
template <int kCg, int kEpi, bool kParts, bool kSets>
__device__ __forceinline__ void results(const Product& g, const Tile& t, int rank, int count,
                                        uint32_t tm, bool have, bool failed,
                                        float (&acc)[kParts ? 4 : 1][32], Stats& st, Turn& turn,
                                        Stats* pair, const RowData& row) {
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3;
  const int side = (int)(threadIdx.x >> 5) / 4 - 1;
  const int r = t.m0 + rank * kRows + quad * 32 + lane;
  const float bad = __int_as_float(0x7FFFFFFF);
  // f(c, columns c .. c + 31) for this warp's blocks below `end`
  auto blocks = [&](int end, auto&& f) {
    if constexpr (kParts) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (32 * side + 64 * j < end) f(32 * side + 64 * j, acc[j]);
    } else {
      for (int c = 32 * side; c < end; c += 64) {
        float v[32];
        __syncwarp();
        if (have) {
          tmem_ld32(tm + c, v);
          tmem_wait(v);
          if constexpr (kSets) {
            for (int j = 1; j < g.kc; ++j) {
              float w[32];
              tmem_ld32(tm + j * g.slot + c, w);
              tmem_wait(w);
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] += w[i];
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = failed ? bad : 0.f;
        }
        f(c, v);
      }
    }
  };
  if constexpr (kEpi == kStats) {
    const int n = min(g.bn, g.vp - t.n0);
    const bool live = r < count;
    const int64_t id = row.id - t.n0;
    const int a = id >= 0 && id < n ? (int)id : -1;
    // sums of 2^u and 2^u u, u = (x - m) s2
    float m = st.m, Z = st.Z, D = st.D, xa = 0.f;
    blocks(n, [&](int c, float(&v)[32]) {
      if (c + 32 > n) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = c + i < n ? v[i] : -INFINITY;
      }
      const float cm = max32(v);
      if (cm > m) {
        const float u = fmaxf((m - cm) * g.s2, -1000.f);
        const float k = exp2f(u);
        D = k * fmaf(Z, u, D);
        Z *= k;
        m = cm;
      }
      // (a row of -inf so far: 2^-inf = 0 against any finite reference)
      const float ref = m == -INFINITY ? 0.f : m;
      const float2 s2 = make_float2(g.s2, g.s2), r2 = make_float2(-ref, -ref);
      float2 z2[2], d2[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) z2[i] = d2[i] = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const float2 u = mul2(add2(make_float2(v[i], v[i + 1]), r2), s2);
        const float2 e = make_float2(ex2_fast(u.x), ex2_fast(u.y));
        z2[i / 2 & 1] = add2(z2[i / 2 & 1], e);
        if (g.want_entropy) d2[i / 2 & 1] = fma2(e, u, d2[i / 2 & 1]);
      }
      z2[0] = add2(z2[0], z2[1]);
      d2[0] = add2(d2[0], d2[1]);
      float d = d2[0].x + d2[0].y;
      if (!(fabsf(d) < INFINITY)) {  // (a logit of -inf: its term is 0, not 0 x inf)
        d = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float u = (v[i] - ref) * g.s2;
          d = fmaf(ex2_fast(u), fmaxf(u, -1000.f), d);
        }
      }
      Z += z2[0].x + z2[0].y;
      D += d;
      if (__any_sync(~0u, a >= c && a < c + 32)) {
#pragma unroll
        for (int i = 0; i < 32; ++i) xa = a == c + i ? v[i] : xa;
      }
    });
    if (a >= 0 && (a >> 5 & 1) == side) g.xa[r] = xa;
    st = Stats{m, Z, D};
    if (!g.run) {
      record(g, st, pair, side, live ? (int64_t)(t.n0 / g.bn) * g.rpad + r : -1);
      st = Stats{-INFINITY, 0.f, 0.f};
    }
  } else if constexpr (kEpi == kGrad) {
    const int n = min(g.bn, g.vp - t.n0);
    const bool live = r < count;
    const float4 q = row.q;
    const int a = live ? (int)row.id - g.v0 - t.n0 : -1;
    const float scale = g.bound ? range_scale(*g.bound) : 1.f;
    const float c0 = -q.y * scale, c1 = -q.z * scale;
    const float2 s2 = make_float2(g.s2, g.s2), r2 = make_float2(-q.x, -q.x);
    const float2 c02 = make_float2(c0, c0), c12 = make_float2(c1, c1);
    __nv_bfloat16* dst = g.d + (int64_t)r * g.ldd + t.n0;
    blocks(g.bn, [&](int c, float(&v)[32]) {
      // (far below the others, -inf among them: 0, not 0 x inf)
      const bool low = g.want_entropy && !((min32(v) - q.x) * g.s2 > -1e20f);
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        float2 u = mul2(add2(make_float2(v[i], v[i + 1]), r2), s2);
        float2 w = make_float2(ex2_fast(u.x), ex2_fast(u.y));
        if (g.want_entropy) {
          if (low) u = make_float2(fmaxf(u.x, -1000.f), fmaxf(u.y, -1000.f));
          w = mul2(w, fma2(c12, u, c02));
        } else {
          w = mul2(w, c02);
        }
        v[i] = w.x, v[i + 1] = w.y;
      }
      if (__any_sync(~0u, a >= c && a < c + 32)) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] += a == c + i ? q.w * scale : 0.f;
      }
      // rows and columns behind the last ones are read by the products to come
      if (!live || c + 32 > n || failed) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = live && c + i < n ? (failed ? bad : v[i]) : 0.f;
      }
      for (int p = 0; p < g.planes; ++p) {
        __nv_bfloat16* to = dst + (int64_t)p * g.rpad * g.ldd + c;
        if (g.fmt == 0) {
#pragma unroll
          for (int i = 0; i < 32; i += 16)
            store32(to + i, Storage<__half>::pack(v + i), Storage<__half>::pack(v + i + 8));
        } else {
#pragma unroll
          for (int i = 0; i < 32; i += 16)
            store32(to + i, Storage<__nv_bfloat16>::pack(v + i), Storage<__nv_bfloat16>::pack(v + i + 8));
        }
        if (p + 1 < g.planes) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            v[i] -= g.fmt == 0 ? __half2float(__float2half_rn(v[i])) : __bfloat162float(__float2bfloat16_rn(v[i]));
        }
      }
    });
  } else {
    const float scale = g.bound ? 1.f / range_scale(*g.bound) : 1.f;
    const int64_t dst = t.weight ? (r < g.vp ? g.v0 + r : -1)
                                        : (r < count ? (g.idx ? g.idx[r] : r) : -1);
    __syncwarp();
    turn.at[lane] = dst < 0    ? -1
                    : t.weight ? dst * g.ost + t.n0
                               : dst / g.T * g.osb + dst % g.T * g.ost + t.n0;
    turn.add_at[lane] = t.weight ? dst * g.asv + t.n0 : 0;
    __syncwarp();
    blocks(min(g.bn, g.K - t.n0), [&](int c, float(&v)[32]) {
      const int n = min(32, g.K - t.n0 - c);
      if (!t.weight && g.acc) {
        // (the last columns are padding; rows without a source have no sums)
        float* sums = g.acc + ((int64_t)t.split * g.rpad + r) * g.ldacc + t.n0 + c;
        if (g.acc_old && dst >= 0) {
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 o = *reinterpret_cast<const float4*>(sums + i);
            v[i] += o.x, v[i + 1] += o.y, v[i + 2] += o.z, v[i + 3] += o.w;
          }
        }
        if (g.acc_new) {
          if (dst >= 0) store_row<float>(sums, nullptr, v, 1.f);
          return;
        }
      }
      const void* add = t.weight ? g.add : nullptr;
      if (g.odt == GRPO_F32)
        store_tile((float*)g.out, (const float*)add, c, v, n, scale, turn);
      else if (g.odt == GRPO_BF16)
        store_tile((__nv_bfloat16*)g.out, (const __nv_bfloat16*)add, c, v, n, scale, turn);
      else
        store_tile((__half*)g.out, (const __half*)add, c, v, n, scale, turn);
    });
  }
}

// The products.  A CTA (kCg 1: tiles of 128 rows) or a pair of CTAs (kCg 2:
// 256 rows, each CTA holds half of either operand's tile) takes tiles in turn;
// one thread asks for the operands' blocks, one issues the products into one
// of two sets of accumulators, eight warps turn the other into results.
//
// An accumulator is rounded towards zero at every step, 16 products long, so
// a sum's error grows with its length and has its sign.  kParts: sums of `sums`
// blocks each are added up in registers, rounded to nearest (fp32 operands,
// and widths whose logits would be off by more than fp32 log-probs are).  kSets:
// a logit's parts have accumulators of their own instead, one tile at a time.
// (kParts spills: 128 sums and 32 operands a thread in the 168 registers that the
// compiler has, 0.9 to 1.5 KB of stores in the code; the tensor pipe is busy 73 to
// 86 % of the time, 91 to 95 without parts.)
//
// Bound by the tensor cores where tokens are many: a tile is 256 x 256, the most
// that two sets of accumulators leave room for, so that an operand's element
// read from L2 serves 256 products, and whatever a result costs (kStats: an
// exponent and four packed fp32 operations for two logits) has to be issued
// beside the next tile's products.  2,048 x 2,048 x 32,768, bf16: kStats 144 us
// (1.90 PFLOP/s, tensor pipe busy 95 %), kGrad 151 us (94 %), kBack 300 us for
// both products (91 %; the ends of its pieces); 16,384 tokens, 9,209 of them
// taking part, x 2,048 x 151,936: 2.77 ms, 99.7 %.  Bound by memory up to 128
// tokens, which take single CTAs with the weight as B: 64 x 4,096 x 32,768 in
// 50 us, 5.4 TB/s, 64 x 4,096 x 151,936 in 190 us, 6.6 TB/s.  One tensor map
// a load of 64 elements (128 bytes) a row: what the swizzle holds; 6 to 12
// stages of them in flight.
//
// The gradient of the logits, d, is rounded to the operands' type for kBack:
// the tensor cores take 16-bit operands, and two planes of d would double the
// work of two of three products.  It adds half a step of the type to each
// term, 1.7e-3 to 2.4e-3 in norm for bf16 (1.7e-3 is the results' own rounding).
// Where dW leaves in fp32, that rounding would be all of its error, and dW takes
// a second plane of d with what the first one lacks: 1.6e-3 becomes 1e-6 to
// 5e-6, and 4,608 x 2,048 x 151,936 bf16 takes 7.40 ms where it took 5.16.
template <int kCg, int kEpi, bool kParts, bool kSets>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ Product g,
                   const __grid_constant__ std::conditional_t<kEpi == kBack, Product, int> w) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_full[kMaxStages], s_empty[kMaxStages], s_done[2], s_free[2];
  __shared__ uint32_t s_tmem;
  __shared__ Turn s_turn[kEpi == kBack ? 8 : 1];
  __shared__ Stats s_pair[kEpi == kStats ? kRows : 1];
  constexpr bool kBmn = kEpi == kBack;
  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = kCg == 2 ? cluster_rank() : 0u;
  const int half = g.bn / kCg;  // columns of B in this CTA
  const uint32_t a_bytes = (uint32_t)g.a_rows * 128u, b_bytes = (uint32_t)half * 128u;
  const uint32_t stage_bytes = a_bytes + ((b_bytes + 1023u) & ~1023u);

  if (threadIdx.x == 0) {
    tma_prefetch(&g.a);
    tma_prefetch(&g.b);
    if constexpr (kEpi == kBack) {
      tma_prefetch(&w.a);
      tma_prefetch(&w.b);
    }
    for (int i = 0; i < g.stages; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&s_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_done[i]), 1);
      mbar_init(smem_u32(&s_free[i]), 8 * kCg);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) tmem_alloc<kCg>(smem_u32(&s_tmem), 512);
  fence_before();
  __syncthreads();
  if (kCg == 2) cluster_sync();
  fence_after();
  const uint32_t tmem = s_tmem;
  launched_early();

  const int count = g.count ? *g.count : g.rows;
  constexpr int kTile = kRows * kCg;  // rows of a tile
  const int mt = (count + kTile - 1) / kTile, per = mt * g.nt;
  const int first = blockIdx.x / kCg, step = gridDim.x / kCg;
  // tiles: (kBack) parts of the reduction, then blocks of mb rows of tiles, in
  // which the rows' tiles come first
  auto place = [&](Tile& x, int u, int mt, int mb, int nt, int bn) {
    const TilePlace at = tile_place(u, mt, mb, nt);
    x.m0 = at.row * kTile;
    x.n0 = at.col * bn;
  };
  // the j-th tile of this cluster: whether there is one, and which
  auto tile = [&](int j, Tile& x) {
    x.weight = false;
    x.split = 0;
    x.k0 = 0;
    x.k1 = g.kb;
    if constexpr (kEpi != kBack) {
      const int i = first + j * step;
      if (i >= per) return false;
      place(x, i, mt, g.mb, g.nt, g.bn);
    } else {
      // dh's tiles, which are long, in turn; then dW's, of which the clusters
      // with one long tile less take as many more as that one lasts
      const int hidden = g.on ? per * g.splits : 0, wmt = (w.vp + kTile - 1) / kTile;
      const int weight = w.on ? wmt * w.nt : 0, wkb = (count + kBlk - 1) / kBlk;
      const int mine = hidden > first ? (hidden - first + step - 1) / step : 0;
      if (j < mine) {
        const int i = first + j * step;
        x.split = i / per;
        place(x, i - x.split * per, mt, g.mb, g.nt, g.bn);
        x.k0 = (int)((int64_t)g.kb * x.split / g.splits);
        x.k1 = (int)((int64_t)g.kb * (x.split + 1) / g.splits);
        return true;
      }
      j -= mine;
      const int busy = hidden % step, idle = step - busy;  // clusters with one tile more, less
      const int lasts = max(wkb * w.pairs, w.least);
      const int64_t more = busy ? (g.kb * g.pairs / g.splits + lasts / 2) / lasts : 0;
      const int extra = (int)min((int64_t)weight, more * idle);
      const int at = first - busy, mine2 = first >= busy && extra > at ? (extra - at + idle - 1) / idle : 0;
      const int i = j < mine2 ? at + j * idle : extra + first + (j - mine2) * step;
      if (i >= weight) return false;
      x.weight = true;
      x.k1 = wkb;
      place(x, i, wmt, w.mb, w.nt, w.bn);
    }
    return true;
  };
  auto of = [&](const Tile& x) -> const Product* {
    if constexpr (kEpi == kBack) return x.weight ? &w : &g;
    else return &g;
  };
  // (kParts) where the part of a tile's n blocks that starts at k ends
  auto part_end = [&](const Product& p, int k, int n) {
    return p.sums ? min(n, k + p.sums * p.pairs) : n;
  };
  constexpr bool two = !kSets;  // tiles in flight
  bool ok = true;

  if (warp >= 4) {
    if constexpr (kParts) registers_up<kManyRegs>();
    // ---- results
    int it = 0;
    Stats st{-INFINITY, 0.f, 0.f};
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
    // (one lane asks: the others would take turns at it with the products' thread)
    auto done = [&](int buf, int phase) {
      bool there = true;
      if (lane == 0) there = mbar_wait(smem_u32(&s_done[buf]), phase & 1);
      return __all_sync(~0u, there) != 0;
    };
    auto release = [&](int buf) {
      fence_before();
      __syncwarp();
      if (lane == 0) {
        const uint32_t bar = smem_u32(&s_free[buf]);
        mbar_arrive_cluster(kCg == 2 ? map_to(bar, 0) : bar);
      }
    };
    auto fill = [](auto& v, float x) {
      for (auto& row : v)
#pragma unroll
        for (int c = 0; c < 32; ++c) row[c] = x;
    };
    Turn& turn = s_turn[kEpi == kBack ? warp - 4 : 0];
    Tile t;
    for (int j = 0; tile(j, t); ++j) {
      const Product& p = *of(t);
      const int n = (t.k1 - t.k0) * p.pairs;
      const RowData row = row_data<kEpi>(g, t, (int)rank, count);
      float acc[kParts ? 4 : 1][32];
      if constexpr (kParts) {
        if (n == 0) fill(acc, 0.f);
        for (int k = 0; k < n; k = part_end(p, k, n)) {
          const int buf = it & 1;
          ok = ok && done(buf, it >> 1);
          if (!ok) {
            fill(acc, __int_as_float(0x7FFFFFFF));
            break;
          }
          fence_after();
          const uint32_t tm = lanes + (uint32_t)buf * 256u + 32u * (uint32_t)(warp / 4 - 1);
          if (k == 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (64 * j < g.bn) tmem_ld32(tm + 64 * j, acc[j]);
#pragma unroll
            for (int j = 0; j < 4; ++j) tmem_wait(acc[j]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (64 * j >= g.bn) break;
              float v[32];
              tmem_ld32(tm + 64 * j, v);
              tmem_wait(v);
#pragma unroll
              for (int c = 0; c < 32; ++c) acc[j][c] += v[c];
            }
          }
          release(buf);
          ++it;
        }
        results<kCg, kEpi, true, false>(p, t, (int)rank, count, 0u, true, !ok, acc, st, turn, s_pair, row);
      } else {
        const int buf = two ? it & 1 : 0;
        if (n > 0) ok = ok && done(buf, two ? it >> 1 : it);
        fence_after();
        results<kCg, kEpi, false, kSets>(p, t, (int)rank, count, lanes + (uint32_t)buf * 256u, n > 0 && ok, !ok,
                                  acc, st, turn, s_pair, row);
        if (n > 0 && ok) release(buf);
        it += n > 0;
      }
    }
    if (kEpi == kStats && g.run) {
      const int r = (warp & 3) * 32 + lane;
      record(g, st, s_pair, warp >= 8, r < count ? (int64_t)blockIdx.x * g.rpad + r : -1);
    }
  } else {
    if constexpr (kParts) registers_down<kFewRegs>();
    // (dW's A lies across the reduction.  Either product's loop is its own code:
    // chosen within the loop, maps and descriptors leave the uniform registers,
    // and the tensor cores wait a fifth of the time.)
    auto each = [&](auto&& run) {
      Tile t;
      for (int j = 0; ok && tile(j, t); ++j) {
        if constexpr (kEpi == kBack) {
          if (t.weight) run(t, w, std::true_type{});
          else run(t, g, std::false_type{});
        } else {
          run(t, g, std::false_type{});
        }
      }
    };
    int st = 0;
    uint32_t ph = 0;
    if (warp == 0) {
      // ---- operands
      const bool one = elect();
      each([&](const Tile& t, const Product& q, auto amn) {
        constexpr bool kAmn = decltype(amn)::value;
        const int m = t.m0 + (int)rank * kRows, n = t.n0 + (int)rank * half;
        // parts of `sums` blocks, each with its six products of planes: the tiles
        // of three planes come from memory once
        const int part = q.sums ? q.sums : t.k1 - t.k0;
        for (int k0 = t.k0; k0 < t.k1 && ok; k0 += part) {
          const int k1 = min(t.k1, k0 + part);
          for (int p = 0; p < q.pairs && ok; ++p) {
            const int2 z = planes_of(q.pairs, p);
            for (int k = k0; k < k1; ++k) {
              if (!(ok = mbar_wait_all(smem_u32(&s_empty[st]), ph ^ 1u))) break;
              uint32_t bar = smem_u32(&s_full[st]);
              const uint32_t sa = smem + st * stage_bytes, sb = sa + a_bytes;
              if (one) {
                if (rank == 0) mbar_expect_tx(bar, (a_bytes + b_bytes) * kCg);
                if (kCg == 2) bar = map_to(bar, 0);
                if (kAmn) {
                  for (int j = 0; j < kRows; j += 64)
                    tma_load<kCg>(sa + j * 128u, &q.a, m + j, k * kBlk, z.x, bar);
                } else {
                  tma_load<kCg>(sa, &q.a, k * kBlk, m, z.x, bar);
                }
                if (kBmn) {
                  const int y = (kAmn ? 0 : g.v0) + k * kBlk;
                  for (int j = 0; j < half; j += 64)
                    tma_load<kCg>(sb + j * 128u, &q.b, n + j, y, z.y, bar);
                } else {
                  tma_load<kCg>(sb, &q.b, k * kBlk, g.v0 + n, z.y, bar);
                }
              }
              __syncwarp();
              if (++st == g.stages) st = 0, ph ^= 1u;
            }
          }
        }
      });
      // nothing of this CTA's is in flight when it ends: every stage asked for
      // has been taken (or, after a wait that ran out, has at least arrived)
      // (a stage never asked for is in the phase that this wait takes as done)
      for (int i = 0; i < g.stages; ++i) {
        if (!mbar_wait_all(ok ? smem_u32(&s_empty[st]) : smem_u32(&s_full[st]), ph ^ 1u)) break;
        if (++st == g.stages) st = 0, ph ^= 1u;
      }
    } else if (warp == 1 && rank == 0) {
      // ---- products
      const bool one = elect();
      const uint32_t full0 = smem_u32(&s_full[0]), empty0 = smem_u32(&s_empty[0]);
      int it = 0;
      each([&](const Tile& t, const Product& p, auto amn) {
        constexpr bool kAmn = decltype(amn)::value;
        constexpr uint32_t kStepA = kAmn ? 128u : 2u, kStepB = kBmn ? 128u : 2u;  // 16 elements, in 16 bytes
        const uint64_t da0 = operand(smem, kAmn), db0 = operand(smem + a_bytes, kBmn);
        const uint32_t idesc = instruction(kRows * kCg, g.bn, g.fmt, kAmn, kBmn);
        const int n = (t.k1 - t.k0) * p.pairs;
        for (int k = 0; k < n && ok; ++it) {
          // a tile, or (kParts) a part of its reduction, into one of two accumulators
          const int buf = two ? it & 1 : 0, end = kParts ? part_end(p, k, n) : n;
          if (!(ok = mbar_wait_all(smem_u32(&s_free[buf]), ((two ? it >> 1 : it) & 1) ^ 1u))) break;
          fence_after();
          uint32_t d = tmem + (uint32_t)buf * 256u;
          int next = kSets ? n / g.kc : 0, set = 0;  // (the first block of the next set)
          bool add = false, here = false;            // (here: the next block has been seen to be there)
          for (; k < end; ++k) {
            if (kSets && k == next && set + 1 < g.kc) {
              ++set;
              next = n * (set + 1) / g.kc;
              d += (uint32_t)g.slot;
              add = false;
            }
            if (!here && !(ok = mbar_wait_all(full0 + 8u * st, ph))) break;
            const uint64_t off = (uint64_t)((uint32_t)st * stage_bytes >> 4), da = da0 + off, db = db0 + off;
            if (one) {
#pragma unroll
              for (int j = 0; j < kBlk / 16; ++j)
                mma<kCg>(d, da + j * kStepA, db + j * kStepB, idesc, add || j != 0);
              commit<kCg>(empty0 + 8u * st);
            }
            __syncwarp();
            add = true;
            if (++st == g.stages) st = 0, ph ^= 1u;
            here = k + 1 < end && __all_sync(~0u, mbar_try(full0 + 8u * st, ph));
          }
          if (one) commit<kCg>(smem_u32(&s_done[buf]));
          __syncwarp();
        }
      });
    }
  }
  if (!ok && g.status) atomicOr(g.status, (unsigned)GRPO_ERR_TIMEOUT);
  __syncwarp();
  fence_before();
  __syncthreads();
  if (kCg == 2) cluster_sync();
  if (warp == 2) tmem_free<kCg>(tmem, 512);
}

// ---------------------------------------------------------------- rows
// Which tokens take part, in their order: idx, and for the gradient each
// row's coefficients,
//   d_v = s dlogp 1[v = a] - 2^u (c0 + c1 u),   u = (x_v - m) s log2 e,
//   c0 = s / Z (dlogp + dH (H - ln Z)),  c1 = s ln 2 / Z dH
// A CTA takes 1,024 tokens and counts those before them itself, so no CTA waits
// for another: latency, 3.5 us for 16,384 tokens (gradient: 5.2) and 9.4 (18) for
// 131,072, where the products that masked tokens would cost take milliseconds.
// The reads grow with the square of the tokens: 0.14 ms (0.28) for 2^20, 1.8
// (3.6) for 2^22, a hundredth of such a batch's products.
static constexpr int kPrepRows = 1024;

struct Header {  // the first 256 bytes of the workspace
  int count;
  unsigned bound;  // of |d| over all rows, as bits
};

struct PrepRows {
  const int64_t* actions;
  const uint8_t* mask;
  int N;
  int64_t V;
  const float* stats;
  const float* entropy;
  const float* dlogp;
  const float* dent;
  float s;
  int* idx;
  float4* coef;  // nullable: the forward pass
  int* target;
  Header* h;
  unsigned* status;
  float *logps, *out_entropy, *out_stats;  // of the tokens that take no part
};

__device__ __forceinline__ bool takes_part(const PrepRows& a, int r) {
  if (a.mask && !a.mask[r]) return false;
  if (!a.coef) return true;
  return (a.dlogp && !(a.dlogp[r] == 0.f)) || (a.dent && !(a.dent[r] == 0.f));
}

__global__ void __launch_bounds__(1024) rows_kernel(const PrepRows a) {
  __shared__ int s_sum[32];
  __shared__ unsigned s_max[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int base = blockIdx.x * kPrepRows, r = base + (int)threadIdx.x;
  launched_early();
  // what this thread's token needs, asked for at once
  const bool mine_in = r < a.N;
  float w = 0.f, h = 0.f, m = 0.f, Z = 1.f, H = 0.f;
  int64_t id = -1;
  bool on = mine_in && (!a.mask || a.mask[r]);
  if (a.coef && mine_in) {
    if (a.dlogp) w = a.dlogp[r], id = a.actions[r];
    if (a.dent) h = a.dent[r], H = a.entropy[r];
    m = a.stats[r], Z = a.stats[(int64_t)a.N + r];
    on = on && (!(w == 0.f) || !(h == 0.f));
  }
  // the tokens before this CTA's (the last one meets them all: it has the bound too)
  int before = 0;
  float wm = 0.f, hm = 0.f;
#pragma unroll 4
  for (int i = threadIdx.x; i < base; i += 1024) {
    const bool in = !a.mask || a.mask[i];
    const float wi = a.dlogp ? a.dlogp[i] : 0.f, hi = a.dent ? a.dent[i] : 0.f;
    const bool part = in && (!a.coef || !(wi == 0.f) || !(hi == 0.f));
    before += part;
    if (part) wm = fmaxf(wm, fabsf(wi)), hm = fmaxf(hm, fabsf(hi));
  }
  before = __reduce_add_sync(~0u, before);
  if (lane == 0) s_sum[warp] = before;
  __syncthreads();
  before = __reduce_add_sync(~0u, s_sum[lane]);
  __syncthreads();
  const unsigned votes = __ballot_sync(~0u, on);
  if (lane == 0) s_sum[warp] = __popc(votes);
  __syncthreads();
  int mine = 0, all = s_sum[lane];
  mine = __reduce_add_sync(~0u, lane < warp ? all : 0);
  all = __reduce_add_sync(~0u, all);
  const int at = before + mine + __popc(votes & ((1u << lane) - 1u));
  if (on) {
    a.idx[at] = r;
    if (a.coef) {
      const float lnZ = logf(Z);
      float c0 = a.s / Z * (w + (a.dent ? h * (H - lnZ) : 0.f));
      int t = -1;
      if (w != 0.f) {
        if (id >= 0 && id < a.V) {
          t = (int)id;
        } else {
          c0 = __int_as_float(0x7FFFFFFF);
          if (a.status) atomicOr(a.status, (unsigned)GRPO_ERR_ACTION_RANGE);
        }
      }
      a.coef[at] = make_float4(m, c0, 0.6931471805599453f * (a.s / Z) * h, a.s * w);
      a.target[at] = t;
      wm = fmaxf(wm, fabsf(w)), hm = fmaxf(hm, fabsf(h));
    }
  } else if (mine_in) {
    if (a.logps) a.logps[r] = 0.f;
    if (a.out_entropy) a.out_entropy[r] = 0.f;
    if (a.out_stats) a.out_stats[r] = 0.f, a.out_stats[(int64_t)a.N + r] = 1.f;
  }
  if (blockIdx.x != gridDim.x - 1) return;
  if (a.coef) {
    // |d| <= s (|dlogp| + |dH| max(1 / e, ln V)); the largest of either give a
    // bound of all (bits order as the values do)
    const float wt = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(wm)));
    const float ht = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(hm)));
    if (lane == 0) s_max[warp] = __float_as_uint(a.s * (wt + ht * (0.37f + logf((float)a.V))));
    __syncthreads();
    const unsigned top = __reduce_max_sync(~0u, s_max[lane]);
    if (threadIdx.x == 0) a.h->bound = top;
  }
  if (threadIdx.x == 0) a.h->count = before + all;
}

// Rows into the layout of the tile loads: [planes][rows][Kp], zeros behind
// row `count` up to a multiple of kPad and behind column K.  A warp takes a row.
// Bound by memory: 10 us for 8.4 MB of hidden states (latency), 26 us for 71 MB
// of fp32 operands into 107 MB of planes (6.9 TB/s), 43 us for 102 MB of rows of
// 1,021 f16 elements, whose words start anywhere.
//
// fp32: x = x0 + x1 + x2, each the rest rounded to bf16 (8 bits and a sign), so
// that 24 bits are kept while the rest is a normal number.
struct PackRows {
  const void* src;
  const int* idx;
  const int* count;  // nullptr: rows
  int rows;
  int64_t T, sb, st;  // source row r: element r / T sb + r % T st
  int64_t K, Kp, plane;
  void* dst;
};

// A row of 16-bit elements that starts anywhere: five aligned words give the
// four of a vector, shifted together where the row starts in the middle of a
// word.  Words that are not wholly inside [begin, end) are not read as such.
__device__ __forceinline__ void pack_shifted(const PackRows& a, const unsigned short* src, int64_t r,
                                             uintptr_t begin, uintptr_t end) {
  const int odd = ((uintptr_t)src & 2) * 8;
  const uintptr_t base = (uintptr_t)src & ~(uintptr_t)3, stop = (uintptr_t)(src + a.K);
#pragma unroll 4
  for (int64_t k = (threadIdx.x & 31) * 8; k < a.Kp; k += 256) {
    const uintptr_t p = base + 2 * k;
    unsigned w[5] = {0u, 0u, 0u, 0u, 0u};
    if (p >= begin && p + 20 <= end) {
#pragma unroll
      for (int i = 0; i < 5; ++i) w[i] = __ldg((const unsigned*)p + i);
    } else {
#pragma unroll
      for (int i = 0; i < 10; ++i) {
        const uintptr_t q = p + 2 * i;
        if (q >= (uintptr_t)src && q < stop) w[i / 2] |= (unsigned)__ldg((const unsigned short*)q) << (i & 1) * 16;
      }
    }
    unsigned v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __funnelshift_r(w[i], w[i + 1], odd);
    const int64_t left = a.K - k;
    if (left < 8) {  // nothing behind the row's end
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (2 * i + 1 >= left) v[i] = 2 * i < left ? v[i] & 0xFFFFu : 0u;
    }
    *reinterpret_cast<uint4*>((unsigned short*)a.dst + r * a.Kp + k) = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

template <typename T>
__device__ __forceinline__ void pack_rows(const PackRows& a, int first, int step) {
  const int count = a.count ? *a.count : a.rows;
  const int end = (count + kPad - 1) / kPad * kPad;
  const int lane = threadIdx.x & 31;
  for (int64_t r = first; r < end; r += step) {  // (the step behind the last row may pass 2^31)
    const bool live = r < count;
    const int64_t from = live ? (a.idx ? a.idx[r] : r) : 0;
    const T* src = (const T*)a.src + from / a.T * a.sb + from % a.T * a.st;
    const bool whole = ((uintptr_t)src & 15) == 0;
    if constexpr (!std::is_same<T, float>::value) {
      if (live && !whole) {
        const int64_t last = a.rows > 0 ? (int64_t)(a.rows - 1) / a.T * a.sb + (a.T - 1) * a.st + a.K : 0;
        pack_shifted(a, (const unsigned short*)src, r, (uintptr_t)a.src,
                     (uintptr_t)((const unsigned short*)a.src + last));
        continue;
      }
    }
    for (int64_t k = lane * 8; k < a.Kp; k += 256) {
      if constexpr (std::is_same<T, float>::value) {
        float f[8];
        if (live && whole && k + 8 <= a.K) {
          const float4 u = __ldg((const float4*)(src + k)), v = __ldg((const float4*)(src + k) + 1);
          f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w;
          f[4] = v.x, f[5] = v.y, f[6] = v.z, f[7] = v.w;
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = live && k + i < a.K ? __ldg(src + k + i) : 0.f;
        }
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[i]));
        __nv_bfloat16* dst = (__nv_bfloat16*)a.dst + r * a.Kp + k;
        if (top < 0x1.FEp127f) {
#pragma unroll
          for (int p = 0; p < 3; ++p) {
            const uint4 h = Storage<__nv_bfloat16>::pack(f);
            *reinterpret_cast<uint4*>(dst + p * a.plane) = h;
            float x[8];
            Storage<__nv_bfloat16>::unpack(h, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] -= x[i];
          }
        } else {
          // values that round beyond bf16 take its largest, and the rest follows
          // in the next plane; infinities stand in the first alone
          for (int p = 0; p < 3; ++p) {
            float h[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              h[i] = __bfloat162float(__float2bfloat16_rn(f[i]));
              if (isinf(h[i]) && !isinf(f[i])) h[i] = copysignf(0x1.FEp127f, f[i]);
              f[i] = isfinite(h[i]) ? f[i] - h[i] : 0.f;
            }
            *reinterpret_cast<uint4*>(dst + p * a.plane) = Storage<__nv_bfloat16>::pack(h);
          }
        }
      } else {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (live && whole && k + 8 <= a.K) {
          v = __ldg((const uint4*)(src + k));
        } else if (live) {  // (the row's end)
          const unsigned short* q = (const unsigned short*)src + k;
          unsigned h[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) h[i] = k + i < a.K ? __ldg(q + i) : 0u;
          v = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
        }
        *reinterpret_cast<uint4*>((T*)a.dst + r * a.Kp + k) = v;
      }
    }
  }
}

// The hidden states' rows by the first CTAs, the weight's by the others.
template <typename T>
__global__ void __launch_bounds__(256) pack_kernel(const PackRows h, const PackRows w, int ctas) {
  launched_early();
  const int warp = threadIdx.x >> 5, cta = blockIdx.x;
  if (cta < ctas) pack_rows<T>(h, cta * 8 + warp, ctas * 8);
  else pack_rows<T>(w, (cta - ctas) * 8 + warp, ((int)gridDim.x - ctas) * 8);
}

// The parts of each row joined: 32 rows a CTA, its warps take tiles in turn.
//   m = max m_i,  Z = sum Z_i 2^((m_i - m) s2),  D likewise; logp, H, (m, Z)
// Latency: 8 us for 2,048 tokens of 128 parts.
struct FoldRows {
  const float4* part;
  const float* xa;
  const int* count;
  int rows, nt, rpad, N;
  const int* idx;
  const int64_t* actions;
  const uint8_t* mask;  // of rows that were not chosen by it
  int64_t V;
  float s, s2;
  float *logps, *entropy, *stats;
  unsigned* status;
};
static constexpr int kFoldWarps = 16, kFoldAhead = 4;

__global__ void __launch_bounds__(32 * kFoldWarps) fold_kernel(const FoldRows a) {
  __shared__ float4 s_part[kFoldWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  launched_early();
  const int count = a.count ? *a.count : a.rows;
  const int r = blockIdx.x * 32 + lane;
  if (blockIdx.x * 32 >= count) return;
  const float4 none = make_float4(-INFINITY, 0.f, 0.f, 0.f);
  float4 x[kFoldAhead + 1];
  x[0] = none;
  if (r < count)
    for (int t = warp; t < a.nt; t += kFoldWarps * kFoldAhead) {
#pragma unroll
      for (int j = 0; j < kFoldAhead; ++j) {
        const int u = t + j * kFoldWarps;
        x[j + 1] = u < a.nt ? a.part[(int64_t)u * a.rpad + r] : none;
      }
      x[0] = join(x, a.s2);
    }
  s_part[warp][lane] = x[0];
  __syncthreads();
  if (warp != 0 || r >= count) return;
  float4 y[kFoldWarps];
#pragma unroll
  for (int w = 0; w < kFoldWarps; ++w) y[w] = s_part[w][lane];
  const float4 z = join(y, a.s2);
  const int src = a.idx ? a.idx[r] : r;
  if (a.mask && !a.mask[src]) {
    if (a.logps) a.logps[src] = 0.f;
    if (a.entropy) a.entropy[src] = 0.f;
    if (a.stats) a.stats[src] = 0.f, a.stats[(int64_t)a.N + src] = 1.f;
    return;
  }
  // a row without a finite maximum (+inf, nothing above -inf) or with a NaN has no distribution
  const float bad = __int_as_float(0x7FFFFFFF);
  const float Z = isfinite(z.x) ? z.y : bad;
  const float lnZ = logf(Z);
  if (a.logps) {
    const int64_t id = a.actions[src];
    const bool in = id >= 0 && id < a.V;
    a.logps[src] = in ? fmaf(a.s, a.xa[r] - z.x, -lnZ) : bad;
    if (!in && a.status) atomicOr(a.status, (unsigned)GRPO_ERR_ACTION_RANGE);
  }
  if (a.entropy) a.entropy[src] = fmaf(-0.6931471805599453f, z.z / Z, lnZ);
  if (a.stats) a.stats[src] = z.x, a.stats[(int64_t)a.N + src] = Z;
}

// The parts of the reduction of dh joined (in a fixed order), rows without a
// gradient set to zero.  Where parts are many, rows are few, and
// eight groups of threads take an eighth each: the gradient of 1 x 1,024 x
// 32,768 in fp32, 304 parts, takes 91 us, 139 with one group, 8 x 2,048 x 32,768
// in bf16, 64 parts, 118 and 133.  With sixteen parts or fewer one group is
// as fast or faster: 300 x 2,048 x 32,768 takes 162 us, 173 with eight.
struct HiddenRows {
  const float* acc;  // nullptr: only the rows without a gradient
  int splits, rpad, N;
  int64_t K, ldacc;
  PrepRows rows;     // which tokens take part
  const int* idx;
  const int* count;
  const unsigned* bound;
  void* out;
  int64_t T, osb, ost;
  int skip_masked;
  int groups;        // of threads, which take parts side by side: 1 or 8
};

template <typename T>
__global__ void __launch_bounds__(256) hidden_kernel(const HiddenRows a) {
  __shared__ float4 s_sum[256];
  launched_early();
  const int per = 256 / a.groups, group = threadIdx.x / per;
  // (sums are padded to 256 columns)
  const int64_t k = ((int64_t)blockIdx.y * per + threadIdx.x % per) * 4;
  // first the tokens, then the packed rows
  const int count = *a.count;
  const int64_t total = (int64_t)a.N + (a.acc ? count : 0);
  for (int64_t j = blockIdx.x; j < total; j += gridDim.x) {
    const bool packed = j >= a.N;
    const int r = (int)(packed ? j - a.N : j);
    if (!packed && (takes_part(a.rows, r) || (a.skip_masked && a.rows.mask && !a.rows.mask[r])))
      continue;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4& x) { v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w; };
    if (packed && k < a.K) {
      const float* p = a.acc + (int64_t)r * a.ldacc + k;
      const int to = a.splits * (group + 1) / a.groups;
#pragma unroll 8
      for (int i = a.splits * group / a.groups; i < to; ++i)
        add(*reinterpret_cast<const float4*>(p + (int64_t)i * a.rpad * a.ldacc));
    }
    if (packed && a.groups > 1) {
      __syncthreads();
      s_sum[threadIdx.x] = v;
      __syncthreads();
      for (int i = 1; i < a.groups && group == 0; ++i) add(s_sum[threadIdx.x + i * per]);
    }
    if (group > 0 || k >= a.K) continue;
    const int64_t dst = packed ? a.idx[r] : r;
    T* out = (T*)a.out + dst / a.T * a.osb + dst % a.T * a.ost + k;
    const float scale = a.bound ? 1.f / range_scale(*a.bound) : 1.f;
    const float f[4] = {v.x * scale, v.y * scale, v.z * scale, v.w * scale};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (k + i < a.K) Storage<T>::store1(out + i, f[i]);
  }
}

// ---------------------------------------------------------------- launches
typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                             const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                             const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return (EncodeFn)p;
  }();
  return fn;
}

// A matrix of 16-bit elements [planes][outer][inner], rows `ld` elements
// apart, in boxes of 64 x `box` elements.
bool encode(CUtensorMap* m, const void* p, bool bf16, int64_t inner, int64_t outer, int64_t planes,
            int64_t ld, int64_t plane, int box) {
  const cuuint64_t dim[3] = {(cuuint64_t)inner, (cuuint64_t)std::max<int64_t>(outer, 1),
                             (cuuint64_t)planes};
  const cuuint64_t str[2] = {(cuuint64_t)ld * 2, (cuuint64_t)(planes > 1 ? plane : ld) * 2};
  const cuuint32_t b[3] = {64, (cuuint32_t)box, 1}, e[3] = {1, 1, 1};
  const EncodeFn fn = encode_fn();
  return fn && fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                  (void*)p, dim, str, b, e, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename... Args>
cudaError_t launch(void (*k)(Args...), dim3 grid, unsigned block, int cluster, int smem,
                   cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(block);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&c, k, args...);
}

int sm_count() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 152;
}

template <int kCg, int kEpi, bool kParts, bool kSets>
cudaError_t launch_product(Product& g, const Product* w, int sms, int tiles, cudaStream_t s) {
  const int half = g.bn / kCg;
  const int stage = g.a_rows * 128 + ((half * 128 + 1023) & ~1023);
  // what the accumulators take has to fit: 512 columns, 256 of each of two tiles
  if (g.bn > 256 || (g.kc > 1 && g.bn > g.slot) || g.kc * g.slot > (g.bufs == 2 ? 256 : 512))
    return cudaErrorInvalidValue;
  // rows of A that are not loaded are read from what lies behind: room for the last stage's
  const int more = (kRows - g.a_rows) * 128 + 1024;
  const int fixed = kEpi == kStats ? (int)(kRows * sizeof(Stats))
                    : kEpi == kBack ? (int)(8 * sizeof(Turn)) : 0;
  const int most = kSmem - fixed;
  g.stages = std::min(kMaxStages, (most - more) / stage);
  const int smem = g.stages * stage + more;
  auto* k = product_kernel<kCg, kEpi, kParts, kSets>;
  // (the limit is the function's, in all threads: never less than any call needs)
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e != cudaSuccess) return e;
  const int grid = std::max(1, std::min(sms / kCg, tiles)) * kCg;
  if constexpr (kEpi == kBack) return launch(k, grid, kThreads, kCg, smem, s, g, *w);
  else return launch(k, grid, kThreads, kCg, smem, s, g, 0);
}

template <int kEpi>
cudaError_t launch_product(Product& g, int cg, int sms, int64_t tiles, cudaStream_t s,
                           const Product* w = nullptr) {
  const int n = (int)std::min<int64_t>(tiles, 1 << 20);
  if (g.sums > 0 || (w && w->sums > 0))
    return cg == 2 ? launch_product<2, kEpi, true, false>(g, w, sms, n, s)
                   : launch_product<1, kEpi, true, false>(g, w, sms, n, s);
  if constexpr (kEpi != kBack) {
    if (g.bufs == 1) return launch_product<1, kEpi, false, true>(g, w, sms, n, s);
  }
  return cg == 2 ? launch_product<2, kEpi, false, false>(g, w, sms, n, s)
                 : launch_product<1, kEpi, false, false>(g, w, sms, n, s);
}

int64_t ceil_to(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool pack_weight(const void* w, grpo_dtype_t dt, int64_t V, int64_t sv) {
  return dt == GRPO_F32 || ((uintptr_t)w & 15) != 0 || (V > 1 && sv % 8 != 0);
}

// What a tile of dW takes at least, in blocks of its products: 8 to 32 give the
// same times but for 2 %, with rows on 16 bytes and without (256 to 2,048 tokens).
static constexpr int kLeast = 16;

// What a call keeps in its workspace.
struct Layout {
  bool direct;  // kStats: every row is taken, as it lies
  int few;      // rows of the form for a handful of tokens; 0: another
  int cg, bn;   // CTAs of a tile, its columns (of the vocabulary)
  int kbn;      // columns of a tile of the width
  int sets;     // logits of one CTA: of accumulators that a reduction is cut into
  int64_t rpad, Kp, planes, dplanes, nt, vc, splits, ldd, ldacc;
  size_t idx, coef, target, xa, part, hidden, weight, d, acc, total;
};

// Blocks of a reduction, 64 elements each, that one accumulator sums up.  A
// logit of 16-bit operands is off by about 2e-8 of its size for each block:
// sharp log-probs (temperature 0.6, deviation 3) by 2.2e-6 at a width of 1,024,
// 4e-6 at 2,048 and 8e-6 at 4,096, where parts of 2,048 make it 4e-6 and cost
// 8 % (4,096 x 4,096 x 128,256: 2,069 and 2,244 us).  Sums of fp32 operands are
// as exact as chains of fp32 additions with 8 (and 5e-5 off in the gradients of
// sharp log-probs without parts).  The gradient of 16-bit operands is rounded
// to 16 bits, 2e-3 of it, and takes one sum; dW in fp32 sums up to 4,096 tokens:
// 8,192 tokens and more are off by 5.5e-6 at most (9.9e-6 and, 20,000, 2.3e-5 in
// one sum; 3.4e-6 in sums of 2,048), and 4,608 x 2,048 x 151,936 takes 7.40 ms
// (7.17 in one sum, 7.56 in sums of 2,048).
static constexpr int kSumsF32 = 8, kSumsWide = 32, kSumsTokens = 64;
// Of the logits' gradient: pieces of 512 MB, but of 2,048 words at least, since
// each piece reads and writes the sums of dh.
static constexpr int64_t kPieceBytes = 512ll << 20, kPieceWords = 2048;

// `exact`: dW in fp32 of 16-bit operands.
Layout layout(const void* weight, grpo_dtype_t dt, int64_t N, int64_t K, int64_t V, int64_t sv,
              bool backward, bool exact) {
  Layout l{};
  const int sms = sm_count();
  l.rpad = ceil_to(std::max<int64_t>(N, 1), kPad);
  l.Kp = ceil_to(K, 64);
  l.planes = dt == GRPO_F32 ? 3 : 1;
  l.dplanes = exact ? 2 : l.planes;
  l.cg = N > kRows ? 2 : 1;
  size_t o = 256;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align256(bytes);
    return at;
  };
  l.idx = take(4 * l.rpad);
  l.few = few_rows(dt, N, K);
  if (l.few) {
    l.direct = !backward;
    l.ldacc = ceil_to(K, 256);
    if (backward) {
      l.coef = take(16 * l.rpad);
      l.target = take(4 * l.rpad);
      l.d = take((size_t)(4 * V * l.few));
      l.splits = few_parts(V, K, sms);
      l.acc = take((size_t)(4 * l.splits * l.few * l.ldacc));
    } else {
      l.xa = take(4 * l.rpad);
      l.part = take((size_t)(16 * sms * l.rpad));
    }
    l.total = o;
    return l;
  }
  // One CTA: a logit's sum in parts, each with its own accumulators, for which
  // tensor memory has room here.  Two of them, and four of 128 columns where a
  // 16-bit width passes 2,048: 64 x 4,096 x 151,936 takes 190 us where two sets
  // of 256 columns take 183, and its entropies are off by 1.4e-6 where 3.1e-6;
  // 1 x 2,048 x 32,768 would take 32 where 30.  The gradient forms its logits in the same
  // order where its results have more than 16 bits.
  const bool wide_sums = l.cg == 1 && (!backward || exact || dt == GRPO_F32);
  l.sets = !wide_sums ? 1 : dt != GRPO_F32 && l.Kp > 64 * kSumsWide ? 4 : 2;
  l.hidden = take((size_t)(2 * l.planes * l.rpad * l.Kp));
  l.weight = take(pack_weight(weight, dt, V, sv) ? (size_t)(2 * l.planes * ceil_to(V, kPad) * l.Kp) : 0);
  if (backward) {
    l.coef = take(16 * l.rpad);
    l.target = take(4 * l.rpad);
    l.kbn = l.cg == 2 || K > 128 ? 256 : K > 64 ? 128 : 64;
    const int64_t whole = ceil_to(V, 256);
    const int64_t fit = std::max<int64_t>(kPieceBytes / (2 * l.dplanes * l.rpad) / 256 * 256, kPieceWords);
    const int64_t pieces = div_up(whole, fit);
    l.vc = ceil_to(div_up(whole, pieces), 256);
    // one CTA: columns so that the SMs' shares of a piece are even
    const int64_t most = l.sets == 4 ? 128 : 256, waves = div_up(l.vc, (int64_t)sms * most);
    l.bn = l.cg == 2 ? 256 : (int)std::min<int64_t>(most, ceil_to(div_up(l.vc, sms * waves), 32));
    l.ldd = ceil_to(div_up(ceil_to(l.vc, 64), l.bn) * l.bn, 64);
    l.d = take((size_t)(2 * l.dplanes * l.rpad * l.ldd));
    // Parts of dh's reduction, at least eight blocks each, so that its tiles last
    // no longer than a third of what a cluster has to do in all (where two of
    // three tokens take no part, half of it).
    const int64_t wide = div_up(K, l.kbn), tile = kRows * l.cg, planes = l.planes == 3 ? 6 : 1;
    const double blocks = (double)(div_up(N, tile) * wide) * (double)(l.vc / 64) +
                          (double)(div_up(l.vc, tile) * wide) * (double)div_up(N, 64);
    const double share = std::max(1.0, blocks * l.cg / sms);
    const int64_t parts = std::max<int64_t>(1, std::min<int64_t>(64, l.vc / 64 * planes / 8));
    l.splits = std::min<int64_t>(parts, (int64_t)(3.0 * (double)(l.vc / 64) / share) + 1);
    l.ldacc = ceil_to(K, 256);
    if (l.splits > 1 || pieces > 1) l.acc = take((size_t)(4 * l.splits * l.rpad * l.ldacc));
  } else {
    l.direct = N <= kRows;
    // one CTA: columns so that the SMs' shares of the vocabulary are even
    const int64_t wide = l.sets == 4 ? 128 : 256, waves = div_up(V, (int64_t)sms * wide);
    l.bn = l.cg == 2 ? 256 : (int)std::min<int64_t>(wide, ceil_to(div_up(V, sms * waves), 16));
    l.nt = div_up(V, l.bn);
    l.xa = take(4 * l.rpad);
    l.part = take((size_t)(16 * (l.direct ? std::min<int64_t>(l.nt, sms) : l.nt) * l.rpad));
  }
  l.total = o;
  return l;
}

// The rows that take part, and the weight where tile loads cannot take it as it lies.
cudaError_t pack(const LinearArgs& a, grpo_dtype_t dt, const Layout& l, const int* idx,
                 const int* count, bool rows, int sms, cudaStream_t s) {
  const PackRows h{a.hidden, idx, count, (int)(a.B * a.T), std::max<int64_t>(a.T, 1), a.sb, a.st,
                   a.K, l.Kp, l.rpad * l.Kp, a.ws + l.hidden};
  const PackRows w{a.weight, nullptr, nullptr, (int)a.V, 1, a.sv, 0, a.K, l.Kp,
                   ceil_to(a.V, kPad) * l.Kp, a.ws + l.weight};
  const int hc = rows ? (int)std::min<int64_t>(l.rpad / 8, sms * 8) : 0;
  const int wc = pack_weight(a.weight, dt, a.V, a.sv) ? (int)std::min<int64_t>(div_up(a.V, 8), sms * 8) : 0;
  if (hc + wc == 0) return cudaSuccess;
  auto* k = dt == GRPO_F32 ? pack_kernel<float> : pack_kernel<__half>;
  return launch(k, hc + wc, 256, 1, 0, s, h, w, hc);
}

// Parts of a reduction of `kb` blocks: none where one accumulator holds it.
int sums_of(grpo_dtype_t dt, int64_t kb) { return dt == GRPO_F32 && kb > kSumsF32 ? kSumsF32 : 0; }
// of 16-bit operands, for fp32 results
int sums_wide(int64_t kb) { return kb > kSumsWide ? kSumsWide : 0; }

FewArgs few(const LinearArgs& a, const Layout& l) {
  FewArgs f{};
  f.hidden = a.hidden;
  f.T = a.T, f.sb = a.sb, f.st = a.st;
  f.N = (int)(a.B * a.T);
  f.rows = l.few;
  f.weight = a.weight;
  f.V = a.V, f.K = a.K, f.sv = a.sv;
  f.s2 = a.s2;
  return f;
}

// of a row of tiles, as its operands lie packed
int64_t row_bytes(const Layout& l) { return 2 * l.planes * kRows * l.cg * l.Kp; }

Product base(const LinearArgs& a, grpo_dtype_t dt, const Layout& l) {
  Product g{};
  g.rows = (int)(a.B * a.T);
  g.K = (int)a.K;
  g.kb = (int)(l.Kp / 64);
  g.splits = 1;
  g.a_rows = kRows;
  g.sums = sums_of(dt, g.kb);
  g.kc = 1;
  g.slot = 256;
  g.bufs = 2;
  g.pairs = dt == GRPO_F32 ? 6 : 1;
  g.fmt = dt == GRPO_F16 ? 0 : 1;
  g.s = a.inv_t;
  g.s2 = a.s2;
  g.rpad = (int)l.rpad;
  g.T = std::max<int64_t>(a.T, 1);
  g.status = a.hdr ? &a.hdr->status : nullptr;
  g.mb = rows_together(row_bytes(l), div_up(a.B * a.T, kRows * l.cg));
  return g;
}

// The order of a logit's sum: forward pass, and gradients of more than 16 bits.
void order(Product& g, grpo_dtype_t dt, const Layout& l) {
  if (dt != GRPO_F32) g.sums = sums_wide(div_up(g.kb, l.sets));
  if (l.cg == 2) return;
  if (!g.sums) g.kc = std::min(l.sets, g.kb * g.pairs);
  if (l.sets == 4) g.slot = 128;
  g.bufs = g.kc == 1 ? 2 : 1;
}

bool encode_weight(CUtensorMap* m, const LinearArgs& a, grpo_dtype_t dt, const Layout& l, int box) {
  if (pack_weight(a.weight, dt, a.V, a.sv))
    return encode(m, a.ws + l.weight, dt != GRPO_F16, l.Kp, a.V, l.planes, l.Kp,
                  ceil_to(a.V, kPad) * l.Kp, box);
  return encode(m, a.weight, dt != GRPO_F16, a.K, a.V, 1, a.V > 1 ? a.sv : ceil_to(a.K, 8), 0, box);
}

}  // namespace

size_t linear_ws(const void* weight, grpo_dtype_t dt, int64_t N, int64_t K, int64_t V, int64_t sv,
                 bool backward) {
  const size_t need = layout(weight, dt, N, K, V, sv, backward, false).total;
  if (!backward || dt == GRPO_F32) return need;
  return std::max(need, layout(weight, dt, N, K, V, sv, true, true).total);
}

cudaError_t launch_linear_logps(const LinearArgs& a, grpo_dtype_t dt, cudaStream_t s) {
  const int64_t N = a.B * a.T;
  const int sms = sm_count();
  const Layout l = layout(a.weight, dt, N, a.K, a.V, a.sv, false, false);
  Header* h = (Header*)a.ws;
  int* idx = l.direct ? nullptr : (int*)(a.ws + l.idx);
  const int* count = l.direct ? nullptr : &h->count;
  unsigned* status = a.hdr ? &a.hdr->status : nullptr;
  cudaError_t e;
  if (!l.direct) {
    PrepRows p{};
    p.mask = a.mask;
    p.N = (int)N;
    p.idx = idx;
    p.h = h;
    p.logps = a.logps;
    p.out_entropy = a.entropy;
    p.out_stats = a.stats;
    if ((e = launch(rows_kernel, div_up(N, kPrepRows), 1024, 1, 0, s, p)) != cudaSuccess) return e;
  }
  auto fold = [&](const float4* part, const float* xa, int parts) {
    const FoldRows f{part, xa, count, (int)N, parts, (int)l.rpad, (int)N, idx, a.actions,
                     l.direct ? a.mask : nullptr, a.V, a.inv_t, a.s2, a.logps, a.entropy, a.stats, status};
    return launch(fold_kernel, div_up(N, 32), 32 * kFoldWarps, 1, 0, s, f);
  };
  if (l.few) {
    FewArgs f = few(a, l);
    f.actions = a.logps ? a.actions : nullptr;
    f.part = (float4*)(a.ws + l.part);
    f.xa = (float*)(a.ws + l.xa);
    f.rpad = (int)l.rpad;
    if ((e = launch_few_stats(f, sms, s)) != cudaSuccess) return e;
    return fold(f.part, f.xa, sms);
  }
  // rows that tile loads can take where they are
  const int64_t apart = a.T == 1 ? a.sb : a.st;
  const bool in_place = l.direct && dt != GRPO_F32 && ((uintptr_t)a.hidden & 15) == 0 &&
                        (a.T == 1 || a.B == 1 || a.sb == a.T * a.st) &&
                        (N == 1 || (apart % 8 == 0 && apart >= 8 && apart <= (int64_t)1 << 36));
  if ((e = pack(a, dt, l, idx, count, !in_place, sms, s)) != cudaSuccess) return e;
  Product g = base(a, dt, l);
  g.count = count;
  g.idx = idx;
  g.actions = a.logps ? a.actions : nullptr;
  g.vp = (int)a.V;
  g.part = (float4*)(a.ws + l.part);
  g.xa = (float*)(a.ws + l.xa);
  g.want_entropy = a.entropy != nullptr;
  g.bn = l.bn;
  g.nt = (int)l.nt;
  order(g, dt, l);
  if (l.direct) {
    g.run = 1;
    g.a_rows = (int)ceil_to(N, 8);
  }
  const bool mapped =
      in_place ? encode(&g.a, a.hidden, dt != GRPO_F16, a.K, N, 1, N == 1 ? ceil_to(a.K, 8) : apart,
                        0, g.a_rows)
               : encode(&g.a, a.ws + l.hidden, dt != GRPO_F16, l.Kp, l.rpad, l.planes, l.Kp,
                        l.rpad * l.Kp, g.a_rows);
  if (!mapped || !encode_weight(&g.b, a, dt, l, g.bn / l.cg)) return cudaErrorUnknown;
  const int64_t tiles = div_up(N, kRows * l.cg) * g.nt;
  if ((e = launch_product<kStats>(g, l.cg, sms, tiles, s)) != cudaSuccess) return e;
  return fold(g.part, g.xa, l.direct ? (int)std::min<int64_t>(sms, tiles) : g.nt);
}

cudaError_t launch_linear_grad(const LinearArgs& a, grpo_dtype_t dt, cudaStream_t s) {
  const int64_t N = a.B * a.T;
  const int sms = sm_count();
  const bool exact = a.dweight && a.wdt == GRPO_F32 && dt != GRPO_F32;
  const Layout l = layout(a.weight, dt, N, a.K, a.V, a.sv, true, exact);
  Header* h = (Header*)a.ws;
  int* idx = (int*)(a.ws + l.idx);
  PrepRows p{};
  p.actions = a.actions;
  p.mask = a.mask;
  p.N = (int)N;
  p.V = a.V;
  p.stats = a.in_stats;
  p.entropy = a.in_entropy;
  p.dlogp = a.dlogp;
  p.dent = a.dent;
  p.s = a.inv_t;
  p.idx = idx;
  p.coef = (float4*)(a.ws + l.coef);
  p.target = (int*)(a.ws + l.target);
  p.h = h;
  p.status = a.hdr ? &a.hdr->status : nullptr;
  cudaError_t e = N > 0 ? launch(rows_kernel, div_up(N, kPrepRows), 1024, 1, 0, s, p)
                        : cudaMemsetAsync(h, 0, sizeof(Header), s);
  if (e != cudaSuccess) return e;
  const bool hidden = a.dhidden && N > 0;
  // the parts of dh joined, zeros where there is no gradient
  auto finish = [&](const float* acc, int parts, int64_t rows, const unsigned* bound) {
    if (!hidden) return cudaSuccess;
    const HiddenRows r{acc, parts, (int)rows, (int)N, a.K,
                       l.ldacc, p, idx, &h->count, bound, a.dhidden, std::max<int64_t>(a.T, 1), a.gsb,
                       a.gst, a.skip_masked, parts > 16 ? 8 : 1};
    auto* k = dt == GRPO_F32    ? hidden_kernel<float>
              : dt == GRPO_BF16 ? hidden_kernel<__nv_bfloat16>
                                : hidden_kernel<__half>;
    return launch(k, dim3((unsigned)std::min<int64_t>(2 * N, sms * 8), (unsigned)div_up(a.K, 1024 / r.groups)), 256, 1, 0,
                  s, r);
  };
  if (l.few) {
    FewArgs f = few(a, l);
    f.idx = idx;
    f.count = &h->count;
    f.coef = p.coef;
    f.target = p.target;
    f.d = (float*)(a.ws + l.d);
    f.acc = hidden ? (float*)(a.ws + l.acc) : nullptr;
    f.ldacc = l.ldacc;
    f.dweight = a.dweight;
    f.gsv = a.gsv;
    f.add = a.add;
    f.asv = a.asv;
    if ((e = launch_few_grad(f, sms, s)) != cudaSuccess) return e;
    if ((e = launch_few_back(f, (int)l.splits, s)) != cudaSuccess) return e;
    return finish(f.acc, (int)l.splits, l.few, nullptr);
  }
  if ((e = pack(a, dt, l, idx, &h->count, true, sms, s)) != cudaSuccess) return e;
  const bool bf16 = dt != GRPO_F16;
  const unsigned* bound = dt == GRPO_F16 ? &h->bound : nullptr;
  const int cg = l.cg;
  const int a_rows = cg == 2 ? kRows : (int)std::max<int64_t>(ceil_to(N, 8), 8);
  const int rows = kRows * cg;
  const int64_t mt = div_up(N, rows);
  for (int64_t v0 = 0; v0 < a.V; v0 += l.vc) {
    const int vp = (int)std::min<int64_t>(l.vc, a.V - v0);
    Product g = base(a, dt, l);
    g.count = &h->count;
    g.idx = idx;
    g.v0 = (int)v0;
    g.vp = vp;
    g.coef = p.coef;
    g.target = p.target;
    g.want_entropy = a.dent != nullptr;
    g.d = (__nv_bfloat16*)(a.ws + l.d);
    g.planes = (int)l.dplanes;
    g.ldd = l.ldd;
    g.bound = bound;
    g.bn = l.bn;
    g.nt = (int)div_up(ceil_to(vp, 64), g.bn);  // (zeros in what dh's last block reads)
    g.a_rows = a_rows;
    if (!encode(&g.a, a.ws + l.hidden, bf16, l.Kp, l.rpad, l.planes, l.Kp, l.rpad * l.Kp, a_rows) ||
        !encode_weight(&g.b, a, dt, l, g.bn / cg))
      return cudaErrorUnknown;
    Product x = g;
    if (exact || dt == GRPO_F32) order(x, dt, l);
    if ((e = launch_product<kGrad>(x, cg, sms, mt * g.nt, s)) != cudaSuccess) return e;
    Product h = g, w = g;
    h.on = a.dhidden && N > 0;
    h.out = a.dhidden;
    h.osb = a.gsb;
    h.ost = a.gst;
    h.odt = dt;
    h.kb = (vp + 63) / 64;
    h.splits = (int)l.splits;
    h.sums = sums_of(dt, div_up(h.kb, h.splits));
    h.acc = l.acc ? (float*)(a.ws + l.acc) : nullptr;
    h.ldacc = l.ldacc;
    h.acc_old = v0 > 0;
    h.acc_new = v0 + vp < a.V || l.splits > 1;
    w.on = a.dweight != nullptr;
    w.out = a.dweight;
    w.ost = a.gsv;
    w.odt = a.wdt;
    w.add = a.add;
    w.asv = a.asv;
    if (exact) w.pairs = 2;
    w.sums = exact ? (div_up(N, 64) > kSumsTokens ? kSumsTokens : 0) : sums_of(dt, div_up(N, 64));
    w.least = kLeast;
    h.bn = w.bn = l.kbn;
    h.nt = w.nt = (int)div_up(a.K, l.kbn);
    h.a_rows = w.a_rows = kRows;
    w.mb = rows_together(row_bytes(l), div_up(vp, rows));
    if (!encode(&h.a, g.d, bf16, l.ldd, l.rpad, l.dplanes, l.ldd, l.rpad * l.ldd, kRows) ||
        !encode_weight(&h.b, a, dt, l, 64) ||
        !encode(&w.a, g.d, bf16, l.ldd, l.rpad, l.dplanes, l.ldd, l.rpad * l.ldd, 64) ||
        !encode(&w.b, a.ws + l.hidden, bf16, l.Kp, l.rpad, l.planes, l.Kp, l.rpad * l.Kp, 64))
      return cudaErrorUnknown;
    const int64_t tiles = h.on * mt * h.nt * h.splits + w.on * div_up(vp, rows) * w.nt;
    if ((e = launch_product<kBack>(h, cg, sms, tiles, s, &w)) != cudaSuccess) return e;
  }
  return finish(l.splits > 1 ? (const float*)(a.ws + l.acc) : nullptr, (int)l.splits, l.rpad, bound);
}

}  // namespace grpo
