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
// (kGrad), and the two products of that gradient (kHidden, kWeight).  The
// gradient of the logits exists for a piece of the vocabulary at a time.
#include <cuda.h>

#include <algorithm>
#include <type_traits>

#include "grpo_linear.cuh"
#include "grpo_tensor.cuh"

namespace grpo {
namespace {

using namespace tc;

enum Epi { kStats, kGrad, kHidden, kWeight };

static constexpr int kThreads = 256;  // warps: loads, products, tensor memory, (idle), 4 of results
static constexpr int kBlk = 64;       // elements of the reduction a stage holds: 128 bytes a row
static constexpr int kRows = 128;     // rows of a CTA's tile (lanes of tensor memory)
static constexpr int kPad = 256;      // packed rows are padded to the rows of a pair's tile
static constexpr int kMaxStages = 8;
static constexpr int kSmemStages = 216 * 1024;

struct Product {
  CUtensorMap a, b;
  const int* count;  // packed rows, on the device; nullptr: rows
  int rows;
  int v0, vp;     // the piece of the vocabulary
  int K;          // width
  int bn, nt;     // columns of a tile, tiles of columns
  int kb;         // blocks of the reduction where it is not over the rows
  int splits;     // parts of the reduction (kHidden)
  int pairs;      // products of planes: 1, or 6 of three planes each
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
  int want_entropy;      // (both): D, c1 wanted
  __nv_bfloat16* d;      // [planes][rpad][ldd]
  int64_t ldd;
  const unsigned* bound; // f16: largest |d|, as bits; nullptr: no scaling
  // kHidden: fp32 sums, or results
  float* acc;            // [splits][rpad][K]
  int acc_old, acc_new;  // sums are there, are left there
  void* out;
  int64_t T, osb, ost;   // rows of the results
  int odt;
  const void* add;       // kWeight
  int64_t asv;
  unsigned* status;
};

struct Tile {
  int m0, n0, k0, k1, split;
};

// Products of planes, the small ones first: x = x0 + x1 + x2 in bf16, and what
// is left out is below 2^-26 of |x| |w|.
__device__ __constant__ signed char kPairs[6][2] = {{0, 2}, {2, 0}, {1, 1}, {0, 1}, {1, 0}, {0, 0}};

// 2^e with the largest |d| times it in [2^13, 2^15): fp16 has no range of its
// own to spare, and 2^-14 / 2^15 of the largest value is still a normal number.
__device__ __forceinline__ float range_scale(unsigned bits) {
  const int e = (int)(bits >> 23) - 127;
  if (bits == 0 || e > 126) return 1.f;
  return __int_as_float((min(14 - e, 126) + 127) << 23);
}

template <typename T>
__device__ __forceinline__ float load1(const T* p) { return Storage<T>::load1(p); }

// 32 results of a row, `n` of them inside, times `scale` plus `add`'s.
template <typename T>
__device__ __forceinline__ void store_row(T* out, const T* add, const float (&v)[32], int n,
                                          float scale) {
  constexpr int kVec = Storage<T>::kVec;
  if (n >= 32 && ((uintptr_t)out & 15) == 0) {
#pragma unroll
    for (int i = 0; i < 32; i += kVec) {
      float f[kVec];
#pragma unroll
      for (int j = 0; j < kVec; ++j) f[j] = v[i + j] * scale;
      if (add) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) f[j] += load1(add + i + j);
      }
      *reinterpret_cast<uint4*>(out + i) = Storage<T>::pack(f);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < n) Storage<T>::store1(out + i, v[i] * scale + (add ? load1(add + i) : 0.f));
  }
}

// ---- results of a tile: thread t has one row, `tm` its accumulators
template <int kEpi>
__device__ __forceinline__ void results(const Product& g, const Tile& t, int rank, int count,
                                        uint32_t tm, bool have, bool failed) {
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3;
  const int r = t.m0 + rank * kRows + quad * 32 + lane;
  const float bad = __int_as_float(0x7FFFFFFF);
  auto load = [&](int c, float (&v)[32]) {
    __syncwarp();
    if (have) {
      tmem_ld32(tm + c, v);
      tmem_wait(v);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = failed ? bad : 0.f;
    }
  };
  if constexpr (kEpi == kStats) {
    const int n = min(g.bn, g.vp - t.n0);
    const bool live = r < count;
    int a = -1;
    if (live && g.actions) {
      const int64_t id = g.actions[g.idx ? g.idx[r] : r] - t.n0;
      a = id >= 0 && id < n ? (int)id : -1;
    }
    float m = -INFINITY, Z = 0.f, D = 0.f, xa = 0.f;
    for (int c = 0; c < n; c += 32) {
      float v[32];
      load(c, v);
      if (c + 32 > n) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = c + i < n ? v[i] : -INFINITY;
      }
      float cm = v[0];
#pragma unroll
      for (int i = 1; i < 32; ++i) cm = fmaxf(cm, v[i]);
      if (cm > m) {
        const float u = fmaxf((m - cm) * g.s2, -1000.f);
        const float k = exp2f(u);
        D = k * (D + Z * u);
        Z *= k;
        m = cm;
      }
      // (a row of -inf so far: 2^-inf = 0 against any finite reference)
      const float ref = m == -INFINITY ? 0.f : m;
      float z = 0.f, d = 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float u = (v[i] - ref) * g.s2;
        const float e = ex2_fast(u);
        z += e;
        d = fmaf(e, fmaxf(u, -1000.f), d);
      }
      Z += z;
      D += d;
      if (__any_sync(~0u, a >= c && a < c + 32)) {
#pragma unroll
        for (int i = 0; i < 32; ++i) xa = a == c + i ? v[i] : xa;
      }
    }
    if (live) {
      g.part[(int64_t)(t.n0 / g.bn) * g.rpad + r] = make_float4(m, Z, D, 0.f);
      if (a >= 0) g.xa[r] = xa;
    }
  } else if constexpr (kEpi == kGrad) {
    const int n = min(g.bn, g.vp - t.n0);
    const bool live = r < count;
    const float4 q = live ? g.coef[r] : make_float4(0.f, 0.f, 0.f, 0.f);
    const int a = live ? g.target[r] - g.v0 - t.n0 : -1;
    const float scale = g.bound ? range_scale(*g.bound) : 1.f;
    const float c0 = -q.y * scale, c1 = -q.z * scale;
    const int planes = g.pairs == 1 ? 1 : 3;
    __nv_bfloat16* row = g.d + (int64_t)r * g.ldd + t.n0;
    for (int c = 0; c < g.bn; c += 32) {
      float v[32];
      load(c, v);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float u = fmaxf((v[i] - q.x) * g.s2, -1000.f);
        v[i] = ex2_fast(u) * fmaf(c1, u, c0);
      }
      if (__any_sync(~0u, a >= c && a < c + 32)) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] += a == c + i ? q.w * scale : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = live && c + i < n ? (failed ? bad : v[i]) : 0.f;
      if (g.fmt == 0) {
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
          float f[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = v[i + j];
          *reinterpret_cast<uint4*>(row + c + i) = Storage<__half>::pack(f);
        }
      } else {
        for (int p = 0; p < planes; ++p) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              f[j] = v[i + j];
              v[i + j] -= __bfloat162float(__float2bfloat16_rn(f[j]));
            }
            *reinterpret_cast<uint4*>(row + (int64_t)p * g.rpad * g.ldd + c + i) =
                Storage<__nv_bfloat16>::pack(f);
          }
        }
      }
    }
  } else {
    const float scale = g.bound ? 1.f / range_scale(*g.bound) : 1.f;
    const int64_t dst = kEpi == kWeight ? (r < g.vp ? g.v0 + r : -1)
                                        : (r < count ? (g.idx ? g.idx[r] : r) : -1);
    const int64_t at = kEpi == kWeight ? dst * g.ost : dst / g.T * g.osb + dst % g.T * g.ost;
    for (int c = 0; c < g.bn && t.n0 + c < g.K; c += 32) {
      const int n = min(32, g.K - t.n0 - c);
      float v[32];
      load(c, v);
      if (dst < 0) continue;
      if constexpr (kEpi == kHidden) {
        if (g.acc) {
          float* acc = g.acc + ((int64_t)t.split * g.rpad + r) * g.K + t.n0 + c;
          if (g.acc_old) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i < n) v[i] += acc[i];
          }
          if (g.acc_new) {
            store_row<float>(acc, nullptr, v, n, 1.f);
            continue;
          }
        }
      }
      const int64_t o = at + t.n0 + c;
      const int64_t ao = kEpi == kWeight ? dst * g.asv + t.n0 + c : 0;
      const bool plus = kEpi == kWeight && g.add;
      if (g.odt == GRPO_F32)
        store_row<float>((float*)g.out + o, plus ? (const float*)g.add + ao : nullptr, v, n, scale);
      else if (g.odt == GRPO_BF16)
        store_row<__nv_bfloat16>((__nv_bfloat16*)g.out + o,
                                 plus ? (const __nv_bfloat16*)g.add + ao : nullptr, v, n, scale);
      else
        store_row<__half>((__half*)g.out + o, plus ? (const __half*)g.add + ao : nullptr, v, n,
                          scale);
    }
  }
}

// The products.  A CTA (kCg 1: tiles of 128 rows) or a pair of CTAs (kCg 2:
// 256 rows, each CTA holds half of either operand's tile) takes tiles in turn;
// one thread asks for the operands' blocks, one issues the products into one
// of two sets of accumulators, four warps turn the other into results.
template <int kCg, int kEpi>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const __grid_constant__ Product g) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t s_full[kMaxStages], s_empty[kMaxStages], s_done[2], s_free[2];
  __shared__ uint32_t s_tmem;
  constexpr bool kAmn = kEpi == kWeight, kBmn = kEpi == kWeight || kEpi == kHidden;
  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = kCg == 2 ? cluster_rank() : 0u;
  const int half = g.bn / kCg;  // columns of B in this CTA
  const uint32_t a_bytes = kRows * 128u, b_bytes = (uint32_t)half * 128u;
  const uint32_t stage_bytes = a_bytes + ((b_bytes + 1023u) & ~1023u);

  if (threadIdx.x == 0) {
    tma_prefetch(&g.a);
    tma_prefetch(&g.b);
    for (int i = 0; i < g.stages; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&s_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_done[i]), 1);
      mbar_init(smem_u32(&s_free[i]), 4 * kCg);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) tmem_alloc<kCg>(smem_u32(&s_tmem), 512);
  fence_before();
  __syncthreads();
  if (kCg == 2) cluster_sync();
  fence_after();
  const uint32_t tmem = s_tmem;

  const int count = g.count ? *g.count : g.rows;
  const int rows = kEpi == kWeight ? g.vp : count;
  const int mt = (rows + kRows * kCg - 1) / (kRows * kCg);
  const int kb = kEpi == kWeight ? (count + kBlk - 1) / kBlk : g.kb;
  const int per = mt * g.nt;
  const int total = per * (kEpi == kHidden ? g.splits : 1);
  // tiles: parts of the reduction, then blocks of mb rows of tiles, in which
  // the rows' tiles come first
  auto tile = [&](int t) {
    Tile x;
    x.split = kEpi == kHidden ? t / per : 0;
    const int u = t - x.split * per;
    const int blk = u / (g.mb * g.nt), left = u - blk * g.mb * g.nt;
    const int w = min(g.mb, mt - blk * g.mb);
    x.m0 = (blk * g.mb + left % w) * kRows * kCg;
    x.n0 = left / w * g.bn;
    x.k0 = 0;
    x.k1 = kb;
    if (kEpi == kHidden) {
      x.k0 = (int)((int64_t)kb * x.split / g.splits);
      x.k1 = (int)((int64_t)kb * (x.split + 1) / g.splits);
    }
    return x;
  };
  const int first = blockIdx.x / kCg, step = gridDim.x / kCg;
  bool ok = true;

  if (warp == 0 && lane == 0) {
    // ---- operands
    int st = 0;
    uint32_t ph = 0;
    for (int i = first; i < total && ok; i += step) {
      const Tile t = tile(i);
      for (int p = 0; p < g.pairs && ok; ++p) {
        const int za = g.pairs == 1 ? 0 : kPairs[p][0], zb = g.pairs == 1 ? 0 : kPairs[p][1];
        for (int k = t.k0; k < t.k1; ++k) {
          if (!(ok = mbar_wait(smem_u32(&s_empty[st]), ph ^ 1u))) break;
          uint32_t bar = smem_u32(&s_full[st]);
          if (rank == 0) mbar_expect_tx(bar, (a_bytes + b_bytes) * kCg);
          if (kCg == 2) bar = map_to(bar, 0);
          const uint32_t sa = smem + st * stage_bytes, sb = sa + a_bytes;
          const int m = t.m0 + (int)rank * kRows, n = t.n0 + (int)rank * half;
          if (kAmn) {
            for (int j = 0; j < kRows; j += 64)
              tma_load<kCg>(sa + j * 128u, &g.a, m + j, k * kBlk, za, bar);
          } else {
            tma_load<kCg>(sa, &g.a, k * kBlk, m, za, bar);
          }
          if (kBmn) {
            const int y = (kEpi == kHidden ? g.v0 : 0) + k * kBlk;
            for (int j = 0; j < half; j += 64)
              tma_load<kCg>(sb + j * 128u, &g.b, n + j, y, zb, bar);
          } else {
            tma_load<kCg>(sb, &g.b, k * kBlk, g.v0 + n, zb, bar);
          }
          if (++st == g.stages) st = 0, ph ^= 1u;
        }
      }
    }
    // nothing of this CTA's is in flight when it ends: every stage asked for
    // has been taken (or, after a wait that ran out, has at least arrived)
    // (a stage never asked for is in the phase that this wait takes as done)
    for (int i = 0; i < g.stages; ++i) {
      if (!mbar_wait(ok ? smem_u32(&s_empty[st]) : smem_u32(&s_full[st]), ph ^ 1u)) break;
      if (++st == g.stages) st = 0, ph ^= 1u;
    }
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // ---- products
    const uint32_t idesc = instruction(kRows * kCg, g.bn, g.fmt, kAmn, kBmn);
    constexpr uint32_t kStepA = kAmn ? 128u : 2u, kStepB = kBmn ? 128u : 2u;  // 16 elements, in 16 bytes
    int st = 0;
    uint32_t ph = 0;
    int it = 0;
    for (int i = first; i < total && ok; i += step) {
      const Tile t = tile(i);
      const int n = (t.k1 - t.k0) * g.pairs;
      if (n == 0) continue;
      const int buf = it & 1;
      if (!(ok = mbar_wait(smem_u32(&s_free[buf]), ((it >> 1) & 1) ^ 1u))) break;
      fence_after();
      const uint32_t d = tmem + (uint32_t)buf * 256u;
      for (int k = 0; k < n; ++k) {
        if (!(ok = mbar_wait(smem_u32(&s_full[st]), ph))) break;
        fence_after();
        const uint32_t sa = smem + st * stage_bytes;
        const uint64_t da = operand(sa, kAmn), db = operand(sa + a_bytes, kBmn);
#pragma unroll
        for (int j = 0; j < kBlk / 16; ++j)
          mma<kCg>(d, da + j * kStepA, db + j * kStepB, idesc, (k | j) != 0);
        commit<kCg>(smem_u32(&s_empty[st]));
        if (++st == g.stages) st = 0, ph ^= 1u;
      }
      commit<kCg>(smem_u32(&s_done[buf]));
      ++it;
    }
  } else if (warp >= 4) {
    // ---- results
    int it = 0;
    for (int i = first; i < total; i += step) {
      const Tile t = tile(i);
      const int buf = it & 1;
      const bool some = (t.k1 - t.k0) * g.pairs > 0;
      if (some && ok) ok = mbar_wait(smem_u32(&s_done[buf]), (it >> 1) & 1);
      ok = __all_sync(~0u, ok);
      fence_after();
      results<kEpi>(g, t, (int)rank, count,
                    tmem + (uint32_t)buf * 256u + ((uint32_t)(warp & 3) << 21), some && ok, !ok);
      fence_before();
      __syncwarp();
      if (lane == 0 && some && ok) {
        const uint32_t bar = smem_u32(&s_free[buf]);
        mbar_arrive_cluster(kCg == 2 ? map_to(bar, 0) : bar);
      }
      it += some;
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
// row's coefficients.  A CTA takes 1,024 tokens and counts those before them
// itself, so no CTA waits for another.
static constexpr int kPrepRows = 1024;

struct Header {  // the first 256 bytes of the workspace, zeroed by the call
  int count;
  unsigned bound;  // largest |d| of any row, as bits
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
  int rpad;
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
  __shared__ int s_sum[33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int base = blockIdx.x * kPrepRows, r = base + (int)threadIdx.x;
  int before = 0;
  for (int i = threadIdx.x; i < base; i += 1024) before += takes_part(a, i);
  before = __reduce_add_sync(~0u, before);
  if (lane == 0) s_sum[warp] = before;
  __syncthreads();
  before = __reduce_add_sync(~0u, s_sum[lane]);
  __syncthreads();
  const bool on = r < a.N && takes_part(a, r);
  const unsigned votes = __ballot_sync(~0u, on);
  if (lane == 0) s_sum[warp] = __popc(votes);
  __syncthreads();
  int mine = 0, all = s_sum[lane];
  mine = __reduce_add_sync(~0u, lane < warp ? all : 0);
  all = __reduce_add_sync(~0u, all);
  const int at = before + mine + __popc(votes & ((1u << lane) - 1u));
  float big = 0.f;
  if (on) {
    a.idx[at] = r;
    if (a.coef) {
      const float m = a.stats[r], Z = a.stats[a.N + r];
      const float w = a.dlogp ? a.dlogp[r] : 0.f, h = a.dent ? a.dent[r] : 0.f;
      const float lnZ = logf(Z);
      float c0 = a.s / Z * (w + (a.dent ? h * (a.entropy[r] - lnZ) : 0.f));
      int t = -1;
      if (w != 0.f) {
        const int64_t id = a.actions[r];
        if (id >= 0 && id < a.V) {
          t = (int)id;
        } else {
          c0 = __int_as_float(0x7FFFFFFF);
          if (a.status) atomicOr(a.status, (unsigned)GRPO_ERR_ACTION_RANGE);
        }
      }
      a.coef[at] = make_float4(m, c0, 0.6931471805599453f * (a.s / Z) * h, a.s * w);
      a.target[at] = t;
      // |p (log p + H)| <= max(1 / e, ln V)
      big = a.s * (fabsf(w) + fabsf(h) * (0.37f + logf((float)a.V)));
    }
  } else if (r < a.N) {
    if (a.logps) a.logps[r] = 0.f;
    if (a.out_entropy) a.out_entropy[r] = 0.f;
    if (a.out_stats) a.out_stats[r] = 0.f, a.out_stats[a.N + r] = 1.f;
  }
  if (a.coef) {
    // (bits order as the values do; a NaN leaves the scale at 1)
    const unsigned top = __reduce_max_sync(~0u, __float_as_uint(big) & 0x7FFFFFFFu);
    if (lane == 0 && top) atomicMax(&a.h->bound, top);
  }
  if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) a.h->count = before + all;
}

// Rows into the layout of the tile loads: [planes][rows][Kp], zeros behind
// row `count` up to a multiple of kPad and behind column K.  A warp takes a row.
struct PackRows {
  const void* src;
  const int* idx;
  const int* count;  // nullptr: rows
  int rows;
  int64_t T, sb, st;  // source row r: element r / T sb + r % T st
  int64_t K, Kp, plane;
  void* dst;
};

template <typename T>
__global__ void __launch_bounds__(256) pack_kernel(const PackRows a) {
  const int count = a.count ? *a.count : a.rows;
  const int end = (count + kPad - 1) / kPad * kPad;
  const int lane = threadIdx.x & 31;
  for (int r = blockIdx.x * 8 + (threadIdx.x >> 5); r < end; r += gridDim.x * 8) {
    const bool live = r < count;
    const int64_t from = live ? (a.idx ? a.idx[r] : r) : 0;
    const T* src = (const T*)a.src + from / a.T * a.sb + from % a.T * a.st;
    const bool whole = ((uintptr_t)src & 15) == 0;
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
#pragma unroll
        for (int p = 0; p < 3; ++p) {
          __nv_bfloat16* dst = (__nv_bfloat16*)a.dst + p * a.plane + r * a.Kp + k;
          float h[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            // (values that round beyond bf16 take its largest; the rest follows in the next plane)
            h[i] = __bfloat162float(__float2bfloat16_rn(f[i]));
            if (isinf(h[i]) && !isinf(f[i])) h[i] = copysignf(0x1.FEp127f, f[i]);
            f[i] = isfinite(h[i]) ? f[i] - h[i] : 0.f;
          }
          *reinterpret_cast<uint4*>(dst) = Storage<__nv_bfloat16>::pack(h);
        }
      } else {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (live && whole && k + 8 <= a.K) {
          v = __ldg((const uint4*)(src + k));
        } else if (live) {
          const unsigned short* q = (const unsigned short*)src + k;
          unsigned h[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) h[i] = k + i < a.K ? __ldg(q + i) : 0u;
          v = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
        }
        *reinterpret_cast<uint4*>((T*)a.dst + (int64_t)r * a.Kp + k) = v;
      }
    }
  }
}

// The parts of each row joined: 32 rows a CTA, its warps take tiles in turn.
struct FoldRows {
  const float4* part;
  const float* xa;
  const int* count;
  int rows, nt, rpad, N;
  const int* idx;
  const int64_t* actions;
  int64_t V;
  float s, s2;
  float *logps, *entropy, *stats;
  unsigned* status;
};

__device__ __forceinline__ void join(float4& x, const float4& y, float s2) {
  const float m = fmaxf(x.x, y.x);
  if (m == -INFINITY) {  // nothing above -inf in either
    x.y += y.y;
    return;
  }
  const float ux = fmaxf((x.x - m) * s2, -1000.f), uy = fmaxf((y.x - m) * s2, -1000.f);
  const float kx = exp2f(ux), ky = exp2f(uy);
  x.z = kx * fmaf(x.y, ux, x.z) + ky * fmaf(y.y, uy, y.z);
  x.y = x.y * kx + y.y * ky;
  x.x = m;
}

__global__ void __launch_bounds__(256) fold_kernel(const FoldRows a) {
  __shared__ float4 s_part[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int count = a.count ? *a.count : a.rows;
  const int r = blockIdx.x * 32 + lane;
  if (blockIdx.x * 32 >= count) return;
  float4 x = make_float4(-INFINITY, 0.f, 0.f, 0.f);
  if (r < count)
    for (int t = warp; t < a.nt; t += 8) join(x, a.part[(int64_t)t * a.rpad + r], a.s2);
  s_part[warp][lane] = x;
  __syncthreads();
  if (warp != 0 || r >= count) return;
#pragma unroll
  for (int w = 1; w < 8; ++w) join(x, s_part[w][lane], a.s2);
  const int src = a.idx ? a.idx[r] : r;
  // a row without a finite maximum (+inf, nothing above -inf) or with a NaN has no distribution
  const float bad = __int_as_float(0x7FFFFFFF);
  const float Z = isfinite(x.x) ? x.y : bad;
  const float lnZ = logf(Z);
  if (a.logps) {
    const int64_t id = a.actions[src];
    const bool in = id >= 0 && id < a.V;
    a.logps[src] = in ? fmaf(a.s, a.xa[r] - x.x, -lnZ) : bad;
    if (!in && a.status) atomicOr(a.status, (unsigned)GRPO_ERR_ACTION_RANGE);
  }
  if (a.entropy) a.entropy[src] = fmaf(-0.6931471805599453f, x.z / Z, lnZ);
  if (a.stats) a.stats[src] = x.x, a.stats[a.N + src] = Z;
}

// The parts of the reduction of dh joined (in their order), rows without a
// gradient set to zero.
struct HiddenRows {
  const float* acc;  // nullptr: only the rows without a gradient
  int splits, rpad, N;
  int64_t K;
  PrepRows rows;     // which tokens take part
  const int* idx;
  const int* count;
  const unsigned* bound;
  void* out;
  int64_t T, osb, ost;
  int skip_masked;
};

template <typename T>
__global__ void __launch_bounds__(256) hidden_kernel(const HiddenRows a) {
  // the first N blocks' worth of rows: tokens; then the packed rows
  const int count = *a.count;
  const int total = a.N + (a.acc ? count : 0);
  for (int j = blockIdx.x; j < total; j += gridDim.x) {
    const bool packed = j >= a.N;
    const int r = packed ? j - a.N : j;
    if (!packed && (takes_part(a.rows, r) || (a.skip_masked && a.rows.mask && !a.rows.mask[r])))
      continue;
    const int64_t dst = packed ? a.idx[r] : r;
    T* out = (T*)a.out + dst / a.T * a.osb + dst % a.T * a.ost;
    const float scale = a.bound ? 1.f / range_scale(*a.bound) : 1.f;
    for (int64_t k = threadIdx.x; k < a.K; k += 256) {
      float v = 0.f;
      if (packed)
        for (int i = 0; i < a.splits; ++i) v += a.acc[((int64_t)i * a.rpad + r) * a.K + k];
      Storage<T>::store1(out + k, v * scale);
    }
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

template <int kCg, int kEpi>
cudaError_t launch_product(Product& g, int sms, int tiles, cudaStream_t s) {
  const int half = g.bn / kCg;
  const int stage = kRows * 128 + ((half * 128 + 1023) & ~1023);
  g.stages = std::min(kMaxStages, kSmemStages / stage);
  const int smem = g.stages * stage + 1024;
  auto* k = product_kernel<kCg, kEpi>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)(std::max(1, std::min(sms / kCg, tiles)) * kCg));
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kCg;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, k, g);
}

template <int kEpi>
cudaError_t launch_product(Product& g, int cg, int sms, int tiles, cudaStream_t s) {
  return cg == 2 ? launch_product<2, kEpi>(g, sms, tiles, s)
                 : launch_product<1, kEpi>(g, sms, tiles, s);
}

int sm_count() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 152;
}

int64_t ceil_to(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

bool pack_weight(const void* w, grpo_dtype_t dt, int64_t V, int64_t sv) {
  return dt == GRPO_F32 || ((uintptr_t)w & 15) != 0 || (V > 1 && sv % 8 != 0);
}

// What a call keeps in its workspace.
struct Layout {
  int64_t rpad, Kp, planes, nt, vc, splits, ldd;
  size_t idx, coef, target, xa, part, hidden, weight, d, acc, total;
};

static constexpr int kSmallTile = 64;                // columns of a tile where tiles are few
static constexpr int64_t kPieceBytes = 512ll << 20;  // of the logits' gradient

Layout layout(const void* weight, grpo_dtype_t dt, int64_t N, int64_t K, int64_t V, int64_t sv,
              bool backward) {
  Layout l{};
  l.rpad = ceil_to(std::max<int64_t>(N, 1), kPad);
  l.Kp = ceil_to(K, 64);
  l.planes = dt == GRPO_F32 ? 3 : 1;
  size_t o = 256;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align256(bytes);
    return at;
  };
  l.idx = take(4 * l.rpad);
  l.hidden = take((size_t)(2 * l.planes * l.rpad * l.Kp));
  l.weight = take(pack_weight(weight, dt, V, sv) ? (size_t)(2 * l.planes * ceil_to(V, kPad) * l.Kp) : 0);
  if (backward) {
    l.coef = take(16 * l.rpad);
    l.target = take(4 * l.rpad);
    const int64_t whole = ceil_to(V, 256);
    const int64_t fit = std::max<int64_t>(kPieceBytes / (2 * l.planes * l.rpad) / 256 * 256, 2048);
    const int64_t pieces = (whole + fit - 1) / fit;
    l.vc = ceil_to((whole + pieces - 1) / pieces, 256);
    l.ldd = l.vc;
    l.d = take((size_t)(2 * l.planes * l.rpad * l.ldd));
    const int64_t tiles = l.rpad / 256 * ((K + 255) / 256);
    l.splits = std::max<int64_t>(1, std::min<int64_t>(76 / tiles, l.vc / 64 / 16));
    if (l.splits > 1 || pieces > 1) l.acc = take((size_t)(4 * l.splits * l.rpad * K));
  } else {
    const int bn = N > kRows ? 256 : kSmallTile;
    l.nt = (V + bn - 1) / bn;
    l.xa = take(4 * l.rpad);
    l.part = take((size_t)(16 * l.nt * l.rpad));
  }
  l.total = o;
  return l;
}

// Rows of `a` (already counted) and the weight where tile loads can take them.
cudaError_t pack(const LinearArgs& a, grpo_dtype_t dt, const Layout& l, const int* idx,
                 const int* count, int sms, cudaStream_t s) {
  PackRows p{a.hidden, idx, count, (int)(a.B * a.T), std::max<int64_t>(a.T, 1), a.sb, a.st, a.K, l.Kp, l.rpad * l.Kp,
             a.ws + l.hidden};
  const int grid = (int)std::min<int64_t>(l.rpad / 8, sms * 8);
  if (dt == GRPO_F32) pack_kernel<float><<<grid, 256, 0, s>>>(p);
  else pack_kernel<__half><<<grid, 256, 0, s>>>(p);
  if (pack_weight(a.weight, dt, a.V, a.sv)) {
    PackRows w{a.weight, nullptr, nullptr, (int)a.V, 1, a.sv, 0, a.K, l.Kp,
               ceil_to(a.V, kPad) * l.Kp, a.ws + l.weight};
    if (dt == GRPO_F32) pack_kernel<float><<<sms * 8, 256, 0, s>>>(w);
    else pack_kernel<__half><<<sms * 8, 256, 0, s>>>(w);
  }
  return cudaGetLastError();
}

Product base(const LinearArgs& a, grpo_dtype_t dt, const Layout& l) {
  Product g{};
  g.rows = (int)(a.B * a.T);
  g.K = (int)a.K;
  g.kb = (int)(l.Kp / 64);
  g.splits = 1;
  g.pairs = dt == GRPO_F32 ? 6 : 1;
  g.fmt = dt == GRPO_F16 ? 0 : 1;
  g.s = a.inv_t;
  g.s2 = a.s2;
  g.rpad = (int)l.rpad;
  g.T = std::max<int64_t>(a.T, 1);
  g.status = a.hdr ? &a.hdr->status : nullptr;
  // 32 MB of the rows at a time, so that they stay in L2 while the vocabulary passes
  g.mb = (int)std::max<int64_t>(1, (32ll << 20) / (2 * l.planes * 256 * l.Kp));
  return g;
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
  return layout(weight, dt, N, K, V, sv, backward).total;
}

cudaError_t launch_linear_logps(const LinearArgs& a, grpo_dtype_t dt, cudaStream_t s) {
  const int64_t N = a.B * a.T;
  const int sms = sm_count();
  const Layout l = layout(a.weight, dt, N, a.K, a.V, a.sv, false);
  Header* h = (Header*)a.ws;
  int* idx = (int*)(a.ws + l.idx);
  unsigned* status = a.hdr ? &a.hdr->status : nullptr;
  cudaError_t e = cudaMemsetAsync(a.ws, 0, 256, s);
  if (e != cudaSuccess) return e;
  PrepRows p{};
  p.mask = a.mask;
  p.N = (int)N;
  p.idx = idx;
  p.rpad = (int)l.rpad;
  p.h = h;
  p.logps = a.logps;
  p.out_entropy = a.entropy;
  p.out_stats = a.stats;
  rows_kernel<<<(unsigned)((N + kPrepRows - 1) / kPrepRows), 1024, 0, s>>>(p);
  if ((e = pack(a, dt, l, idx, &h->count, sms, s)) != cudaSuccess) return e;
  Product g = base(a, dt, l);
  g.count = &h->count;
  g.idx = idx;
  g.actions = a.logps ? a.actions : nullptr;
  g.vp = (int)a.V;
  g.part = (float4*)(a.ws + l.part);
  g.xa = (float*)(a.ws + l.xa);
  const int cg = N > kRows ? 2 : 1;
  g.bn = cg == 2 ? 256 : kSmallTile;
  g.nt = (int)l.nt;
  if (!encode(&g.a, a.ws + l.hidden, dt != GRPO_F16, l.Kp, l.rpad, l.planes, l.Kp, l.rpad * l.Kp, kRows) ||
      !encode_weight(&g.b, a, dt, l, g.bn / cg))
    return cudaErrorUnknown;
  const int64_t tiles = l.rpad / (kRows * cg) * g.nt;
  if ((e = launch_product<kStats>(g, cg, sms, (int)std::min<int64_t>(tiles, 1 << 20), s)) != cudaSuccess) return e;
  FoldRows f{g.part, g.xa, g.count, g.rows, g.nt, g.rpad, (int)N, idx, a.actions, a.V, a.inv_t,
             a.s2, a.logps, a.entropy, a.stats, status};
  fold_kernel<<<(unsigned)((N + 31) / 32), 256, 0, s>>>(f);
  return cudaGetLastError();
}

cudaError_t launch_linear_grad(const LinearArgs& a, grpo_dtype_t dt, cudaStream_t s) {
  const int64_t N = a.B * a.T;
  const int sms = sm_count();
  const Layout l = layout(a.weight, dt, N, a.K, a.V, a.sv, true);
  Header* h = (Header*)a.ws;
  int* idx = (int*)(a.ws + l.idx);
  unsigned* status = a.hdr ? &a.hdr->status : nullptr;
  cudaError_t e = cudaMemsetAsync(a.ws, 0, 256, s);
  if (e != cudaSuccess) return e;
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
  p.rpad = (int)l.rpad;
  p.h = h;
  p.status = status;
  if (N > 0) rows_kernel<<<(unsigned)((N + kPrepRows - 1) / kPrepRows), 1024, 0, s>>>(p);
  if ((e = pack(a, dt, l, idx, &h->count, sms, s)) != cudaSuccess) return e;
  const bool bf16 = dt != GRPO_F16;
  const unsigned* bound = dt == GRPO_F16 ? &h->bound : nullptr;
  const int cg = N > kRows ? 2 : 1;
  const int mt = (int)(l.rpad / (kRows * cg));
  auto count = [&](int64_t n) { return (int)std::min<int64_t>(n, 1 << 20); };
  for (int64_t v0 = 0; v0 < a.V; v0 += l.vc) {
    const int vp = (int)std::min<int64_t>(l.vc, a.V - v0);
    Product g = base(a, dt, l);
    g.count = &h->count;
    g.idx = idx;
    g.v0 = (int)v0;
    g.vp = vp;
    g.coef = p.coef;
    g.target = p.target;
    g.d = (__nv_bfloat16*)(a.ws + l.d);
    g.ldd = l.ldd;
    g.bound = bound;
    g.bn = cg == 2 ? 256 : kSmallTile;
    g.nt = (vp + g.bn - 1) / g.bn;
    if (!encode(&g.a, a.ws + l.hidden, bf16, l.Kp, l.rpad, l.planes, l.Kp, l.rpad * l.Kp, kRows) ||
        !encode_weight(&g.b, a, dt, l, g.bn / cg))
      return cudaErrorUnknown;
    if ((e = launch_product<kGrad>(g, cg, sms, count((int64_t)mt * g.nt), s)) != cudaSuccess) return e;
    if (a.dweight) {
      Product w = g;
      w.out = a.dweight;
      w.ost = a.gsv;
      w.odt = a.wdt;
      w.add = a.add;
      w.asv = a.asv;
      w.bn = cg == 2 ? 256 : kSmallTile;
      w.nt = (int)((a.K + w.bn - 1) / w.bn);
      if (!encode(&w.a, g.d, bf16, l.ldd, l.rpad, l.planes, l.ldd, l.rpad * l.ldd, 64) ||
          !encode(&w.b, a.ws + l.hidden, bf16, l.Kp, l.rpad, l.planes, l.Kp, l.rpad * l.Kp, 64))
        return cudaErrorUnknown;
      const int64_t tiles = (vp + kRows * cg - 1) / (kRows * cg) * (int64_t)w.nt;
      if ((e = launch_product<kWeight>(w, cg, sms, count(tiles), s)) != cudaSuccess) return e;
    }
    if (a.dhidden && N > 0) {
      Product w = g;
      w.out = a.dhidden;
      w.osb = a.gsb;
      w.ost = a.gst;
      w.odt = dt;
      w.bn = cg == 2 ? 256 : kSmallTile;
      w.nt = (int)((a.K + w.bn - 1) / w.bn);
      w.kb = (vp + 63) / 64;
      w.splits = (int)l.splits;
      w.acc = l.acc ? (float*)(a.ws + l.acc) : nullptr;
      w.acc_old = v0 > 0;
      w.acc_new = v0 + vp < a.V || l.splits > 1;
      if (!encode(&w.a, g.d, bf16, l.ldd, l.rpad, l.planes, l.ldd, l.rpad * l.ldd, kRows) ||
          !encode_weight(&w.b, a, dt, l, 64))
        return cudaErrorUnknown;
      if ((e = launch_product<kHidden>(w, cg, sms, count((int64_t)mt * w.nt * w.splits), s)) != cudaSuccess)
        return e;
    }
  }
  if (a.dhidden && N > 0) {
    HiddenRows r{l.splits > 1 ? (const float*)(a.ws + l.acc) : nullptr, (int)l.splits, (int)l.rpad,
                 (int)N, a.K, p, idx, &h->count, bound, a.dhidden, a.T, a.gsb, a.gst, a.skip_masked};
    const int grid = (int)std::min<int64_t>(2 * N, sms * 8);
    if (dt == GRPO_F32) hidden_kernel<float><<<grid, 256, 0, s>>>(r);
    else if (dt == GRPO_BF16) hidden_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(r);
    else hidden_kernel<__half><<<grid, 256, 0, s>>>(r);
  }
  return cudaGetLastError();
}

}  // namespace grpo
