// grpo_linear_few.cu -- the head's log-probs and their gradient for fp32 and at
// most sixteen tokens.
//
//   x_v = sum_k h_k W_vk          a warp has four words, a lane every 32nd vector
//   dW_v = sum_t d_tv h_t,  dh_t = sum_v d_tv W_v   a thread has a vector of columns
//
// The weight's bytes are what such a call takes time for.  The tensor cores'
// form would first split it into bf16 planes: 1.5 times the bytes written, then
// read.  Here each product reads the weight once, as it is, and multiplies on
// the ordinary cores, in fp32, in a fixed order.  Time of a call with a weight
// of 151936 x 4096 (2.49 GB; 360 us at the copy's rate), this form : planes --
// 1 token 419 us, 4 447, 8 541, 16 1,076 : 1,710 at any; 128256 x 4096 and its
// gradient (2.1 GB read twice, written once), 1 token 1,015 us, 8 1,526,
// 16 2,304 : 3,300; 32768 x 1024 and its gradient, 1 token 95 us, 8 149,
// 16 208 : 240.  Beyond sixteen the planes are the faster form of the two; from 17
// to about 60 tokens of such wide weights neither is as fast as a product of the
// library's (24 tokens of 151936 x 4096: planes 1,716, a form on it 1,412).
#include <algorithm>

#include "grpo_linear.cuh"
#include "grpo_vec.cuh"

namespace grpo {
namespace {

static constexpr int kVec = 4, kThreads = 512, kWarps = kThreads / 32;
static constexpr int kHiddenBytes = 200 * 1024;  // of shared memory for the hidden states

__device__ __forceinline__ void launched_early() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void sum_up(float& m, float& Z, float& D, float x, float s2) {
  if (x > m) {
    const float u = fmaxf((m - x) * s2, -1000.f), k = exp2f(u);
    D = k * fmaf(Z, u, D);
    Z *= k;
    m = x;
  }
  const float u = (x - (m == -INFINITY ? 0.f : m)) * s2, e = ex2_fast(u);
  Z += e;
  D = fmaf(e, fmaxf(u, -1000.f), D);
}

// kGrad: the gradient of the logits, [V][rows]; else a record a CTA and row.
// The hidden states lie in shared memory; each of their vectors read serves
// four words (two where sixteen rows' sums leave no registers for more).
// Reads 6.0 TB/s with one row, 4.6 with eight (the fp32 cores and shared memory
// take about as long as memory then).  Rows that do not fit go in two launches.
template <int kRows, bool kGrad>
__global__ void __launch_bounds__(kThreads, 1) few_logits_kernel(const FewArgs a) {
  constexpr int kWords = kRows > 8 ? 2 : 4;
  extern __shared__ float4 s_mem[];
  __shared__ float4 s_part[kWarps][kRows];
  float* s_h = reinterpret_cast<float*>(s_mem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int K = (int)a.K, Kp = (K + 32 * kVec - 1) / (32 * kVec) * (32 * kVec);
  launched_early();
  const int count = a.count ? *a.count : a.N;
  for (int t = 0; t < kRows; ++t) {
    const bool in = a.first + t < count;
    const int64_t r = in ? (a.idx ? a.idx[a.first + t] : a.first + t) : 0;
    const float* row = (const float*)a.hidden + r / a.T * a.sb + r % a.T * a.st;
    for (int k = threadIdx.x; k < Kp; k += kThreads)
      s_h[t * Kp + k] = in && k < K ? __ldg(row + k) : 0.f;
  }
  // this lane's row, where it has one
  const int mine = a.first + lane;
  const bool live = lane < kRows && mine < count;
  float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
  int64_t id = -1;
  if (live) {
    if (kGrad) q = a.coef[mine], id = a.target[mine];
    else if (a.actions) id = a.actions[mine];
  }
  float m = -INFINITY, Z = 0.f, D = 0.f;
  __syncthreads();
  for (int64_t v0 = ((int64_t)blockIdx.x * kWarps + warp) * kWords; v0 < a.V;
       v0 += (int64_t)gridDim.x * kWarps * kWords) {
    float acc[kWords][kRows];
#pragma unroll
    for (int w = 0; w < kWords; ++w)
#pragma unroll
      for (int t = 0; t < kRows; ++t) acc[w][t] = 0.f;
    const float* word = (const float*)a.weight + v0 * a.sv + lane * kVec;
#pragma unroll 2
    for (int k = 0; k < Kp; k += 32 * kVec) {
      uint4 raw[kWords];
#pragma unroll
      for (int w = 0; w < kWords; ++w)
        raw[w] = v0 + w < a.V ? load_vec<float>(word + w * a.sv + k, K - k - lane * kVec) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int t = 0; t < kRows; ++t) {
        const float4 h = *reinterpret_cast<const float4*>(s_h + t * Kp + k + lane * kVec);
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          acc[w][t] = fmaf(h.x, __uint_as_float(raw[w].x), acc[w][t]);
          acc[w][t] = fmaf(h.y, __uint_as_float(raw[w].y), acc[w][t]);
          acc[w][t] = fmaf(h.z, __uint_as_float(raw[w].z), acc[w][t]);
          acc[w][t] = fmaf(h.w, __uint_as_float(raw[w].w), acc[w][t]);
        }
      }
    }
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      float x = 0.f;
#pragma unroll
      for (int t = 0; t < kRows; ++t) {
        float y = acc[w][t];
#pragma unroll
        for (int o = 16; o; o >>= 1) y += __shfl_xor_sync(~0u, y, o);
        x = lane == t ? y : x;
      }
      const int64_t v = v0 + w;
      if (v >= a.V) break;
      if constexpr (kGrad) {
        const float u = fmaxf((x - q.x) * a.s2, -1000.f);
        const float d = (id == v ? q.w : 0.f) - ex2_fast(u) * fmaf(q.z, u, q.y);
        if (lane < kRows) a.d[v * a.rows + mine] = live ? d : 0.f;
      } else {
        sum_up(m, Z, D, x, a.s2);
        if (live && id == v) a.xa[mine] = x;
      }
    }
  }
  if constexpr (!kGrad) {
    if (lane < kRows) s_part[warp][lane] = make_float4(m, Z, D, 0.f);
    __syncthreads();
    if (warp != 0 || !live) return;
    float top = -INFINITY;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_part[w][lane].x);
    const float ref = top == -INFINITY ? 0.f : top;
    float4 y = make_float4(top, 0.f, 0.f, 0.f);
    for (int w = 0; w < kWarps; ++w) {
      const float4 p = s_part[w][lane];
      const float u = fmaxf((p.x - ref) * a.s2, -1000.f), k = exp2f(u);
      y.y += p.y * k;
      y.z += k * fmaf(p.y, u, p.z);
    }
    a.part[(int64_t)blockIdx.x * a.rpad + mine] = y;
  }
}

// Both products of the gradient in one pass over the weight: dW's rows go out as
// they are summed, dh's sums stay in registers, one part of them a CTA.
// Words blockIdx.x of gridDim.x parts of the vocabulary, columns blockIdx.y.
static constexpr int kBackThreads = 256, kStage = 64;  // words whose gradients are staged

template <int kRows>
__global__ void __launch_bounds__(kBackThreads) few_back_kernel(const FewArgs a) {
  constexpr int kAhead = 8;
  __shared__ float s_d[kStage * kRows];
  launched_early();
  const int count = *a.count;
  const int64_t k = ((int64_t)blockIdx.y * kBackThreads + threadIdx.x) * kVec;
  const int n = (int)max((int64_t)0, min((int64_t)kVec, a.K - k));
  float h[kRows][kVec], acc[kRows][kVec];
#pragma unroll
  for (int t = 0; t < kRows; ++t) {
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (t < count) {
      const int64_t r = a.idx[t];
      raw = load_vec((const float*)a.hidden + r / a.T * a.sb + r % a.T * a.st + k, n);
    }
    Storage<float>::unpack(raw, h[t]);
#pragma unroll
    for (int i = 0; i < kVec; ++i) acc[t][i] = 0.f;
  }
  const int64_t from = a.V * blockIdx.x / gridDim.x, to = a.V * (blockIdx.x + 1) / gridDim.x;
  for (int64_t s0 = from; s0 < to; s0 += kStage) {
    const int words = (int)min((int64_t)kStage, to - s0);
    __syncthreads();
    for (int i = threadIdx.x; i < words * kRows; i += kBackThreads) s_d[i] = a.d[s0 * kRows + i];
    __syncthreads();
    for (int w0 = 0; w0 < words; w0 += kAhead) {
      uint4 raw[kAhead], more[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int64_t v = s0 + w0 + j;
        const int in = w0 + j < words ? n : 0;
        raw[j] = a.acc ? load_vec((const float*)a.weight + v * a.sv + k, in) : make_uint4(0, 0, 0, 0);
        more[j] = a.add ? load_vec((const float*)a.add + v * a.asv + k, in) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (w0 + j >= words) break;
        float d[kRows], x[kVec], y[kVec];
#pragma unroll
        for (int t = 0; t < kRows; ++t) d[t] = s_d[(w0 + j) * kRows + t];
        Storage<float>::unpack(raw[j], x);
        if (a.acc) {
#pragma unroll
          for (int t = 0; t < kRows; ++t)
#pragma unroll
            for (int i = 0; i < kVec; ++i) acc[t][i] = fmaf(d[t], x[i], acc[t][i]);
        }
        if (a.dweight) {
          Storage<float>::unpack(more[j], x);
#pragma unroll
          for (int i = 0; i < kVec; ++i) y[i] = 0.f;
#pragma unroll
          for (int t = 0; t < kRows; ++t)
#pragma unroll
            for (int i = 0; i < kVec; ++i) y[i] = fmaf(d[t], h[t][i], y[i]);
#pragma unroll
          for (int i = 0; i < kVec; ++i) y[i] += x[i];
          store_vec<float, kVec>((float*)a.dweight + (s0 + w0 + j) * a.gsv + k, n, y);
        }
      }
    }
  }
  if (a.acc) {
#pragma unroll
    for (int t = 0; t < kRows; ++t)
      store_vec<float, kVec>(a.acc + ((int64_t)blockIdx.x * kRows + t) * a.ldacc + k, n, acc[t]);
  }
}

cudaError_t launch(void (*k)(const FewArgs), dim3 grid, unsigned block, int smem, cudaStream_t s,
                   const FewArgs& a) {
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3(block);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, k, a);
}

int64_t hidden_bytes(int64_t K, int rows) { return (K + 127) / 128 * 128 * 4 * rows; }

// rows of one launch
int rows_at_once(int64_t K, int rows) {
  return hidden_bytes(K, rows) <= kHiddenBytes ? rows : rows / 2;
}

template <int kRows, bool kGrad>
cudaError_t logits(const FewArgs& a, int ctas, cudaStream_t s) {
  auto* k = few_logits_kernel<kRows, kGrad>;
  const int smem = (int)hidden_bytes(a.K, kRows);
  // (the limit is the function's, in all threads: never less than any call needs)
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kHiddenBytes);
  return e != cudaSuccess ? e : launch(k, dim3((unsigned)ctas), kThreads, smem, s, a);
}

template <bool kGrad>
cudaError_t all_logits(FewArgs a, int ctas, cudaStream_t s) {
  const int once = rows_at_once(a.K, a.rows);
  cudaError_t e = cudaSuccess;
  for (a.first = 0; a.first < a.rows && e == cudaSuccess; a.first += once) switch (once) {
      case 1: e = logits<1, kGrad>(a, ctas, s); break;
      case 2: e = logits<2, kGrad>(a, ctas, s); break;
      case 4: e = logits<4, kGrad>(a, ctas, s); break;
      case 8: e = logits<8, kGrad>(a, ctas, s); break;
      default: e = logits<16, kGrad>(a, ctas, s);
    }
  return e;
}

}  // namespace

int few_rows(grpo_dtype_t dt, int64_t N, int64_t K) {
  if (dt != GRPO_F32 || N < 1 || N > 16) return 0;
  int rows = 1;
  while (rows < N) rows *= 2;
  const int once = rows_at_once(K, rows);
  return once && hidden_bytes(K, once) <= kHiddenBytes ? rows : 0;
}

int few_parts(int64_t V, int64_t K, int sms) {
  const int64_t cols = kBackThreads * kVec, slices = (K + cols - 1) / cols;
  return (int)std::max<int64_t>(1, std::min<int64_t>(2 * sms / slices, (V + 7) / 8));
}

cudaError_t launch_few_stats(const FewArgs& a, int ctas, cudaStream_t s) {
  return all_logits<false>(a, ctas, s);
}

cudaError_t launch_few_grad(const FewArgs& a, int sms, cudaStream_t s) {
  const int words = kWarps * 4;
  return all_logits<true>(a, (int)std::min<int64_t>(sms, (a.V + words - 1) / words), s);
}

cudaError_t launch_few_back(const FewArgs& a, int parts, cudaStream_t s) {
  const int64_t cols = kBackThreads * kVec;
  const dim3 grid((unsigned)parts, (unsigned)((a.K + cols - 1) / cols));
  switch (a.rows) {
    case 1: return launch(few_back_kernel<1>, grid, kBackThreads, 0, s, a);
    case 2: return launch(few_back_kernel<2>, grid, kBackThreads, 0, s, a);
    case 4: return launch(few_back_kernel<4>, grid, kBackThreads, 0, s, a);
    case 8: return launch(few_back_kernel<8>, grid, kBackThreads, 0, s, a);
    default: return launch(few_back_kernel<16>, grid, kBackThreads, 0, s, a);
  }
}

}  // namespace grpo
