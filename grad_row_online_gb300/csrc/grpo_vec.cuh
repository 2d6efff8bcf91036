// grpo_vec.cuh -- 16-byte pieces of rows that may start anywhere and end
// anywhere: read, written as they are or from fp32.
#pragma once

#include "grpo_internal.cuh"

namespace grpo {

// `n` (at most a 16-byte vector's) elements of a row as they lie, zeros behind them
template <typename T>
__device__ __forceinline__ uint4 load_vec(const T* p, int n) {
  constexpr int kVec = Storage<T>::kVec;
  if (n >= kVec && ((uintptr_t)p & 15) == 0) return __ldg(reinterpret_cast<const uint4*>(p));
  if constexpr (kVec == 4) {
    const unsigned* q = reinterpret_cast<const unsigned*>(p);
    return make_uint4(n > 0 ? __ldg(q) : 0u, n > 1 ? __ldg(q + 1) : 0u, n > 2 ? __ldg(q + 2) : 0u,
                      n > 3 ? __ldg(q + 3) : 0u);
  } else {
    const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
    unsigned h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = i < n ? __ldg(q + i) : 0u;
    return make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
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

// a vector as it lies, `n` elements of it inside
template <typename T>
__device__ __forceinline__ void store_raw(T* p, int n, const uint4& v) {
  constexpr int kVec = Storage<T>::kVec;
  if (n >= kVec && ((uintptr_t)p & 15) == 0) {
    *reinterpret_cast<uint4*>(p) = v;
  } else {
    const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (i < n) {
        if constexpr (kVec == 4) reinterpret_cast<unsigned*>(p)[i] = w[i];
        else reinterpret_cast<unsigned short*>(p)[i] = (unsigned short)(w[i / 2] >> (i & 1) * 16);
      }
  }
}

}  // namespace grpo
