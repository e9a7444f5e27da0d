// row_io.h -- rows of bf16, fp16 or fp32 values in pieces of eight (private to
// libnf4): the loads and stores that the int8 encoder and the routing kernels
// share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "int8.h"
#include "nf4_device.h"

namespace rowio {

using nf4dev::u32x4;

// Rows of K elements lie back to back, so with an odd K a row starts at any
// multiple of the element size.  gfx950 reads and writes global memory at any
// byte address; these types tell the compiler that it may not assume more than
// the element's alignment.
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_a2 __attribute__((aligned(2)));

__device__ __host__ constexpr int dtype_bytes(int dt) { return dt == INT8_FP32 ? 4 : 2; }

// Eight consecutive elements as loaded.
template <int DT>
struct Piece {
  u32x4 v[DT == INT8_FP32 ? 2 : 1];
};

// Elements [at, at + 8) of the row at p, all of which exist.  STREAM: read once, and
// not worth a place in the caches.
template <int DT, bool STREAM = false>
__device__ __forceinline__ Piece<DT> whole_piece(const void* p, int64_t at) {
  Piece<DT> r;
  const char* a = static_cast<const char*>(p) + at * dtype_bytes(DT);
  // (spelled out: a template would lose the types' alignment)
  if constexpr (DT == INT8_FP32) {
    const u32x4_a4* v = reinterpret_cast<const u32x4_a4*>(a);
    r.v[0] = STREAM ? __builtin_nontemporal_load(v) : *v;
    r.v[1] = STREAM ? __builtin_nontemporal_load(v + 1) : v[1];
  } else {
    const u32x4_a2* v = reinterpret_cast<const u32x4_a2*>(a);
    r.v[0] = STREAM ? __builtin_nontemporal_load(v) : *v;
  }
  return r;
}

// Elements [at, at + 8) of the n elements at p; those past n are zero.
template <int DT>
__device__ __forceinline__ Piece<DT> load_piece(const void* p, int64_t at, int64_t n) {
  Piece<DT> r;
  const char* a = static_cast<const char*>(p) + at * dtype_bytes(DT);
  if (at + 8 <= n) return whole_piece<DT>(p, at);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (DT == INT8_FP32) {
      r.v[i >> 2][i & 3] = at + i < n ? reinterpret_cast<const uint32_t*>(a)[i] : 0u;
    } else {
      const uint32_t h = at + i < n ? reinterpret_cast<const uint16_t*>(a)[i] : 0u;
      r.v[0][i >> 1] = i & 1 ? r.v[0][i >> 1] | (h << 16) : h;
    }
  }
  return r;
}

template <int DT>
__device__ __forceinline__ void store_whole_piece(void* p, int64_t at, const Piece<DT>& r) {
  char* a = static_cast<char*>(p) + at * dtype_bytes(DT);
  if constexpr (DT == INT8_FP32) {
    *reinterpret_cast<u32x4_a4*>(a) = r.v[0];
    *reinterpret_cast<u32x4_a4*>(a + 16) = r.v[1];
  } else {
    *reinterpret_cast<u32x4_a2*>(a) = r.v[0];
  }
}

template <int DT>
__device__ __forceinline__ void store_piece(void* p, int64_t at, int64_t n, const Piece<DT>& r) {
  char* a = static_cast<char*>(p) + at * dtype_bytes(DT);
  if (at + 8 <= n) return store_whole_piece<DT>(p, at, r);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (at + i < n) {
      if constexpr (DT == INT8_FP32)
        reinterpret_cast<uint32_t*>(a)[i] = r.v[i >> 2][i & 3];
      else
        reinterpret_cast<uint16_t*>(a)[i] = static_cast<uint16_t>(r.v[0][i >> 1] >> (16 * (i & 1)));
    }
}

// Element i of a piece as fp32 (exact).
template <int DT>
__device__ __forceinline__ float element(const Piece<DT>& r, int i) {
  if constexpr (DT == INT8_FP32) {
    const uint32_t w = r.v[i >> 2][i & 3];  // a copy: bit_cast of a vector's element takes element 0
    return __builtin_bit_cast(float, w);
  } else {
    const uint32_t w = r.v[0][i >> 1];
    if constexpr (DT == INT8_BF16)
      return __builtin_bit_cast(float, i & 1 ? w & 0xFFFF0000u : w << 16);
    else
      return nf4dev::f16_to_f32(static_cast<uint16_t>(w >> (16 * (i & 1))));
  }
}

// Eight fp32 values rounded to nearest even.
template <int DT>
__device__ __forceinline__ Piece<DT> make_piece(const float (&f)[8]) {
  Piece<DT> r;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    if constexpr (DT == INT8_FP32) {
      r.v[i >> 2][i & 3] = __builtin_bit_cast(uint32_t, f[i]);
      r.v[i >> 2][(i & 3) + 1] = __builtin_bit_cast(uint32_t, f[i + 1]);
    } else {
      r.v[0][i >> 1] = nf4dev::pack_pair<DT>(f[i], f[i + 1]);
    }
  }
  return r;
}

inline bool known_dtype(int32_t dt) { return dt == INT8_BF16 || dt == INT8_FP16 || dt == INT8_FP32; }

// Runs f with the type as a constant.
template <class F>
inline void with_dtype(int32_t dt, F&& f) {
  switch (dt) {
    case INT8_BF16: f(std::integral_constant<int, INT8_BF16>{}); break;
    case INT8_FP16: f(std::integral_constant<int, INT8_FP16>{}); break;
    default: f(std::integral_constant<int, INT8_FP32>{}); break;
  }
}

}  // namespace rowio
