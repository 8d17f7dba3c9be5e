// row_io.hpp -- eight consecutive elements of a row of f32 or bf16, to and from f32 registers.
//
// Rows start wherever their stride puts them: an odd stride leaves them aligned to one element
// only.  The 16-byte accesses are therefore written as copies of unaligned vectors, which the
// hardware serves in one instruction (global memory takes vector accesses at any byte), and
// only the last, partial group of a row goes element by element.
#pragma once

#include "common.hpp"

namespace moe {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

// One vector from and to memory; PASS: past the caches, for what is not read again soon.
template <bool PASS, typename V, typename P>
__device__ __forceinline__ void put(P* p, V v) {
  if constexpr (PASS)
    __builtin_nontemporal_store(v, p);
  else
    *p = v;
}
template <bool PASS, typename P>
__device__ __forceinline__ auto get(const P* p) {
  if constexpr (PASS)
    return __builtin_nontemporal_load(p);
  else
    return *p;
}

// Eight elements from p; those at n and beyond are not read and are 0.
__device__ __forceinline__ void load8(const float* p, int n, float (&v)[8]) {
  if (n >= 8) {
    const f32x4 a = *reinterpret_cast<const f32x4_any*>(p), b = *reinterpret_cast<const f32x4_any*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.0f;
  }
}

__device__ __forceinline__ void load8(const uint16_t* p, int n, float (&v)[8]) {
  if (n >= 8) {
    const u32x4 a = *reinterpret_cast<const u32x4_any*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? bf16_bits_to_f32(p[i]) : 0.0f;
  }
}

// load8 in two halves: what memory holds, and its values, so that several loads can be on their way.  PASS: past
// the caches, for rows that are read once.
template <typename E>
struct Raw8;
template <>
struct Raw8<uint16_t> {
  u32x4 a;
  template <bool PASS>
  __device__ __forceinline__ void load(const uint16_t* p, int n) {
    if (n >= 8) {
      a = get<PASS>(reinterpret_cast<const u32x4_any*>(p));
    } else {
      a = u32x4{0, 0, 0, 0};
      if (n > 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          a[i] = (2 * i < n ? p[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)p[2 * i + 1] << 16 : 0u);
      }
    }
  }
  __device__ __forceinline__ float operator[](int i) const {
    return __uint_as_float(i & 1 ? a[i / 2] & 0xffff0000u : a[i / 2] << 16);
  }
};
template <>
struct Raw8<float> {
  float v[8];
  template <bool PASS>
  __device__ __forceinline__ void load(const float* p, int n) {
    if (n >= 8) {
      const f32x4 lo = get<PASS>(reinterpret_cast<const f32x4_any*>(p)), hi = get<PASS>(reinterpret_cast<const f32x4_any*>(p + 4));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = lo[i];
        v[4 + i] = hi[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.0f;
    }
  }
  __device__ __forceinline__ float operator[](int i) const { return v[i]; }
};

// Two f32 to two bf16, round to nearest even (the conversion instruction of gfx950).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const bf16x2 v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}

template <bool PASS = false>
__device__ __forceinline__ void store8(float* p, int n, const float (&v)[8]) {
  if (n >= 8) {
    put<PASS>(reinterpret_cast<f32x4_any*>(p), f32x4{v[0], v[1], v[2], v[3]});
    put<PASS>(reinterpret_cast<f32x4_any*>(p + 4), f32x4{v[4], v[5], v[6], v[7]});
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = v[i];
  }
}

template <bool PASS = false>
__device__ __forceinline__ void store8(uint16_t* p, int n, const float (&v)[8]) {
  u32x4 a;
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
  if (n >= 8) {
    put<PASS>(reinterpret_cast<u32x4_any*>(p), a);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint16_t)(a[i / 2] >> (16 * (i & 1)));
  }
}

// Reductions over lanes without the trip through LDS that a general shuffle takes: within 16 lanes by
// data-parallel permutes (exchange with lane ^ 1, ^ 2, then mirrored over 8 and 16 lanes, whose halves agree by
// then), across them by swapping 16- and 32-lane halves.  Every lane gets the result.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xf, 0xf, true));
}
struct Add {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct Max {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
template <typename Op>
__device__ __forceinline__ float reduce16(float v, Op op) {
  v = op(v, dpp<0xb1>(v));   // quad_perm 1 0 3 2
  v = op(v, dpp<0x4e>(v));   // quad_perm 2 3 0 1
  v = op(v, dpp<0x141>(v));  // row_half_mirror
  return op(v, dpp<0x140>(v));  // row_mirror
}
template <typename Op>
__device__ __forceinline__ float reduce64(float v, Op op) {
  v = reduce16(v, op);
  const uint32_t a = __float_as_uint(v);
  const auto p = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  v = op(__uint_as_float(p[0]), __uint_as_float(p[1]));
  const uint32_t b = __float_as_uint(v);
  const auto q = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return op(__uint_as_float(q[0]), __uint_as_float(q[1]));
}

}  // namespace moe
