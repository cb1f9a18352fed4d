// Device helpers of the low-precision layer operators (the norm and its
// gradient, MX quantisation): chunks of eight elements, wave and workgroup
// reductions, and the roundings to 8 and 4 bits.
#pragma once

#include "skg_device.hpp"

namespace skg {

// A chunk is eight consecutive elements of a row: 16 bytes of a 16-bit type
// (one load instruction), 32 of fp32.  Rows may start at any element: the
// vector types below promise only the element's own alignment, which the
// hardware's unaligned global accesses take as they are.
template <int DT>
struct Elem;
template <>
struct Elem<DT_F16> {
  typedef uint16_t raw;
  SKG_DEV static float get(raw r) { return (float)__builtin_bit_cast(_Float16, r); }
  SKG_DEV static raw put(float v) { return to_f16_bits(v); }
};
template <>
struct Elem<DT_BF16> {
  typedef uint16_t raw;
  SKG_DEV static float get(raw r) { return __builtin_bit_cast(float, (uint32_t)r << 16); }
  SKG_DEV static raw put(float v) { return to_bf16_bits(v); }
};
template <>
struct Elem<DT_F32> {
  typedef uint32_t raw;
  SKG_DEV static float get(raw r) { return __builtin_bit_cast(float, r); }
  SKG_DEV static raw put(float v) { return __builtin_bit_cast(uint32_t, v); }
};

template <int DT>
struct Chunk {
  typedef typename Elem<DT>::raw raw;
  raw v[8];
  SKG_DEV float get(int i) const { return Elem<DT>::get(v[i]); }
  SKG_DEV void put(int i, float f) { v[i] = Elem<DT>::put(f); }
};
template <class C>
struct __attribute__((packed, aligned(sizeof(typename C::raw)))) Loose {
  C c;
};

// The first n (1 .. 8) elements to p.  The two paths' pointers are kept apart:
// joined by the compiler, whole chunks too would be stored in pieces (reading
// 8192x8192 e2m1 codes back took 52 us so, and 32 with whole stores).
template <int DT>
SKG_DEV void store_chunk(typename Elem<DT>::raw* p, int n, const Chunk<DT>& c) {
  if (n >= 8) {
    reinterpret_cast<Loose<Chunk<DT>>*>(p)->c = c;
  } else {
    asm volatile("" : "+v"(p));
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = c.v[i];
  }
}

// Elements e0 .. e0+7 of a row of cols elements in two steps, so that a row's
// loads are issued together, without a branch: the load takes the last
// eight elements instead where these reach past the end, and place_chunk
// then moves what is wanted into place and zeroes the rest.
// TAIL: 0 where cols is a multiple of eight, 1 where it is not, 2 where it is
// less than eight.
template <int DT, int TAIL>
SKG_DEV Chunk<DT> load_within(const typename Elem<DT>::raw* row, int e0, int cols) {
  if constexpr (TAIL < 2) {
    return reinterpret_cast<const Loose<Chunk<DT>>*>(row + min(e0, cols - 8))->c;
  } else {
    Chunk<DT> c;
#pragma unroll
    for (int i = 0; i < 8; ++i) c.v[i] = row[min(i, cols - 1)];
    return c;
  }
}
template <int DT, int TAIL>
SKG_DEV void place_chunk(Chunk<DT>& c, int e0, int cols) {
  constexpr int W = sizeof(c) / 4, E = 8 / W;  // words, elements in each
  struct Words {
    uint32_t w[W];
  };
  Words u = __builtin_bit_cast(Words, c);
  if (TAIL && e0 < cols && cols - e0 < 8) {
    const int d = TAIL == 1 ? e0 - (cols - 8) : 0, n = cols - e0;
#pragma unroll
    for (int b = 4; b >= E; b >>= 1)
#pragma unroll
      for (int i = 0; i < W; ++i) u.w[i] = d & b ? (i + b / E < W ? u.w[i + b / E] : 0) : u.w[i];
    if constexpr (E == 2) {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        u.w[i] = d & 1 ? u.w[i] >> 16 | (i + 1 < W ? u.w[i + 1] << 16 : 0) : u.w[i];
        u.w[i] = 2 * i + 1 < n ? u.w[i] : 2 * i < n ? u.w[i] & 0xffffu : 0;
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) u.w[i] = i < n ? u.w[i] : 0;
    }
  }
#pragma unroll
  for (int i = 0; i < W; ++i) u.w[i] = e0 < cols ? u.w[i] : 0;
  c = __builtin_bit_cast(Chunk<DT>, u);
}

// --- reductions --------------------------------------------------------------
struct OpSum {
  typedef float T;
  SKG_DEV static float zero() { return 0.f; }
  SKG_DEV static float op(float a, float b) { return a + b; }
};
// Largest of non-negative floats as their bit patterns: the order is the
// same, and a NaN, whose pattern is above infinity's, is kept.
struct OpMaxBits {
  typedef uint32_t T;
  SKG_DEV static uint32_t zero() { return 0u; }
  SKG_DEV static uint32_t op(uint32_t a, uint32_t b) { return a > b ? a : b; }
};
SKG_DEV uint32_t abs_bits(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu; }
SKG_DEV float from_bits(uint32_t b) { return __builtin_bit_cast(float, b); }

template <class Op, int CTRL, int ROWS = 0xf>
SKG_DEV typename Op::T dpp_step(typename Op::T v) {
  const int o = __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, Op::zero()), __builtin_bit_cast(int, v), CTRL,
                                            ROWS, 0xf, false);
  return Op::op(v, __builtin_bit_cast(typename Op::T, o));
}
// Over the four lanes of a quad (32 elements: an MX block).
template <class Op>
SKG_DEV typename Op::T quad_reduce(typename Op::T v) {
  v = dpp_step<Op, 0xB1>(v);
  return dpp_step<Op, 0x4E>(v);
}
// Over the wave, in a fixed order, without LDS traffic: within rows of 16
// lanes by data-parallel primitives, then across the rows; the result is
// wave-uniform.
template <class Op>
SKG_DEV typename Op::T wave_reduce(typename Op::T v) {
  v = quad_reduce<Op>(v);
  v = dpp_step<Op, 0x141>(v);       // mirror within half rows
  v = dpp_step<Op, 0x140>(v);       // mirror within rows
  v = dpp_step<Op, 0x142, 0xa>(v);  // last lane of a row onto the next row
  v = dpp_step<Op, 0x143, 0xc>(v);  // lane 31 onto the upper half
  return __builtin_bit_cast(typename Op::T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}
// Over a group of LANES neighbouring lanes (8 .. 64); every lane has the
// result.
template <class Op, int LANES>
SKG_DEV typename Op::T lanes_reduce(typename Op::T v) {
  if constexpr (LANES == 64) {
    return wave_reduce<Op>(v);
  } else {
    v = quad_reduce<Op>(v);
    v = dpp_step<Op, 0x141>(v);
    if constexpr (LANES >= 16) v = dpp_step<Op, 0x140>(v);
    if constexpr (LANES >= 32) v = Op::op(v, __shfl_xor(v, 16));
    return v;
  }
}
// Over a group of LANES lanes or, with 64, of WAVES waves; `slot` is WAVES
// words of LDS that nobody else uses until the next workgroup barrier.
template <class Op, int WAVES, int LANES>
SKG_DEV typename Op::T group_reduce(typename Op::T v, SKG_LDS uint32_t* slot) {
  v = lanes_reduce<Op, LANES>(v);
  if constexpr (WAVES > 1) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = __builtin_bit_cast(uint32_t, v);
    __syncthreads();
    v = __builtin_bit_cast(typename Op::T, (uint32_t)slot[0]);
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v = Op::op(v, __builtin_bit_cast(typename Op::T, (uint32_t)slot[w]));
  }
  return v;
}

// 1 / sqrt(v) within half an ulp or so: the hardware's reciprocal square
// root and one Newton step.  A subnormal v, which the instruction takes for
// zero, is scaled by an even power of two.  Infinite for a zero, 0 for an
// infinite v, NaN for a NaN.
SKG_DEV float rsqrt_refined(float v) {
  const bool small = v < 0x1p-126f;
  const float u = small ? v * 0x1p+64f : v;
  const float r = __builtin_amdgcn_rsqf(u);
  const float e = __builtin_fmaf(-u * r, r, 1.f);
  const float n = __builtin_fmaf(0.5f * r, e, r);
  const float f = u > 0.f && u < 3e38f ? n : r;
  return small ? f * 0x1p+32f : f;
}

// --- MX codes ------------------------------------------------------------------
// E8M0 code of a block whose largest magnitude has the bits `top`: the
// exponent of that magnitude less the format's largest one (2 for e2m1, 8
// for e4m3), so the block's largest element lands in the format's top binade
// and is rounded or saturated there.  255 where the block holds an infinity
// or NaN.
template <int EMAX>
SKG_DEV uint32_t mx_code(uint32_t top) {
  const int e = (int)(top >> 23);
  return e == 255 ? 255u : (uint32_t)(e > EMAX ? e - EMAX : 0);
}
// 1 / 2^(code - 127); 0 for the NaN code, whose block holds zeros.  code
// is at most 252 otherwise, so the result is a normal number.
SKG_DEV float mx_inverse(uint32_t code) { return code == 255 ? 0.f : from_bits((254u - code) << 23); }
// 2^(code - 127); the NaN code gives NaN.
SKG_DEV float mx_value(uint32_t code) {
  return from_bits(code == 255 ? 0x7fc00000u : code ? code << 23 : 0x00400000u);
}

// Eight values to e4m3 / e2m1 codes, round to nearest even, saturating; the
// first element in the low bits.
SKG_DEV uint2 pack_e4m3(const float (&v)[8]) {
  float c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = __builtin_amdgcn_fmed3f(v[i], -448.f, 448.f);
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(c[4], c[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(c[6], c[7], hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}
// The same for values already within +-448 (up to rounding) or NaN, which
// stays NaN.
SKG_DEV uint2 pack_e4m3_nan(const float (&v)[8]) {
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}
SKG_DEV uint32_t pack_e2m1(const float (&v)[8]) {
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], 1.f, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], 1.f, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], 1.f, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], 1.f, 3);
  return q;
}

template <class V>
SKG_DEV void store_loose(void* p, const V& v) {
  struct __attribute__((packed, aligned(1))) L {
    V v;
  };
  reinterpret_cast<L*>(p)->v = v;
}
template <class V>
SKG_DEV V load_loose(const void* p) {
  struct __attribute__((packed, aligned(1))) L {
    V v;
  };
  return reinterpret_cast<const L*>(p)->v;
}

}  // namespace skg
