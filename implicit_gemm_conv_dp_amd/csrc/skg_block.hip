// Quantisation to 8-bit codes with an fp32 scale for each block: 128 elements
// along a row, along a column (written transposed), or 128 x 128.
//
// With top the largest magnitude of a block and MAX the format's largest value
// (448 for e4m3, 57344 for e5m2): the scale is d = max(top / MAX, 2^-126) in fp32
// and a code is the one nearest to x MAX / top (x / 2^-126 where d is that
// bound), the even one of two.  16-bit inputs often lie just between two codes
// (x MAX is exact in fp32), so the quotient is rounded correctly before it is
// rounded to a code: a reciprocal and one residual step, four operations an
// element.  One that is not just between two codes is 2^-16 of itself away from
// there, so its rounding to fp32 stays on its side.  fp32 inputs' quotients can be
// closer than that: of those that come near a border the side is decided exactly.
//
// A workgroup takes 128 x 128 elements, from one read for every output that is
// asked for: the rows' codes go straight from registers, the columns' by way of
// LDS, so both take whole 128-byte runs.  Bound by memory traffic: 16384 x 4096 bf16
// both ways takes 54 us alone, 60 us one call after another, 4.5 to 5 TB/s of reads
// and writes (a large copy: 5.4).
#include <algorithm>
#include <exception>
#include <string>

#include "skg_internal.hpp"
#include "skg_lowp.hpp"

namespace skg {
namespace {

struct BlockParams {
  const char* x;
  char *q, *qt;
  float *s, *st;
  int64_t rows, cols, kq, kqt;
  int64_t ldx, ldq, ldqt;  // elements
  int64_t rblocks, cblocks;  // ceil(rows / 128), ceil(cols / 128)
  uint32_t across, first;  // tiles along the columns; tile of the launch's first workgroup
};

// How a block's elements become codes: v -> v a / t, rounded correctly.
struct Quotient {
  float a, t, inv, d;
};
template <bool E5M2>
SKG_DEV Quotient block_quotient(uint32_t top) {
  constexpr float MAX = E5M2 ? 57344.f : 448.f;
  Quotient r;
  const float m = from_bits(top);
  // m / MAX, rounded correctly (checked for every fp32 m of this branch's range).
  constexpr float INV = 1.f / MAX;
  const float over = m * INV;
  r.d = __builtin_fmaf(__builtin_fmaf(-over, MAX, m), INV, over);
  if (m < MAX * 0x1p-126f) {
    r.d = 0x1p-126f;
    r.a = 0x1p+126f;
    r.t = r.inv = 1.f;
  } else {
    // Both sides of the quotient by the power of two that brings top into
    // [1, 2): no step leaves the range of fp32.
    const uint32_t e = top >> 23;
    const float p = from_bits(e >= 254 ? 0x00400000u : (254u - e) << 23);
    r.a = MAX * p;
    r.t = m * p;
    // To 2^-24: a code's quotient takes a residual step, which squares the error.
    const float inv = __builtin_amdgcn_rcpf(r.t);
    r.inv = __builtin_fmaf(__builtin_fmaf(-r.t, inv, 1.f), inv, inv);
  }
  // An infinity or NaN makes the whole block NaN.
  if (top >= 0x7f800000u) r.a = r.d = __builtin_nanf("");
  return r;
}
SKG_DEV float quotient(float v, const Quotient& r) {
  const float n = v * r.a, q = n * r.inv;
  const float over = __builtin_fmaf(q, r.t, -n);  // (this way round a -0 stays one)
  return __builtin_fmaf(-over, r.inv, q);
}
// The same for an fp32 element, whose product with a is not exact, from a quotient q at
// most three steps of fp32 off: a number on the real quotient's side of every border
// between codes, or on the border.  Borders have few bits, so none but q rounded to a
// multiple of eight steps can lie between the two; what v a exceeds that times t by is
// exact but for the last addition, which keeps its sign.
SKG_DEV float quotient_side(float v, float q, const Quotient& r) {
  const uint32_t b = (__builtin_bit_cast(uint32_t, q) + 4) & ~7u;
  const float n = v * r.a, lost = __builtin_fmaf(v, r.a, -n);
  const float left = __builtin_fmaf(-from_bits(b), r.t, n) + lost;
  const int side = (int)(__builtin_bit_cast(uint32_t, left) ^ b) >> 31 | 1;  // away from zero or towards it
  return from_bits(b + (left == 0.f ? 0 : side));
}
template <bool E5M2>
SKG_DEV uint2 pack_codes(const float (&v)[8]) {
  if constexpr (!E5M2) {
    return pack_e4m3_nan(v);
  } else {
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_bf8_f32(v[0], v[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_bf8_f32(v[2], v[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_bf8_f32(v[4], v[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_bf8_f32(v[6], v[7], hi, true);
    return make_uint2((uint32_t)lo, (uint32_t)hi);
  }
}
// The largest magnitude of eight elements, as fp32 bits; 16-bit ones are compared
// as they are, two at a time.
template <int DT>
SKG_DEV uint32_t top_bits(const Chunk<DT>& c) {
  if constexpr (DT == DT_F32) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = OpMaxBits::op(m, abs_bits(c.get(j)));
    return m;
  } else {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    struct Words {
      uint32_t w[4];
    };
    const Words u = __builtin_bit_cast(Words, c);
    u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, u.w[i] & 0x7fff7fffu));
    Chunk<DT> top;
    top.v[0] = __builtin_bit_cast(typename Elem<DT>::raw, (uint16_t)(m[0] > m[1] ? m[0] : m[1]));
    return abs_bits(top.get(0));
  }
}
template <int DT, bool E5M2>
SKG_DEV uint2 block_codes(const Chunk<DT>& c, const Quotient& r) {
  float v[8];
  if constexpr (DT != DT_F32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = quotient(c.get(j), r);
  } else {
    // A product with the rounded a / t is at most three steps of fp32 off.  That is
    // enough unless it is within four of a border: just between two normal codes, where
    // the bit after a code's last one is set and no later one, or between subnormal
    // ones, below the smallest normal one (zeros aside).  Then the sides of all eight
    // are decided.  Of normal data it is one wave in 30: 16384 x 4096 to e4m3 both ways
    // takes 86 us (88 with a residual step for each element, which is not enough; 107
    // with an exact remainder for each).  Of bf16 values held in fp32, whose quotients
    // often are borders, it is most: 95 us (83), and 512 x 1152 to e5m2 8.0 (6.7).
    constexpr int HALF = E5M2 ? 20 : 19;
    constexpr uint32_t NORMAL = (E5M2 ? 127u - 14u : 127u - 6u) << 24;
    const float rate = r.a * r.inv;
    uint32_t border = ~0u, small = ~0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = c.get(j) * rate;
      const uint32_t b = __builtin_bit_cast(uint32_t, v[j]);
      border = min(border, (b + (1u << HALF) + 4) << (31 - HALF));
      small = min(small, (b << 1) - 1);  // (zeros wrap around)
    }
    if (border <= 8u << (31 - HALF) || small < NORMAL - 1) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = quotient_side(c.get(j), v[j], r);
    }
  }
  return pack_codes<E5M2>(v);
}

constexpr int kB = 128;
// A row of the tile in LDS is 8 bytes longer than its elements, and 16-bit
// groups of four columns are exchanged in every other 32 rows: the 64 reads of a
// wave (16 row groups, 4 column groups) fall on all banks evenly.
template <int DT>
struct BTile {
  static constexpr int THREADS = 512, ES = sizeof(typename Elem<DT>::raw);
  static constexpr int N = kB * kB / 8 / THREADS;  // chunks a thread
  static constexpr int P = kB * ES + 8, GB = 4 * ES;
  SKG_DEV static SKG_LDS char* at(SKG_LDS char* tile, int r, int g) {
    return tile + r * P + (ES == 2 ? g ^ ((r >> 5 & 1) << 2) : g) * GB;
  }
};

// TALL: one scale for the whole tile.  COLS: the transposed codes are wanted.
template <int DT, bool E5M2, bool TALL, bool COLS, int TAIL>
SKG_DEV void block_tile(const BlockParams& p, SKG_LDS char* tile, SKG_LDS uint32_t* slots) {
  typedef typename Elem<DT>::raw raw;
  typedef BTile<DT> T;
  const uint32_t id = p.first + blockIdx.x, down = id / p.across;
  const int64_t r0 = (int64_t)down * kB, kb = id - down * p.across, c0 = kb * kB;
  Chunk<DT> in[T::N];
#pragma unroll
  for (int u = 0; u < T::N; ++u) {
    const int k = u * T::THREADS + threadIdx.x;
    const int64_t r = min(r0 + k / 16, p.rows - 1);
    if (p.rows > 0 && p.cols > 0)
      in[u] = load_within<DT, TAIL>(reinterpret_cast<const raw*>(p.x) + r * p.ldx, (int)c0 + k % 16 * 8, (int)p.cols);
    else
      in[u] = Chunk<DT>{};
  }
  uint32_t top[T::N], all = 0;
#pragma unroll
  for (int u = 0; u < T::N; ++u) {
    const int k = u * T::THREADS + threadIdx.x, r = k / 16, g = k % 16 * 2;
    place_chunk<DT, TAIL>(in[u], (int)c0 + g * 4, (int)p.cols);
    if (r0 + r >= p.rows) in[u] = Chunk<DT>{};
    top[u] = top_bits(in[u]);
    if constexpr (TALL)
      all = OpMaxBits::op(all, top[u]);
    else
      top[u] = lanes_reduce<OpMaxBits, 16>(top[u]);
    if constexpr (COLS) {
      typedef uint32_t words __attribute__((ext_vector_type(T::GB / 4), aligned(8)));
      struct Two {
        words w[2];
      };
      const Two two = __builtin_bit_cast(Two, in[u]);
      *(SKG_LDS words*)T::at(tile, r, g) = two.w[0];
      *(SKG_LDS words*)T::at(tile, r, g + 1) = two.w[1];
    }
  }
  Quotient whole;
  if constexpr (TALL) {
    all = wave_reduce<OpMaxBits>(all);
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = all;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < T::THREADS / 64; ++w) all = OpMaxBits::op(all, slots[w]);
    whole = block_quotient<E5M2>(all);
    if (threadIdx.x == 0) {
      if (p.q && r0 < p.rows && c0 < p.kq) p.s[kb * p.rblocks + down] = whole.d;
      if (COLS && c0 < p.cols && r0 < p.kqt) p.st[(int64_t)down * p.cblocks + kb] = whole.d;
    }
  }
  if (p.q && c0 < p.kq) {
#pragma unroll
    for (int u = 0; u < T::N; ++u) {
      const int k = u * T::THREADS + threadIdx.x;
      const int64_t r = r0 + k / 16;
      const Quotient o = TALL ? whole : block_quotient<E5M2>(top[u]);
      if (r < p.rows) {
        store_loose(p.q + r * p.ldq + c0 + k % 16 * 8, block_codes<DT, E5M2>(in[u], o));
        if (!TALL && k % 16 == 0) p.s[kb * p.rows + r] = o.d;
      }
    }
  }
  if constexpr (COLS) {
    if (!TALL) __syncthreads();
    const int oct = threadIdx.x & 15, grp = threadIdx.x >> 4;
    const int64_t k0 = r0 + oct * 8;
    struct Group {
      raw v[4];
    };
    Chunk<DT> v[4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      typedef uint32_t words __attribute__((ext_vector_type(T::GB / 4), aligned(8)));
      const Group e = __builtin_bit_cast(Group, *(const SKG_LDS words*)T::at(tile, oct * 8 + i, grp));
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j].v[i] = e.v[j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t line = c0 + grp * 4 + j;
      Quotient o;
      if constexpr (TALL) {
        o = whole;
      } else {
        o = block_quotient<E5M2>(lanes_reduce<OpMaxBits, 16>(top_bits(v[j])));
      }
      if (line < p.cols && k0 < p.kqt) {
        store_loose(p.qt + line * p.ldqt + k0, block_codes<DT, E5M2>(v[j], o));
        if (!TALL && oct == 0) p.st[(int64_t)down * p.cols + line] = o.d;
      }
    }
  }
}

template <int DT, bool E5M2, bool TALL, bool COLS>
__global__ __launch_bounds__(BTile<DT>::THREADS) void block_quant_kernel(BlockParams p) {
  typedef BTile<DT> T;
  __shared__ __attribute__((aligned(16))) char tile_[COLS ? kB * T::P : 16];
  __shared__ uint32_t slots_[8];
  SKG_LDS char* tile = (SKG_LDS char*)tile_;
  SKG_LDS uint32_t* slots = (SKG_LDS uint32_t*)slots_;
  if (!(p.cols & 7)) return block_tile<DT, E5M2, TALL, COLS, 0>(p, tile, slots);
  if (p.cols >= 8) return block_tile<DT, E5M2, TALL, COLS, 1>(p, tile, slots);
  block_tile<DT, E5M2, TALL, COLS, 2>(p, tile, slots);
}

bool row_type(int dt) { return dt == SKG_F16 || dt == SKG_BF16 || dt == SKG_F32; }
bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int check_side(const void* q, const void* s, int64_t kq, int64_t axis, int64_t ldq) {
  if (kq < axis || kq % kB) return unsupported("kq and kqt must be multiples of 128 and cover the quantised axis");
  if (ldq < kq) return unsupported("leading dimension too small");
  if (kq > INT32_MAX - 4096) return unsupported("dimension too large");
  if (!s) return unsupported("codes need their scales");
  if (!aligned_to(s, 4)) return unsupported("pointers must be aligned to their elements");
  return SKG_OK;
}

int run_block_quant(const skg_block_quant_args_t* a, hipStream_t st) {
  if (!a) return unsupported("null arguments");
  if (!row_type(a->dtype)) return unsupported("elements come from f16, bf16 or f32");
  if (a->dtype_q != SKG_F8E4M3 && a->dtype_q != SKG_F8E5M2) return unsupported("block codes are e4m3 or e5m2");
  if (a->block != SKG_BLOCK_1x128 && a->block != SKG_BLOCK_128x128) return unsupported("unknown block shape");
  if (a->rows < 0 || a->cols < 0) return unsupported("rows and cols must not be negative");
  const int64_t most = INT32_MAX - 4096;  // rounded up to tiles within 32 bits
  if (a->rows > most || a->cols > most) return unsupported("dimension too large");
  if (a->ldx < a->cols) return unsupported("leading dimension too small");
  int rc;
  if (a->q && (rc = check_side(a->q, a->scales, a->kq, a->cols, a->ldq))) return rc;
  if (a->qt && (rc = check_side(a->qt, a->scales_t, a->kqt, a->rows, a->ldqt))) return rc;
  if (!a->q && !a->qt) return unsupported("neither q nor qt is asked for");
  // Tiles that some output needs.
  const int64_t down = std::max(a->q ? ceil_div(a->rows, kB) : 0, a->qt ? ceil_div(a->kqt, kB) : 0);
  const int64_t across = std::max(a->q ? ceil_div(a->kq, kB) : 0, a->qt ? ceil_div(a->cols, kB) : 0);
  if (down == 0 || across == 0) return SKG_OK;
  if (a->rows > 0 && a->cols > 0 && !a->x) return unsupported("null x");
  if (!aligned_to(a->x, elem_bytes(a->dtype))) return unsupported("pointers must be aligned to their elements");
  int cus = 0;
  rc = check_device(&cus);
  if (rc) return rc;
  BlockParams p;
  p.x = static_cast<const char*>(a->x);
  p.q = static_cast<char*>(a->q);
  p.qt = static_cast<char*>(a->qt);
  p.s = a->scales;
  p.st = a->scales_t;
  p.rows = a->rows;
  p.cols = a->cols;
  p.kq = a->kq;
  p.kqt = a->qt ? a->kqt : 0;
  p.ldx = a->ldx;
  p.ldq = a->ldq;
  p.ldqt = a->ldqt;
  p.rblocks = ceil_div(a->rows, kB);
  p.cblocks = ceil_div(a->cols, kB);
  p.across = (uint32_t)across;
  auto launch = [&](auto dt, auto e5, auto tall, auto cols) {
    constexpr int DT = decltype(dt)::value, THREADS = BTile<DT>::THREADS;
    const int64_t tiles = down * across;
    if (tiles > INT32_MAX) return unsupported("too many tiles");
    // Tiles in launches of fewer than 2^32 threads.
    constexpr int64_t most = kMostThreads / THREADS;
    for (int64_t t0 = 0; t0 < tiles; t0 += most) {
      BlockParams q = p;
      q.first = (uint32_t)t0;
      hipLaunchKernelGGL((block_quant_kernel<DT, decltype(e5)::value, decltype(tall)::value, decltype(cols)::value>),
                         dim3((unsigned)std::min(most, tiles - t0)), dim3(THREADS), 0, st, q);
    }
    return SKG_OK;
  };
  auto by_form = [&](auto dt, auto e5) {
    typedef std::integral_constant<bool, true> yes;
    typedef std::integral_constant<bool, false> no;
    if (a->block == SKG_BLOCK_128x128) return a->qt ? launch(dt, e5, yes{}, yes{}) : launch(dt, e5, yes{}, no{});
    return a->qt ? launch(dt, e5, no{}, yes{}) : launch(dt, e5, no{}, no{});
  };
  auto by_fmt = [&](auto dt) {
    if (a->dtype_q == SKG_F8E5M2) return by_form(dt, std::integral_constant<bool, true>{});
    return by_form(dt, std::integral_constant<bool, false>{});
  };
  if (a->dtype == SKG_F16)
    rc = by_fmt(std::integral_constant<int, DT_F16>{});
  else if (a->dtype == SKG_BF16)
    rc = by_fmt(std::integral_constant<int, DT_BF16>{});
  else
    rc = by_fmt(std::integral_constant<int, DT_F32>{});
  if (rc) return rc;
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return hip_failure(std::string("launch: ") + hipGetErrorString(e));
  return SKG_OK;
}

}  // namespace
}  // namespace skg

using namespace skg;

extern "C" int skg_run_block_quant(const skg_block_quant_args_t* a, void* stream) {
  try {
    clear_error();
    return run_block_quant(a, static_cast<hipStream_t>(stream));
  } catch (const std::exception& ex) {
    return hip_failure(std::string("exception: ") + ex.what());
  } catch (...) {
    return hip_failure("unknown exception");
  }
}
