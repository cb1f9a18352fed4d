// MX quantisation along the rows or, transposed, along the columns, and
// reading back.
//
// A block is 32 consecutive elements of the quantised axis.  With top the
// largest magnitude of the block and E its fp32 exponent field, the block's
// E8M0 code is max(E - emax, 0) (emax 2 for e2m1, 8 for e4m3) and its elements
// are round-to-nearest-even, saturating, of x / 2^(code - 127).  Dividing by a
// power of two is exact, so each element is rounded once.  A block that
// holds an infinity or a NaN gets code 255 (NaN) and zero elements.
#include <algorithm>
#include <exception>
#include <string>

#include "skg_internal.hpp"
#include "skg_lowp.hpp"

namespace skg {
namespace {

struct MxParams {
  const char* x;
  char* q;
  uint8_t* sc;
  int64_t rows, cols, kq;  // kq: elements written along the quantised axis
  int64_t ldx, ldq;        // elements
  uint32_t first;          // along the columns: tile of the launch's first workgroup
};

// Along the rows and reading back: U chunks of eight elements a thread, four
// neighbouring lanes a block.  Chunks are numbered through the lines (fewer
// than 2^31 a launch); cpr, a multiple of four, is how many a line has.  Bound
// by memory traffic; U loads in flight a thread keep it streaming.
struct Walk {
  uint32_t chunks, cpr;
  FastDiv div;  // by cpr
};
template <int U, class F>
SKG_DEV void walk_chunks(const Walk& w, F&& f) {
  static_for<0, U>([&](auto u_) {
    constexpr int u = decltype(u_)::value;
    const uint32_t g = (blockIdx.x * U + u) * 256 + threadIdx.x;
    const uint32_t at = g < w.chunks ? g : w.chunks - 1;
    const uint32_t line = fdiv(at, w.div);
    f(u_, g < w.chunks, (int64_t)line, (int)(at - line * w.cpr));
  });
}

template <int DT, bool F4, int U, int TAIL>
SKG_DEV void mx_quant_chunks(const MxParams& p, const Walk& w) {
  typedef typename Elem<DT>::raw raw;
  Chunk<DT> in[U];
  walk_chunks<U>(w, [&](auto u, bool, int64_t row, int c) {
    if (TAIL < 2 || p.cols > 0)
      in[u] = load_within<DT, TAIL>(reinterpret_cast<const raw*>(p.x) + row * p.ldx, c * 8, (int)p.cols);
    else
      in[u] = Chunk<DT>{};
  });
  walk_chunks<U>(w, [&](auto u, bool live, int64_t row, int c) {
    place_chunk<DT, TAIL>(in[u], c * 8, (int)p.cols);
    float v[8];
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = in[u].get(j);
      top = OpMaxBits::op(top, abs_bits(v[j]));
    }
    const uint32_t code = mx_code<F4 ? 2 : 8>(quad_reduce<OpMaxBits>(top));
    const float inv = mx_inverse(code);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = code == 255 ? 0.f : v[j] * inv;
    if (live) {
      if constexpr (F4)
        store_loose(p.q + row * (p.ldq / 2) + (int64_t)c * 4, pack_e2m1(v));
      else
        store_loose(p.q + row * p.ldq + (int64_t)c * 8, pack_e4m3(v));
      if ((c & 3) == 0) p.sc[row * (p.kq / 32) + (c >> 2)] = (uint8_t)code;
    }
  });
}
template <int DT, bool F4, int U>
__global__ __launch_bounds__(256) void mx_quant_kernel(MxParams p, Walk w) {
  // (No columns at all, only padding to write, belongs with less than eight.)
  if (p.cols < 8) return mx_quant_chunks<DT, F4, U, 2>(p, w);
  if (p.cols & 7) return mx_quant_chunks<DT, F4, U, 1>(p, w);
  mx_quant_chunks<DT, F4, U, 0>(p, w);
}

template <int DT, bool F4, int U, bool TAIL>
SKG_DEV void mx_dequant_chunks(const MxParams& p, const Walk& w) {
  typedef typename Elem<DT>::raw raw;
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  uint2 q[U];
  uint32_t sc[U];
  walk_chunks<U>(w, [&](auto u, bool, int64_t row, int c) {
    sc[u] = p.sc[row * (p.kq / 32) + (c >> 2)];
    if constexpr (F4)
      q[u].x = load_loose<uint32_t>(p.q + row * (p.ldq / 2) + (int64_t)c * 4);
    else
      q[u] = load_loose<uint2>(p.q + row * p.ldq + (int64_t)c * 8);
  });
  walk_chunks<U>(w, [&](auto u, bool live, int64_t row, int c) {
    const float d = mx_value(sc[u]);
    f32x2 v[4];
    if constexpr (F4) {
      v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u].x, 1.f, 0);
      v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u].x, 1.f, 1);
      v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u].x, 1.f, 2);
      v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u].x, 1.f, 3);
    } else {
      v[0] = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[u].x, false);
      v[1] = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[u].x, true);
      v[2] = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[u].y, false);
      v[3] = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[u].y, true);
    }
    Chunk<DT> out;
#pragma unroll
    for (int j = 0; j < 8; ++j) out.put(j, v[j >> 1][j & 1] * d);
    const int64_t n = p.cols - (int64_t)c * 8;
    if (live && n > 0)
      store_chunk<DT>(reinterpret_cast<raw*>(const_cast<char*>(p.x)) + row * p.ldx + (int64_t)c * 8,
                      TAIL && n < 8 ? (int)n : 8, out);
  });
}
template <int DT, bool F4, int U>
__global__ __launch_bounds__(256) void mx_dequant_kernel(MxParams p, Walk w) {
  if (p.cols & 7)
    mx_dequant_chunks<DT, F4, U, true>(p, w);
  else
    mx_dequant_chunks<DT, F4, U, false>(p, w);
}

// Along the columns, written transposed: a 128 x 128 tile of x through LDS
// (16384x4096 bf16 to e4m3 45 us; 47 with 64 columns, 60 with 32: shorter
// runs of each row).  A
// thread then takes eight rows of four columns, so that four neighbouring
// lanes hold a block of each of the four and sixteen write 128 codes of a
// line together.  16-bit elements: rows of 136 bytes with groups of four
// columns exchanged in every other 32 rows put the 64 reads of a wave (16
// row groups, 4 column groups) on all banks evenly; fp32's 264 do without.
constexpr int kTRows = 128, kTCols = 128;
template <int DT>
struct TTile {
  static constexpr int TR = kTRows, TC = kTCols, THREADS = TC * 4, ES = sizeof(typename Elem<DT>::raw);
  static constexpr int P = TC * ES + 8, GB = 4 * ES;  // row pitch, group bytes
};
template <int DT, bool F4, int TAIL>
SKG_DEV void mx_quant_t_tile(const MxParams& p, SKG_LDS char* tile) {
  typedef typename Elem<DT>::raw raw;
  typedef TTile<DT> T;
  constexpr int TR = T::TR, TC = T::TC, ES = T::ES, P = T::P, GB = T::GB;
  struct Group {
    raw v[4];
  };
  auto at = [&](int r, int g) { return tile + r * P + (ES == 2 ? g ^ ((r >> 5 & 1) << 2) : g) * GB; };
  // Tiles of the same rows follow one another, so that x's rows are read
  // through (the other order took 50 us for 42 at 8192x8192 bf16 to e2m1, on
  // tiles of 64 columns).
  const uint32_t id = p.first + blockIdx.x, across = (uint32_t)((p.cols + TC - 1) / TC), down = id / across;
  const int64_t r0 = (int64_t)down * TR, c0 = (int64_t)(id - down * across) * TC;
  constexpr int N = TR * TC / 8 / T::THREADS;
  Chunk<DT> in[N];
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int k = u * T::THREADS + threadIdx.x;
    const int64_t r = min(r0 + k / (TC / 8), p.rows - 1);
    if (p.rows > 0)
      in[u] = load_within<DT, TAIL>(reinterpret_cast<const raw*>(p.x) + r * p.ldx, (int)c0 + k % (TC / 8) * 8, (int)p.cols);
  }
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int k = u * T::THREADS + threadIdx.x, r = k / (TC / 8), g = k % (TC / 8) * 2;
    place_chunk<DT, TAIL>(in[u], (int)c0 + g * 4, (int)p.cols);
    if (r0 + r >= p.rows) in[u] = Chunk<DT>{};
    typedef uint32_t words __attribute__((ext_vector_type(GB / 4), aligned(8)));
    struct Two {
      words w[2];
    };
    const Two two = __builtin_bit_cast(Two, in[u]);
    *(SKG_LDS words*)at(r, g) = two.w[0];
    *(SKG_LDS words*)at(r, g + 1) = two.w[1];
  }
  __syncthreads();
  const int oct = threadIdx.x & 15, grp = threadIdx.x >> 4;
  const int64_t k0 = r0 + oct * 8;
  float v[4][8];
  uint32_t top[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    typedef uint32_t words __attribute__((ext_vector_type(GB / 4), aligned(8)));
    const Group e = __builtin_bit_cast(Group, *(const SKG_LDS words*)at(oct * 8 + i, grp));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j][i] = Elem<DT>::get(e.v[j]);
      top[j] = OpMaxBits::op(top[j], abs_bits(v[j][i]));
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t line = c0 + grp * 4 + j;
    const uint32_t code = mx_code<F4 ? 2 : 8>(quad_reduce<OpMaxBits>(top[j]));
    const float inv = mx_inverse(code);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[j][i] = code == 255 ? 0.f : v[j][i] * inv;
    if (line < p.cols && k0 < p.kq) {
      if constexpr (F4)
        store_loose(p.q + line * (p.ldq / 2) + k0 / 2, pack_e2m1(v[j]));
      else
        store_loose(p.q + line * p.ldq + k0, pack_e4m3(v[j]));
      if ((oct & 3) == 0) p.sc[line * (p.kq / 32) + k0 / 32] = (uint8_t)code;
    }
  }
}

template <int DT, bool F4>
__global__ __launch_bounds__(TTile<DT>::THREADS) void mx_quant_t_kernel(MxParams p) {
  __shared__ __attribute__((aligned(16))) char tile[TTile<DT>::TR * TTile<DT>::P];
  if (!(p.cols & 7)) return mx_quant_t_tile<DT, F4, 0>(p, (SKG_LDS char*)tile);
  if (p.cols >= 8) return mx_quant_t_tile<DT, F4, 1>(p, (SKG_LDS char*)tile);
  mx_quant_t_tile<DT, F4, 2>(p, (SKG_LDS char*)tile);
}

bool row_type(int dt) { return dt == SKG_F16 || dt == SKG_BF16 || dt == SKG_F32; }
bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int run_mx(const skg_mx_args_t* a, bool quant, hipStream_t st) {
  if (!a) return unsupported("null arguments");
  if (!row_type(a->dtype)) return unsupported("MX elements come from and go to f16, bf16 or f32");
  if (a->dtype_q != SKG_F8E4M3 && a->dtype_q != SKG_F4E2M1) return unsupported("MX codes are e4m3 or e2m1");
  const bool f4 = a->dtype_q == SKG_F4E2M1;
  if (a->rows < 0 || a->cols < 0) return unsupported("rows and cols must not be negative");
  if (!quant && a->transpose) return unsupported("reading back does not transpose");
  const int64_t axis = a->transpose ? a->rows : a->cols, lines = a->transpose ? a->cols : a->rows;
  if (a->kq < axis || a->kq % 32) return unsupported("kq must be a multiple of 32 and cover the quantised axis");
  if (a->ldx < a->cols || a->ldq < a->kq) return unsupported("leading dimension too small");
  if (f4 && a->ldq % 2) return unsupported("ldq of e2m1 codes must be even");
  const int64_t most = INT32_MAX - 4096;  // rounded up to tiles within 32 bits
  if (a->rows > most || a->cols > most || a->kq > most) return unsupported("dimension too large");
  if (lines == 0 || a->kq == 0) return SKG_OK;
  const bool reads = quant ? axis > 0 : true;
  if ((!a->x && reads && a->cols > 0) || !a->q || !a->scales) return unsupported("null x, q or scales");
  if (!aligned_to(a->x, elem_bytes(a->dtype))) return unsupported("pointers must be aligned to their elements");
  int cus = 0;
  int rc = check_device(&cus);
  if (rc) return rc;
  MxParams p;
  p.x = static_cast<const char*>(a->x);
  p.q = static_cast<char*>(a->q);
  p.sc = static_cast<uint8_t*>(a->scales);
  p.rows = a->rows;
  p.cols = a->cols;
  p.kq = a->kq;
  p.ldx = a->ldx;
  p.ldq = a->ldq;
  p.first = 0;
  auto by_type = [&](auto launch) {
    auto by_fmt = [&](auto dt) {
      if (f4)
        launch(dt, std::integral_constant<bool, true>{});
      else
        launch(dt, std::integral_constant<bool, false>{});
    };
    if (a->dtype == SKG_F16)
      by_fmt(std::integral_constant<int, DT_F16>{});
    else if (a->dtype == SKG_BF16)
      by_fmt(std::integral_constant<int, DT_BF16>{});
    else
      by_fmt(std::integral_constant<int, DT_F32>{});
  };
  if (a->transpose) {
    const int64_t tiles = ceil_div(a->kq, kTRows) * ceil_div(a->cols, kTCols);
    if (tiles > INT32_MAX) return unsupported("too many tiles to transpose");
    // Tiles in launches of fewer than 2^32 threads.
    by_type([&](auto dt, auto f4_) {
      constexpr int DT = decltype(dt)::value, THREADS = TTile<DT>::THREADS;
      constexpr int64_t most = kMostThreads / THREADS;
      for (int64_t t0 = 0; t0 < tiles; t0 += most) {
        MxParams q = p;
        q.first = (uint32_t)t0;
        hipLaunchKernelGGL((mx_quant_t_kernel<DT, decltype(f4_)::value>), dim3((unsigned)std::min(most, tiles - t0)),
                           dim3(THREADS), 0, st, q);
      }
    });
  } else {
    Walk w;
    w.cpr = (uint32_t)(a->kq / 8);
    w.div = make_fastdiv(w.cpr);
    // Lines in launches of fewer than 2^31 chunks.
    const int64_t most = std::max<int64_t>(1, (INT32_MAX - 4095) / w.cpr);
    for (int64_t r0 = 0; r0 < a->rows; r0 += most) {
      const int64_t n = std::min<int64_t>(most, a->rows - r0);
      w.chunks = (uint32_t)(n * w.cpr);
      MxParams q = p;
      q.rows = n;
      q.x += r0 * a->ldx * elem_bytes(a->dtype);
      q.q += row_bytes(a->dtype_q, r0 * a->ldq);
      q.sc += r0 * (a->kq / 32);
      // Many chunks: four a thread (8192x8192 bf16 to e2m1 33 us, 5.2 TB/s,
      // and back 32).  Few: one, for the sake of more workgroups.
      const int u = w.chunks >= (1u << 20) ? 4 : 1;
      const dim3 grid((unsigned)ceil_div(w.chunks, 256 * u));
      by_type([&](auto dt, auto f4_) {
        constexpr int DT = decltype(dt)::value;
        constexpr bool F4 = decltype(f4_)::value;
        if (quant && u == 4)
          hipLaunchKernelGGL((mx_quant_kernel<DT, F4, 4>), grid, dim3(256), 0, st, q, w);
        else if (quant)
          hipLaunchKernelGGL((mx_quant_kernel<DT, F4, 1>), grid, dim3(256), 0, st, q, w);
        else if (u == 4)
          hipLaunchKernelGGL((mx_dequant_kernel<DT, F4, 4>), grid, dim3(256), 0, st, q, w);
        else
          hipLaunchKernelGGL((mx_dequant_kernel<DT, F4, 1>), grid, dim3(256), 0, st, q, w);
      });
    }
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return hip_failure(std::string("launch: ") + hipGetErrorString(e));
  return SKG_OK;
}

int run_mx_guarded(const skg_mx_args_t* a, bool quant, void* stream) {
  try {
    clear_error();
    return run_mx(a, quant, static_cast<hipStream_t>(stream));
  } catch (const std::exception& ex) {
    return hip_failure(std::string("exception: ") + ex.what());
  } catch (...) {
    return hip_failure("unknown exception");
  }
}

}  // namespace
}  // namespace skg

extern "C" {
int skg_run_mx_quant(const skg_mx_args_t* a, void* stream) { return skg::run_mx_guarded(a, true, stream); }
int skg_run_mx_dequant(const skg_mx_args_t* a, void* stream) { return skg::run_mx_guarded(a, false, stream); }
}  // extern "C"
