// MX quantisation along the rows or, transposed, along the columns, and
// reading back.
//
// A block is 32 consecutive elements of the quantised axis.  With top the
// largest magnitude of the block and E its fp32 exponent field, the block's
// E8M0 code is max(E - emax, 0) (emax 2 for e2m1, 8 for e4m3) and its elements
// are round-to-nearest-even, saturating, of x / 2^(code - 127).  Dividing by a
// power of two is exact, so each element is rounded once.  A block that
// holds an infinity or a NaN gets code 255 (NaN) and zero elements.
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
};

// Along the rows: a chunk of eight elements a thread, four neighbouring
// lanes a block.  Bound by memory traffic.
template <int DT, bool F4>
__global__ __launch_bounds__(256) void mx_quant_kernel(MxParams p, int64_t chunks, uint32_t cpr) {
  typedef typename Elem<DT>::raw raw;
  // Whole quads of chunks: cpr is a multiple of four.
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t g0 = (int64_t)blockIdx.x * 256; g0 < chunks; g0 += step) {
    const int64_t g = g0 + threadIdx.x;
    const bool live = g < chunks;
    const int64_t row = live ? g / cpr : 0;
    const int c = (int)(g - row * cpr);
    float v[8];
    uint32_t top = 0;
    Chunk<DT> in = Chunk<DT>{};
    const int64_t n = p.cols - (int64_t)c * 8;
    if (live && n > 0) in = load_chunk<DT>(reinterpret_cast<const raw*>(p.x) + row * p.ldx + (int64_t)c * 8, n < 8 ? (int)n : 8);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = in.get(j);
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
  }
}

// Along the columns, written transposed: a 128 x 64 tile of x through LDS;
// thread (column, block) then holds one whole block.
template <int DT, bool F4>
__global__ __launch_bounds__(256) void mx_quant_t_kernel(MxParams p) {
  typedef typename Elem<DT>::raw raw;
  constexpr int TR = 128, TC = 64, PITCH = TC + 8;
  __shared__ __attribute__((aligned(16))) raw tile[TR * PITCH];
  const int64_t r0 = (int64_t)blockIdx.x * TR, c0 = (int64_t)blockIdx.y * TC;
#pragma unroll
  for (int u = 0; u < TR * TC / 8 / 256; ++u) {
    const int k = u * 256 + threadIdx.x, r = k / (TC / 8), c = k % (TC / 8) * 8;
    Chunk<DT> in = Chunk<DT>{};
    const int64_t n = p.cols - (c0 + c);
    if (r0 + r < p.rows && n > 0)
      in = load_chunk<DT>(reinterpret_cast<const raw*>(p.x) + (r0 + r) * p.ldx + c0 + c, n < 8 ? (int)n : 8);
    *reinterpret_cast<Chunk<DT>*>(&tile[r * PITCH + c]) = in;
  }
  __syncthreads();
  const int col = threadIdx.x >> 2, blk = threadIdx.x & 3;
  const int64_t k0 = r0 + blk * 32;
  if (c0 + col >= p.cols || k0 >= p.kq) return;
  float v[32];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    v[i] = Elem<DT>::get(tile[(blk * 32 + i) * PITCH + col]);
    top = OpMaxBits::op(top, abs_bits(v[i]));
  }
  const uint32_t code = mx_code<F4 ? 2 : 8>(top);
  const float inv = mx_inverse(code);
  uint32_t q[F4 ? 4 : 8];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    float e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = code == 255 ? 0.f : v[u * 8 + j] * inv;
    if constexpr (F4) {
      q[u] = pack_e2m1(e);
    } else {
      const uint2 b = pack_e4m3(e);
      q[2 * u] = b.x;
      q[2 * u + 1] = b.y;
    }
  }
  char* o = p.q + (c0 + col) * (F4 ? p.ldq / 2 : p.ldq) + (F4 ? k0 / 2 : k0);
#pragma unroll
  for (int u = 0; u < (F4 ? 1 : 2); ++u) store_loose(o + 16 * u, make_uint4(q[4 * u], q[4 * u + 1], q[4 * u + 2], q[4 * u + 3]));
  p.sc[(c0 + col) * (p.kq / 32) + k0 / 32] = (uint8_t)code;
}

// Reading back: a chunk of eight codes a thread.
template <int DT, bool F4>
__global__ __launch_bounds__(256) void mx_dequant_kernel(MxParams p, int64_t chunks, uint32_t cpr) {
  typedef typename Elem<DT>::raw raw;
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < chunks; g += step) {
    const int64_t row = g / cpr;
    const int c = (int)(g - row * cpr);
    const float d = mx_value(p.sc[row * (p.kq / 32) + (c >> 2)]);
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    f32x2 v[4];
    if constexpr (F4) {
      const uint32_t q = load_loose<uint32_t>(p.q + row * (p.ldq / 2) + (int64_t)c * 4);
      v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 0);
      v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 1);
      v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 2);
      v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 3);
    } else {
      const uint2 q = load_loose<uint2>(p.q + row * p.ldq + (int64_t)c * 8);
      v[0] = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.x, false);
      v[1] = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.x, true);
      v[2] = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.y, false);
      v[3] = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.y, true);
    }
    Chunk<DT> out;
#pragma unroll
    for (int j = 0; j < 8; ++j) out.put(j, v[j >> 1][j & 1] * d);
    const int64_t n = p.cols - (int64_t)c * 8;
    if (n > 0) store_chunk<DT>(reinterpret_cast<raw*>(const_cast<char*>(p.x)) + row * p.ldx + (int64_t)c * 8, n < 8 ? (int)n : 8, out);
  }
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
  if (a->rows > INT32_MAX || a->cols > INT32_MAX || a->kq > INT32_MAX) return unsupported("dimension too large");
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
    const int64_t gx = ceil_div(a->kq, 128), gy = ceil_div(a->cols, 64);
    if (gy > 65535) return unsupported("too many columns to transpose");
    const dim3 grid((unsigned)gx, (unsigned)gy);
    by_type([&](auto dt, auto f4_) {
      hipLaunchKernelGGL((mx_quant_t_kernel<decltype(dt)::value, decltype(f4_)::value>), grid, dim3(256), 0, st, p);
    });
  } else {
    const uint32_t cpr = (uint32_t)(a->kq / 8);
    const int64_t chunks = a->rows * (int64_t)cpr;
    const int64_t blocks = ceil_div(chunks, 256);
    const unsigned grid = (unsigned)(blocks < 65536 ? blocks : 65536);
    by_type([&](auto dt, auto f4_) {
      if (quant)
        hipLaunchKernelGGL((mx_quant_kernel<decltype(dt)::value, decltype(f4_)::value>), dim3(grid), dim3(256), 0, st, p, chunks, cpr);
      else
        hipLaunchKernelGGL((mx_dequant_kernel<decltype(dt)::value, decltype(f4_)::value>), dim3(grid), dim3(256), 0, st, p, chunks, cpr);
    });
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
