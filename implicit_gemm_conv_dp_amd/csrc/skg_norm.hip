// Root-mean-square norm with the residual's addition and quantised outputs,
// and its gradient.
//
// Forward, one row of C columns:
//   h = round(x + r)            (the row's type; what is stored and normed)
//   s = 1 / sqrt(mean(h^2) + eps)                       (fp32)
//   y = h * s * w, written in the row's type, as e4m3 codes with one fp32
//   scale d = max(max|y| / 448, 2^-126) a row, or as MX blocks of e4m3 / e2m1.
// Backward, g = dy * w:
//   dx = s * (g - h * s^2 * mean(g h)) + dres,   dw = sum over rows dy * h * s.
//
// Both read every operand once and keep the row in registers between the
// reductions, so they are bound by memory traffic, or for a few rows by the
// latency of one load, one or two reductions and one store.
#include <exception>
#include <string>

#include "skg_internal.hpp"
#include "skg_lowp.hpp"

namespace skg {
namespace {

enum { OUT_SAME = 0, OUT_E4M3_ROW = 1, OUT_E4M3_MX = 2, OUT_E2M1_MX = 3 };

struct NormParams {
  const char *x, *r, *w;
  char *h, *y;
  void* scale;
  float* rstd;
  int rows, cols, w_f32;
  int64_t ldx, ldr, ldh, ldy;  // elements
  float eps, inv_cols;
};

// Weight elements of a chunk, as fp32 (1 without a weight).
template <int DT>
SKG_DEV void load_weight(float (&w)[8], const char* p, int w_f32, int e0, int n) {
  if (!p) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 1.f;
  } else if (DT == DT_F32 || w_f32) {
    const Chunk<DT_F32> c = load_chunk<DT_F32>(reinterpret_cast<const uint32_t*>(p) + e0, n);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = c.get(j);
  } else {
    const Chunk<DT> c = load_chunk<DT>(reinterpret_cast<const typename Elem<DT>::raw*>(p) + e0, n);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = c.get(j);
  }
}

// 1 / sqrt(v) within half an ulp or so: the hardware's reciprocal square
// root and one Newton step.  0 for an infinite v, NaN for a NaN.
SKG_DEV float rsqrt_refined(float v) {
  const float r = __builtin_amdgcn_rsqf(v);
  const float e = __builtin_fmaf(-v * r, r, 1.f);
  const float n = __builtin_fmaf(0.5f * r, e, r);
  return r > 0.f && v < 3e38f ? n : r;
}

// One row by a group of 64 * WAVES threads, NCH chunks of eight columns
// each.  TAIL: the columns are not a multiple of eight.
template <int DT, int OUT, int WAVES, int NCH, bool TAIL>
SKG_DEV void norm_row(const NormParams& p, int row, int t, SKG_LDS uint32_t* slots) {
  typedef typename Elem<DT>::raw raw;
  constexpr int G = 64 * WAVES;
  const raw* x = reinterpret_cast<const raw*>(p.x) + row * p.ldx;
  Chunk<DT> hx[NCH];
  auto left = [&](int i) {
    const int n = p.cols - (t + i * G) * 8;
    return TAIL ? n : n > 0 ? 8 : 0;
  };
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    if (left(i) > 0)
      hx[i] = load_chunk<DT>(x + (t + i * G) * 8, left(i));
    else
      hx[i] = Chunk<DT>{};
  }
  if (p.r) {
    const raw* r = reinterpret_cast<const raw*>(p.r) + row * p.ldr;
    Chunk<DT> hr[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      if (left(i) > 0)
        hr[i] = load_chunk<DT>(r + (t + i * G) * 8, left(i));
      else
        hr[i] = Chunk<DT>{};
    }
#pragma unroll
    for (int i = 0; i < NCH; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) hx[i].put(j, hx[i].get(j) + hr[i].get(j));
  }
  if (p.h) {
    raw* h = reinterpret_cast<raw*>(p.h) + row * p.ldh;
#pragma unroll
    for (int i = 0; i < NCH; ++i)
      if (left(i) > 0) store_chunk<DT>(h + (t + i * G) * 8, left(i), hx[i]);
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    float part = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) part = __builtin_fmaf(hx[i].get(j), hx[i].get(j), part);
    sum += part;
  }
  sum = group_reduce<OpSum, WAVES>(sum, slots);
  const float s = rsqrt_refined(sum * p.inv_cols + p.eps);
  if (p.rstd && t == 0) p.rstd[row] = s;

  if constexpr (OUT == OUT_SAME) {
    raw* y = reinterpret_cast<raw*>(p.y) + row * p.ldy;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      if (left(i) > 0) {
        float w[8];
        load_weight<DT>(w, p.w, p.w_f32, (t + i * G) * 8, left(i));
        Chunk<DT> c;
#pragma unroll
        for (int j = 0; j < 8; ++j) c.put(j, hx[i].get(j) * s * w[j]);
        store_chunk<DT>(y + (t + i * G) * 8, left(i), c);
      }
    }
  } else if constexpr (OUT == OUT_E4M3_ROW) {
    // y / d = h w 448 / max|h w|: the row's factor s cancels, and for
    // 16-bit inputs h w and h w 448 are exact in fp32.  The quotient is
    // rounded correctly (a reciprocal, then one residual step), so values
    // that lie on a border between two codes, which 16-bit inputs often
    // do, round to even and not by the noise of a scaled product.
    float v[NCH][8];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      float w[8];
      if (left(i) > 0) {
        load_weight<DT>(w, p.w, p.w_f32, (t + i * G) * 8, left(i));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] = hx[i].get(j) * w[j];
        const uint32_t b = abs_bits(v[i][j]);
        if (!TAIL || j < left(i)) top = OpMaxBits::op(top, b);
      }
    }
    top = group_reduce<OpMaxBits, WAVES>(top, slots + WAVES);
    const float m = from_bits(top);
    float d = m * s / 448.f;
    // Rows of ordinary size; the others (empty rows, infinities, NaN, and
    // magnitudes whose products leave the range of fp32) take the
    // definition step by step.
    const bool usual = m > 0x1p-100f && m < 0x1p+100f && d >= 0x1p-126f;
    if (usual) {
      const float rcp = 1.f / m;
#pragma unroll
      for (int i = 0; i < NCH; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float num = v[i][j] * 448.f, q = num * rcp;
          v[i][j] = __builtin_fmaf(__builtin_fmaf(-q, m, num), rcp, q);
        }
    } else {
      uint32_t ty = 0;
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        float w[8] = {};
        if (left(i) > 0) load_weight<DT>(w, p.w, p.w_f32, (t + i * G) * 8, left(i));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[i][j] = left(i) > 0 ? hx[i].get(j) * s * w[j] : 0.f;
          if (!TAIL || j < left(i)) ty = OpMaxBits::op(ty, abs_bits(v[i][j]));
        }
      }
      ty = group_reduce<OpMaxBits, WAVES>(ty, slots + 2 * WAVES);
      d = from_bits(ty) / 448.f;
      if (d < 0x1p-126f) d = 0x1p-126f;  // a NaN stays
#pragma unroll
      for (int i = 0; i < NCH; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] / d;
    }
    if (t == 0) reinterpret_cast<float*>(p.scale)[row] = d;
    uint8_t* y = reinterpret_cast<uint8_t*>(p.y) + row * p.ldy;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      if (left(i) > 0) {
        const uint2 q = pack_e4m3_nan(v[i]);
        uint8_t* o = y + (t + i * G) * 8;
        if (left(i) >= 8) {
          store_loose(o, q);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < left(i)) o[j] = (uint8_t)((j < 4 ? q.x : q.y) >> (8 * (j & 3)));
        }
      }
    }
  } else {
    // MX: four neighbouring lanes hold a block.
    constexpr bool F4 = OUT == OUT_E2M1_MX;
    char* y = p.y + row * (F4 ? p.ldy / 2 : p.ldy);
    uint8_t* sc = reinterpret_cast<uint8_t*>(p.scale) + (int64_t)row * (p.cols / 32);
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = t + i * G;
      float w[8], v[8];
      uint32_t top = 0;
      if (left(i) > 0) load_weight<DT>(w, p.w, p.w_f32, c * 8, 8);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = left(i) > 0 ? hx[i].get(j) * s * w[j] : 0.f;
        top = OpMaxBits::op(top, abs_bits(v[j]));
      }
      const uint32_t code = mx_code<F4 ? 2 : 8>(quad_reduce<OpMaxBits>(top));
      const float inv = mx_inverse(code);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = code == 255 ? 0.f : v[j] * inv;
      if (left(i) > 0) {
        if constexpr (F4)
          store_loose(y + c * 4, pack_e2m1(v));
        else
          store_loose(y + c * 8, pack_e4m3(v));
        if ((c & 3) == 0) sc[c >> 2] = (uint8_t)code;
      }
    }
  }
}

template <int DT, int OUT, int WAVES, int NCH>
__global__ __launch_bounds__(WAVES == 1 ? 256 : 64 * WAVES) void rmsnorm_kernel(NormParams p) {
  __shared__ uint32_t slots_[3 * WAVES];
  SKG_LDS uint32_t* slots = (SKG_LDS uint32_t*)slots_;
  const int row = WAVES == 1 ? blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  const int t = WAVES == 1 ? threadIdx.x & 63 : threadIdx.x;
  if (row >= p.rows) return;  // whole waves, which meet no barrier (WAVES is 1)
  if (p.cols & 7)
    norm_row<DT, OUT, WAVES, NCH, true>(p, row, t, slots);
  else
    norm_row<DT, OUT, WAVES, NCH, false>(p, row, t, slots);
}

// --- backward ------------------------------------------------------------------
struct NormBwdParams {
  const char *dy, *h, *w, *dres;
  const float* rstd;
  char* dx;
  float* partial;  // [groups][cols], or nullptr without dw
  int rows, cols, w_f32, groups;
  int64_t lddy, ldh, ldr, lddx;
  float inv_cols;
};

// A group of 64 * WAVES threads takes rows g, g + groups, ...; each thread
// keeps the sums of dw of its columns.
template <int DT, int WAVES, int NCH, bool TAIL>
SKG_DEV void norm_bwd_rows(const NormBwdParams& p, int g, int t, SKG_LDS uint32_t* slots) {
  typedef typename Elem<DT>::raw raw;
  constexpr int G = 64 * WAVES;
  auto left = [&](int i) {
    const int n = p.cols - (t + i * G) * 8;
    return TAIL ? n : n > 0 ? 8 : 0;
  };
  float w[NCH][8], dw[NCH][8];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = w[i][j] = 0.f;
    if (left(i) > 0) load_weight<DT>(w[i], p.w, p.w_f32, (t + i * G) * 8, left(i));
  }
  int flip = 0;
  for (int row = g; row < p.rows; row += p.groups, flip ^= WAVES) {
    const raw* dyp = reinterpret_cast<const raw*>(p.dy) + row * p.lddy;
    const raw* hp = reinterpret_cast<const raw*>(p.h) + row * p.ldh;
    const raw* rp = reinterpret_cast<const raw*>(p.dres) + (p.dres ? row * p.ldr : 0);
    Chunk<DT> dy[NCH], h[NCH], r[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      dy[i] = h[i] = r[i] = Chunk<DT>{};
      if (left(i) > 0) {
        dy[i] = load_chunk<DT>(dyp + (t + i * G) * 8, left(i));
        h[i] = load_chunk<DT>(hp + (t + i * G) * 8, left(i));
        if (p.dres) r[i] = load_chunk<DT>(rp + (t + i * G) * 8, left(i));
      }
    }
    const float s = p.rstd[row];
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      float part = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = h[i].get(j) * s;
        part = __builtin_fmaf(dy[i].get(j) * w[i][j], n, part);
        dw[i][j] = __builtin_fmaf(dy[i].get(j), n, dw[i][j]);
      }
      dot += part;
    }
    // Two sets of slots in turn: one barrier a row.
    dot = group_reduce<OpSum, WAVES>(dot, slots + flip) * p.inv_cols;
    if (p.dx) {
      raw* dx = reinterpret_cast<raw*>(p.dx) + row * p.lddx;
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        if (left(i) > 0) {
          Chunk<DT> c;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float n = h[i].get(j) * s;
            const float v = s * __builtin_fmaf(-n, dot, dy[i].get(j) * w[i][j]);
            c.put(j, p.dres ? v + r[i].get(j) : v);
          }
          store_chunk<DT>(dx + (t + i * G) * 8, left(i), c);
        }
      }
    }
  }
  if (p.partial) {
    float* o = p.partial + (int64_t)g * p.cols;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      if (left(i) > 0) {
        Chunk<DT_F32> c;
#pragma unroll
        for (int j = 0; j < 8; ++j) c.put(j, dw[i][j]);
        store_chunk<DT_F32>(reinterpret_cast<uint32_t*>(o) + (t + i * G) * 8, left(i), c);
      }
    }
  }
}

template <int DT, int WAVES, int NCH>
__global__ __launch_bounds__(WAVES == 1 ? 256 : 64 * WAVES) void rmsnorm_bwd_kernel(NormBwdParams p) {
  __shared__ uint32_t slots_[2 * WAVES];
  SKG_LDS uint32_t* slots = (SKG_LDS uint32_t*)slots_;
  const int g = WAVES == 1 ? blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  const int t = WAVES == 1 ? threadIdx.x & 63 : threadIdx.x;
  if (g >= p.groups) return;  // whole waves, which meet no barrier (WAVES is 1)
  if (p.cols & 7)
    norm_bwd_rows<DT, WAVES, NCH, true>(p, g, t, slots);
  else
    norm_bwd_rows<DT, WAVES, NCH, false>(p, g, t, slots);
}

// dw[c] = sum over the groups of partial[g][c], in a fixed order: 64 columns
// by 4 runs of groups a workgroup, then the four runs.  Without groups (no
// rows) it writes zeros.
__global__ __launch_bounds__(256) void norm_dw_kernel(const float* __restrict__ partial, float* __restrict__ dw, int groups, int cols) {
  __shared__ float part[4][64];
  const int lane = threadIdx.x & 63, run = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  float sum = 0.f;
  if (c < cols)
    for (int g = run; g < groups; g += 4) sum += partial[(int64_t)g * cols + c];
  part[run][lane] = sum;
  __syncthreads();
  if (run == 0 && c < cols) dw[c] = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
}

// --- host ------------------------------------------------------------------------

// How a row is spread: waves a row and chunks a thread, the first of the
// list that holds the row.
struct Spread {
  int waves, nch;
};
constexpr Spread kSpreads[] = {{1, 1}, {1, 2}, {1, 4}, {4, 2}, {4, 4}, {16, 2}, {16, 4}};
constexpr int kSpreadCount = sizeof(kSpreads) / sizeof(kSpreads[0]);
int spread_of(int64_t cols) {
  for (int i = 0; i < kSpreadCount; ++i)
    if (cols <= int64_t(kSpreads[i].waves) * kSpreads[i].nch * 512) return i;
  return -1;
}

template <int DT, int OUT, int I = 0>
void launch_norm(const NormParams& p, int spread, hipStream_t st) {
  if constexpr (I < kSpreadCount) {
    if (spread == I) {
      constexpr int W = kSpreads[I].waves, N = kSpreads[I].nch;
      const unsigned grid = W == 1 ? (unsigned)((p.rows + 3) / 4) : (unsigned)p.rows;
      hipLaunchKernelGGL((rmsnorm_kernel<DT, OUT, W, N>), dim3(grid), dim3(W == 1 ? 256 : 64 * W), 0, st, p);
    } else {
      launch_norm<DT, OUT, I + 1>(p, spread, st);
    }
  }
}
template <int DT>
void launch_norm(const NormParams& p, int out, int spread, hipStream_t st) {
  switch (out) {
    case OUT_SAME: return launch_norm<DT, OUT_SAME>(p, spread, st);
    case OUT_E4M3_ROW: return launch_norm<DT, OUT_E4M3_ROW>(p, spread, st);
    case OUT_E4M3_MX: return launch_norm<DT, OUT_E4M3_MX>(p, spread, st);
    default: return launch_norm<DT, OUT_E2M1_MX>(p, spread, st);
  }
}
template <int DT, int I = 0>
void launch_norm_bwd(const NormBwdParams& p, int spread, hipStream_t st) {
  if constexpr (I < kSpreadCount) {
    if (spread == I) {
      constexpr int W = kSpreads[I].waves, N = kSpreads[I].nch;
      const unsigned grid = W == 1 ? (unsigned)((p.groups + 3) / 4) : (unsigned)p.groups;
      hipLaunchKernelGGL((rmsnorm_bwd_kernel<DT, W, N>), dim3(grid), dim3(W == 1 ? 256 : 64 * W), 0, st, p);
    } else {
      launch_norm_bwd<DT, I + 1>(p, spread, st);
    }
  }
}

bool row_type(int dt) { return dt == SKG_F16 || dt == SKG_BF16 || dt == SKG_F32; }
bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int check_norm(const skg_norm_args_t* a) {
  if (!a) return unsupported("null arguments");
  if (!row_type(a->dtype)) return unsupported("the norm's rows are f16, bf16 or f32");
  if (a->dtype_w != a->dtype && a->dtype_w != SKG_F32) return unsupported("the weight has the rows' type or f32");
  const bool same = a->dtype_y == a->dtype;
  const bool f8 = a->dtype_y == SKG_F8E4M3, f4 = a->dtype_y == SKG_F4E2M1;
  if (!same && !f8 && !f4) return unsupported("the norm's output has the rows' type, e4m3 or e2m1");
  const bool mx = a->scale_mode == SKG_SCALE_MX_E8M0;
  if (!same && !mx && a->scale_mode != SKG_SCALE_ROWCOL) return unsupported("the norm's scales are one a row or MX blocks");
  if (f4 && !mx) return unsupported("e2m1 output needs MX block scales");
  if (a->rows < 0 || a->cols <= 0) return unsupported("rows must not be negative and cols must be positive");
  if (a->rows > INT32_MAX) return unsupported("too many rows");
  if (a->cols > SKG_NORM_MAX_COLS) return unsupported("rows longer than SKG_NORM_MAX_COLS");
  if (!same && mx && a->cols % 32) return unsupported("MX output needs cols to be a multiple of 32");
  if (a->ldx < a->cols || (a->residual && a->ldr < a->cols) || (a->h && a->ldh < a->cols) || a->ldy < a->cols)
    return unsupported("leading dimension too small");
  if (f4 && a->ldy % 2) return unsupported("ldy of e2m1 codes must be even");
  if (!(a->eps >= 0.f)) return unsupported("eps must not be negative");
  return SKG_OK;
}

int run_norm(const skg_norm_args_t* a, hipStream_t st) {
  int rc = check_norm(a);
  if (rc) return rc;
  const bool same = a->dtype_y == a->dtype;
  if (a->rows == 0) return SKG_OK;
  if (!a->x || !a->y) return unsupported("null x or y");
  if (!same && !a->y_scale) return unsupported("a quantised output needs its scales");
  const size_t es = elem_bytes(a->dtype);
  if (!aligned_to(a->x, es) || !aligned_to(a->residual, es) || !aligned_to(a->h, es) || !aligned_to(a->weight, elem_bytes(a->dtype_w)) ||
      !aligned_to(a->rstd, 4) || (same && !aligned_to(a->y, es)) ||
      (!same && a->scale_mode == SKG_SCALE_ROWCOL && !aligned_to(a->y_scale, 4)))
    return unsupported("pointers must be aligned to their elements");
  int cus = 0;
  rc = check_device(&cus);
  if (rc) return rc;
  NormParams p;
  p.x = static_cast<const char*>(a->x);
  p.r = static_cast<const char*>(a->residual);
  p.w = static_cast<const char*>(a->weight);
  p.h = static_cast<char*>(a->h);
  p.y = static_cast<char*>(a->y);
  p.scale = a->y_scale;
  p.rstd = a->rstd;
  p.rows = (int)a->rows;
  p.cols = (int)a->cols;
  p.w_f32 = a->dtype_w == SKG_F32;
  p.ldx = a->ldx;
  p.ldr = a->ldr;
  p.ldh = a->ldh;
  p.ldy = a->ldy;
  p.eps = a->eps;
  p.inv_cols = 1.f / (float)a->cols;
  const int out = same ? OUT_SAME : a->dtype_y == SKG_F4E2M1 ? OUT_E2M1_MX : a->scale_mode == SKG_SCALE_MX_E8M0 ? OUT_E4M3_MX : OUT_E4M3_ROW;
  const int spread = spread_of(a->cols);
  if (a->dtype == SKG_F16)
    launch_norm<DT_F16>(p, out, spread, st);
  else if (a->dtype == SKG_BF16)
    launch_norm<DT_BF16>(p, out, spread, st);
  else
    launch_norm<DT_F32>(p, out, spread, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return hip_failure(std::string("launch: ") + hipGetErrorString(e));
  return SKG_OK;
}

int check_norm_bwd(const skg_norm_bwd_args_t* a) {
  if (!a) return unsupported("null arguments");
  if (!row_type(a->dtype)) return unsupported("the norm's rows are f16, bf16 or f32");
  if (a->dtype_w != a->dtype && a->dtype_w != SKG_F32) return unsupported("the weight has the rows' type or f32");
  if (a->rows < 0 || a->cols <= 0) return unsupported("rows must not be negative and cols must be positive");
  if (a->rows > INT32_MAX) return unsupported("too many rows");
  if (a->cols > SKG_NORM_MAX_COLS) return unsupported("rows longer than SKG_NORM_MAX_COLS");
  if (a->lddy < a->cols || a->ldh < a->cols || (a->dres && a->lddres < a->cols) || (a->dx && a->lddx < a->cols))
    return unsupported("leading dimension too small");
  return SKG_OK;
}

// Groups of rows, each with one row of partial dw sums.
int bwd_groups(const skg_norm_bwd_args_t* a) {
  const int64_t most = kSpreads[spread_of(a->cols)].waves == 1 ? 2048 : 512;
  return (int)(a->rows < most ? a->rows : most);
}

int run_norm_bwd(const skg_norm_bwd_args_t* a, void* ws, size_t ws_bytes, hipStream_t st) {
  int rc = check_norm_bwd(a);
  if (rc) return rc;
  if (a->rows > 0 && (!a->dy || !a->h || !a->rstd)) return unsupported("null dy, h or rstd");
  if (!a->dx && !a->dw) return unsupported("neither dx nor dw is asked for");
  const size_t es = elem_bytes(a->dtype);
  if (!aligned_to(a->dy, es) || !aligned_to(a->h, es) || !aligned_to(a->dres, es) || !aligned_to(a->dx, es) ||
      !aligned_to(a->weight, elem_bytes(a->dtype_w)) || !aligned_to(a->rstd, 4) || !aligned_to(a->dw, 4))
    return unsupported("pointers must be aligned to their elements");
  const int groups = bwd_groups(a);
  const size_t need = a->dw ? size_t(groups) * a->cols * 4 : 0;
  if (need > ws_bytes) return unsupported("workspace too small for this call");
  if (need && (!ws || !aligned_to(ws, 16))) return unsupported("workspace must be 16-byte aligned device memory");
  int cus = 0;
  rc = check_device(&cus);
  if (rc) return rc;
  hipError_t e = hipSuccess;
  if (a->rows > 0) {
    NormBwdParams p;
    p.dy = static_cast<const char*>(a->dy);
    p.h = static_cast<const char*>(a->h);
    p.w = static_cast<const char*>(a->weight);
    p.dres = static_cast<const char*>(a->dres);
    p.rstd = a->rstd;
    p.dx = static_cast<char*>(a->dx);
    p.partial = a->dw ? static_cast<float*>(ws) : nullptr;
    p.rows = (int)a->rows;
    p.cols = (int)a->cols;
    p.w_f32 = a->dtype_w == SKG_F32;
    p.groups = groups;
    p.lddy = a->lddy;
    p.ldh = a->ldh;
    p.ldr = a->lddres;
    p.lddx = a->lddx;
    p.inv_cols = 1.f / (float)a->cols;
    const int spread = spread_of(a->cols);
    if (a->dtype == SKG_F16)
      launch_norm_bwd<DT_F16>(p, spread, st);
    else if (a->dtype == SKG_BF16)
      launch_norm_bwd<DT_BF16>(p, spread, st);
    else
      launch_norm_bwd<DT_F32>(p, spread, st);
    e = hipGetLastError();
    if (e != hipSuccess) return hip_failure(std::string("launch: ") + hipGetErrorString(e));
  }
  if (a->dw) {
    hipLaunchKernelGGL(norm_dw_kernel, dim3((unsigned)ceil_div(a->cols, 64)), dim3(256), 0, st,
                       static_cast<const float*>(ws), a->dw, groups, (int)a->cols);
    e = hipGetLastError();
    if (e != hipSuccess) return hip_failure(std::string("launch: ") + hipGetErrorString(e));
  }
  return SKG_OK;
}

}  // namespace
}  // namespace skg

using namespace skg;

extern "C" {

int skg_run_rmsnorm(const skg_norm_args_t* a, void* stream) {
  try {
    clear_error();
    return run_norm(a, static_cast<hipStream_t>(stream));
  } catch (const std::exception& ex) {
    return hip_failure(std::string("exception: ") + ex.what());
  } catch (...) {
    return hip_failure("unknown exception");
  }
}

int skg_rmsnorm_bwd_workspace_bytes(const skg_norm_bwd_args_t* a, size_t* out) {
  try {
    clear_error();
    const int rc = check_norm_bwd(a);
    if (rc) return rc;
    if (!out) return unsupported("null output");
    *out = a->dw ? size_t(bwd_groups(a)) * a->cols * 4 : 0;
    return SKG_OK;
  } catch (...) {
    return hip_failure("exception in skg_rmsnorm_bwd_workspace_bytes");
  }
}

int skg_run_rmsnorm_bwd(const skg_norm_bwd_args_t* a, void* ws, size_t ws_bytes, void* stream) {
  try {
    clear_error();
    return run_norm_bwd(a, ws, ws_bytes, static_cast<hipStream_t>(stream));
  } catch (const std::exception& ex) {
    return hip_failure(std::string("exception: ") + ex.what());
  } catch (...) {
    return hip_failure("unknown exception");
  }
}

}  // extern "C"
