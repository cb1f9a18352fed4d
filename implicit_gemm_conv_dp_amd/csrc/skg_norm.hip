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
// latency of one load, one or two reductions and one store.  A large copy
// reaches 5.2 to 5.4 TB/s here, two reads and a write 5.8 to 5.9.  Measured:
// 8192x8192 bf16 with a residual to e4m3 with row scales 81 us (5.8 TB/s), 4864x4096 to bf16
// 31 us (5.1), gradient of 16384x4096 bf16 with a residual 102 us (5.3).
#include <algorithm>
#include <exception>
#include <string>

#include "skg_internal.hpp"
#include "skg_lowp.hpp"

namespace skg {
namespace {

// Most workgroups of the gradient, each with a row of partial sums of dw.
constexpr int kMostGroups = 1024;
// Rows and what they are rounded up to or stepped by stay within 32 bits.
constexpr int64_t kMostRows = INT32_MAX - 65536;

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

// How rows are spread over threads: groups of LANES lanes, or with 64 of
// WAVES waves, each take whole rows, NCH chunks of eight columns a thread.  A
// workgroup of 256 threads holds GROUPS groups of a wave or less.
template <int WAVES_, int LANES_, int NCH_>
struct Spread {
  static constexpr int WAVES = WAVES_, LANES = LANES_, NCH = NCH_;
  static constexpr int SIZE = WAVES * LANES, COLS = SIZE * NCH * 8;
  static constexpr int THREADS = WAVES == 1 ? 256 : 64 * WAVES;
  static constexpr int GROUPS = THREADS / SIZE;
  // Most workgroups of the gradient: 2048 to 4096 waves in flight, and no more
  // rows of partial sums than that takes (16384x4096 bf16: 512 groups 104 us,
  // 1024 113, 256 112; 16384x1111: 1024 47 us, 512 70; 4096x16384: 256 112 us,
  // 128 133).
  static constexpr int MOST = WAVES >= 8 ? 256 : WAVES == 4 ? 512 : 1024;
  static_assert(LANES == 64 || WAVES == 1, "a group of several waves has whole ones");
};

constexpr int kSmallSpread = 64;  // columns of the first spread, the one that rows of less than eight take

// The weights of a thread's columns, as fp32 (1 without a weight).
template <int DT, class S, int TAIL>
SKG_DEV void load_weights(float (&w)[S::NCH][8], const char* p, int w_f32, int t, int cols) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < S::NCH; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) w[i][j] = 1.f;
  } else if (DT == DT_F32 || w_f32) {
    Chunk<DT_F32> c[S::NCH];
#pragma unroll
    for (int i = 0; i < S::NCH; ++i)
      c[i] = load_within<DT_F32, TAIL>(reinterpret_cast<const uint32_t*>(p), (t + i * S::SIZE) * 8, cols);
#pragma unroll
    for (int i = 0; i < S::NCH; ++i) {
      place_chunk<DT_F32, TAIL>(c[i], (t + i * S::SIZE) * 8, cols);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[i][j] = c[i].get(j);
    }
  } else {
    Chunk<DT> c[S::NCH];
#pragma unroll
    for (int i = 0; i < S::NCH; ++i)
      c[i] = load_within<DT, TAIL>(reinterpret_cast<const typename Elem<DT>::raw*>(p), (t + i * S::SIZE) * 8, cols);
#pragma unroll
    for (int i = 0; i < S::NCH; ++i) {
      place_chunk<DT, TAIL>(c[i], (t + i * S::SIZE) * 8, cols);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[i][j] = c[i].get(j);
    }
  }
}
// A thread's chunks of one row.
template <int DT, class S, int TAIL>
SKG_DEV void load_row(Chunk<DT> (&c)[S::NCH], const char* base, int64_t row, int64_t ld, int t, int cols) {
  const typename Elem<DT>::raw* p = reinterpret_cast<const typename Elem<DT>::raw*>(base) + row * ld;
#pragma unroll
  for (int i = 0; i < S::NCH; ++i) c[i] = load_within<DT, TAIL>(p, (t + i * S::SIZE) * 8, cols);
}
template <int DT, class S, int TAIL>
SKG_DEV void place_row(Chunk<DT> (&c)[S::NCH], int t, int cols) {
#pragma unroll
  for (int i = 0; i < S::NCH; ++i) place_chunk<DT, TAIL>(c[i], (t + i * S::SIZE) * 8, cols);
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

// What is done with a row once it is summed and stored: y in its type.
// `slots` are words of LDS that only this row's reductions use.
template <int DT, int OUT, class S, int TAIL>
SKG_DEV void norm_output(const NormParams& p, int row, bool live, int t, float s, const Chunk<DT> (&hx)[S::NCH],
                         const float (&w)[S::NCH][8], SKG_LDS uint32_t* slots) {
  typedef typename Elem<DT>::raw raw;
  constexpr int NCH = S::NCH, G = S::SIZE;
  // Columns of chunk i that exist, if the row does.
  auto left = [&](int i) {
    const int n = p.cols - (t + i * G) * 8;
    return !live ? 0 : TAIL ? n : n > 0 ? 8 : 0;
  };
  if constexpr (OUT == OUT_SAME) {
    raw* y = reinterpret_cast<raw*>(p.y) + row * p.ldy;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      Chunk<DT> c;
#pragma unroll
      for (int j = 0; j < 8; ++j) c.put(j, hx[i].get(j) * s * w[i][j]);
      if (left(i) > 0) store_chunk<DT>(y + (t + i * G) * 8, left(i), c);
    }
  } else if constexpr (OUT == OUT_E4M3_ROW) {
    // y / d = h w 448 / max|h w|: the row's factor s cancels.  For bf16 rows
    // and weights h w 448 is exact in fp32 (with f16 or f32 the products
    // are rounded).  The quotient is rounded to fp32 correctly (a reciprocal,
    // then one residual step) and then to a code, so values exactly between
    // two codes, which bf16 inputs often have (1 in 62 at 8192x8192), go to the
    // even one and not where the noise of a scaled product takes them.
    float v[NCH][8];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NCH; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] = hx[i].get(j) * w[i][j];
        top = OpMaxBits::op(top, abs_bits(v[i][j]));
      }
    top = group_reduce<OpMaxBits, S::WAVES, S::LANES>(top, slots);
    const float m = from_bits(top);
    float d = m * s / 448.f;
    // Rows of ordinary size; the others (empty rows, infinities, NaN, and
    // magnitudes whose products leave the range of fp32) take the
    // definition step by step.
    const bool usual = m > 0x1p-100f && m < 0x1p+100f && d >= 0x1p-126f;
    // The rows of a wave's groups decide together: both reductions need
    // every lane.
    if (S::LANES == 64 ? usual : __all(usual)) {
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
      float y[NCH][8];
#pragma unroll
      for (int i = 0; i < NCH; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          y[i][j] = (t + i * G) * 8 + j < p.cols ? hx[i].get(j) * s * w[i][j] : 0.f;
          ty = OpMaxBits::op(ty, abs_bits(y[i][j]));
        }
      ty = group_reduce<OpMaxBits, S::WAVES, S::LANES>(ty, slots + S::WAVES);
      float dy = from_bits(ty) / 448.f;
      if (dy < 0x1p-126f) dy = 0x1p-126f;  // a NaN stays
      const float rcp = 1.f / m;
#pragma unroll
      for (int i = 0; i < NCH; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float num = v[i][j] * 448.f, q = num * rcp;
          v[i][j] = usual ? __builtin_fmaf(__builtin_fmaf(-q, m, num), rcp, q) : y[i][j] / dy;
        }
      d = usual ? d : dy;
    }
    if (t == 0 && live) reinterpret_cast<float*>(p.scale)[row] = d;
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
      float v[8];
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = hx[i].get(j) * s * w[i][j];
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

// One row a group: enough workgroups are in flight to hide a row's latencies,
// and measured no slower than a loop over rows with or without the next
// row's loads issued ahead (8192x8192 to e4m3: 86 us, 87 and 103).
template <int DT, int OUT, class S, int TAIL>
SKG_DEV void norm_row(const NormParams& p, SKG_LDS uint32_t* slots) {
  typedef typename Elem<DT>::raw raw;
  constexpr int NCH = S::NCH, G = S::SIZE;
  const int t = threadIdx.x % G, row = blockIdx.x * S::GROUPS + threadIdx.x / G;
  const bool live = row < p.rows;  // every lane takes part in the reductions
  const int from = min(row, p.rows - 1);
  Chunk<DT> x[NCH], r[NCH];
  load_row<DT, S, TAIL>(x, p.x, from, p.ldx, t, p.cols);
  if (p.r) load_row<DT, S, TAIL>(r, p.r, from, p.ldr, t, p.cols);
  float w[NCH][8];
  load_weights<DT, S, TAIL>(w, p.w, p.w_f32, t, p.cols);
  place_row<DT, S, TAIL>(x, t, p.cols);
  if (p.r) {
    place_row<DT, S, TAIL>(r, t, p.cols);
#pragma unroll
    for (int i = 0; i < NCH; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i].put(j, x[i].get(j) + r[i].get(j));
  }
  if (p.h && live) {
    raw* h = reinterpret_cast<raw*>(p.h) + row * p.ldh;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int n = p.cols - (t + i * G) * 8;
      if (n > 0) store_chunk<DT>(h + (t + i * G) * 8, TAIL ? n : 8, x[i]);
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    float part = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) part = __builtin_fmaf(x[i].get(j), x[i].get(j), part);
    sum += part;
  }
  sum = group_reduce<OpSum, S::WAVES, S::LANES>(sum, slots);
  const float s = rsqrt_refined(sum * p.inv_cols + p.eps);
  if (p.rstd && t == 0 && live) p.rstd[row] = s;
  norm_output<DT, OUT, S, TAIL>(p, row, live, t, s, x, w, slots + S::WAVES);
}

template <int DT, int OUT, class S>
__global__ __launch_bounds__(S::THREADS) void rmsnorm_kernel(NormParams p) {
  __shared__ uint32_t slots_[3 * S::WAVES];
  SKG_LDS uint32_t* slots = (SKG_LDS uint32_t*)slots_;
  if (!(p.cols & 7)) return norm_row<DT, OUT, S, 0>(p, slots);
  if constexpr (S::COLS == kSmallSpread) {
    if (p.cols < 8) return norm_row<DT, OUT, S, 2>(p, slots);
  }
  norm_row<DT, OUT, S, 1>(p, slots);
}

// --- backward ------------------------------------------------------------------
struct NormBwdParams {
  const char *dy, *h, *w, *dres;
  const float* rstd;
  char* dx;
  float* partial;  // [workgroups][cols] (few rows: dw itself), or nullptr without dw
  int rows, cols, w_f32;
  int64_t lddy, ldh, ldr, lddx;
  float inv_cols;
};

// Each thread keeps the sums of dw of its columns; the groups of a workgroup
// are added at the end, in a fixed order, through LDS.
template <int DT, class S, int TAIL>
SKG_DEV void norm_bwd_rows(const NormBwdParams& p, SKG_LDS float* lds) {
  typedef typename Elem<DT>::raw raw;
  constexpr int NCH = S::NCH, G = S::SIZE;
  SKG_LDS uint32_t* slots = (SKG_LDS uint32_t*)lds;
  const int t = threadIdx.x % G, sub = threadIdx.x / G, step = gridDim.x * S::GROUPS;
  float w[NCH][8], dw[NCH][8];
  load_weights<DT, S, TAIL>(w, p.w, p.w_f32, t, p.cols);
#pragma unroll
  for (int i = 0; i < NCH; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
  int flip = 0;
  for (int base = blockIdx.x * S::GROUPS; base < p.rows; base += step, flip ^= S::WAVES) {
    const int row = min(base + sub, p.rows - 1);
    const bool live = base + sub < p.rows;
    Chunk<DT> dy[NCH], h[NCH], r[NCH];
    load_row<DT, S, TAIL>(dy, p.dy, row, p.lddy, t, p.cols);
    load_row<DT, S, TAIL>(h, p.h, row, p.ldh, t, p.cols);
    if (p.dres && p.dx) load_row<DT, S, TAIL>(r, p.dres, row, p.ldr, t, p.cols);
    const float s = p.rstd[row];
    place_row<DT, S, TAIL>(dy, t, p.cols);
    place_row<DT, S, TAIL>(h, t, p.cols);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      float part = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = h[i].get(j) * s;
        part = __builtin_fmaf(dy[i].get(j) * w[i][j], n, part);
        dw[i][j] = live ? __builtin_fmaf(dy[i].get(j), n, dw[i][j]) : dw[i][j];
      }
      dot += part;
    }
    if (!p.dx) continue;
    // Two sets of slots in turn: one barrier a row.
    dot = group_reduce<OpSum, S::WAVES, S::LANES>(dot, slots + flip) * p.inv_cols;
    if (p.dres) place_row<DT, S, TAIL>(r, t, p.cols);
    if (live) {
      raw* dx = reinterpret_cast<raw*>(p.dx) + row * p.lddx;
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        const int left = p.cols - (t + i * G) * 8;
        Chunk<DT> c;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float n = h[i].get(j) * s;
          const float v = s * __builtin_fmaf(-n, dot, dy[i].get(j) * w[i][j]);
          c.put(j, p.dres ? v + r[i].get(j) : v);
        }
        if (left > 0) store_chunk<DT>(dx + (t + i * G) * 8, TAIL ? left : 8, c);
      }
    }
  }
  if (!p.partial) return;
  float* o = p.partial + (int64_t)blockIdx.x * p.cols;
  if constexpr (S::GROUPS == 1) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int left = p.cols - (t + i * G) * 8;
      Chunk<DT_F32> c;
#pragma unroll
      for (int j = 0; j < 8; ++j) c.put(j, dw[i][j]);
      if (left > 0) store_chunk<DT_F32>(reinterpret_cast<uint32_t*>(o) + (t + i * G) * 8, left, c);
    }
  } else {
    // (The loop of these spreads has no barriers and uses no LDS.)
#pragma unroll
    for (int i = 0; i < NCH; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) lds[sub * S::COLS + (t + i * G) * 8 + j] = dw[i][j];
    __syncthreads();
    for (int c = threadIdx.x; c < p.cols; c += S::THREADS) {
      float sum = 0.f;
#pragma unroll
      for (int g = 0; g < S::GROUPS; ++g) sum += lds[g * S::COLS + c];
      o[c] = sum;
    }
  }
}

template <int DT, class S>
__global__ __launch_bounds__(S::THREADS) void rmsnorm_bwd_kernel(NormBwdParams p) {
  __shared__ float lds[S::GROUPS == 1 ? 2 * S::WAVES : S::GROUPS * S::COLS];
  if (!(p.cols & 7)) return norm_bwd_rows<DT, S, 0>(p, (SKG_LDS float*)lds);
  if constexpr (S::COLS == kSmallSpread) {
    if (p.cols < 8) return norm_bwd_rows<DT, S, 2>(p, (SKG_LDS float*)lds);
  }
  norm_bwd_rows<DT, S, 1>(p, (SKG_LDS float*)lds);
}

// Few rows, both gradients at once: the first workgroups take the rows (dx), the
// others 32 columns each (dw), which read dy and h again, from the cache.
// One launch and no workspace instead of two and one.
constexpr int kSmallThreads = 1024, kRuns = 32, kSmallCols = 16384, kSmallRows = 1024, kSmallElements = 1 << 20;

template <int N>
SKG_DEV float tree_sum(float (&v)[N]) {
#pragma unroll
  for (int n = N / 2; n; n >>= 1)
#pragma unroll
    for (int k = 0; k < n; ++k) v[k] += v[k + n];
  return v[0];
}

template <int DT, class S, int TAIL>
SKG_DEV void norm_bwd_row(const NormBwdParams& p, SKG_LDS uint32_t* slots) {
  typedef typename Elem<DT>::raw raw;
  constexpr int NCH = S::NCH, G = S::SIZE, GROUPS = kSmallThreads / G;
  const int t = threadIdx.x % G, grp = threadIdx.x / G, at = blockIdx.x * GROUPS + grp;
  const int row = min(at, p.rows - 1);
  Chunk<DT> dy[NCH], h[NCH], r[NCH];
  load_row<DT, S, TAIL>(dy, p.dy, row, p.lddy, t, p.cols);
  load_row<DT, S, TAIL>(h, p.h, row, p.ldh, t, p.cols);
  if (p.dres) load_row<DT, S, TAIL>(r, p.dres, row, p.ldr, t, p.cols);
  const float s = p.rstd[row];
  float w[NCH][8];
  load_weights<DT, S, TAIL>(w, p.w, p.w_f32, t, p.cols);
  place_row<DT, S, TAIL>(dy, t, p.cols);
  place_row<DT, S, TAIL>(h, t, p.cols);
  float dot = 0.f;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    float part = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) part = __builtin_fmaf(dy[i].get(j) * w[i][j], h[i].get(j) * s, part);
    dot += part;
  }
  dot = lanes_reduce<OpSum, S::LANES>(dot);
  if constexpr (S::WAVES > 1) {
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = __builtin_bit_cast(uint32_t, dot);
    __syncthreads();
    dot = 0.f;
#pragma unroll
    for (int k = 0; k < S::WAVES; ++k) dot += __builtin_bit_cast(float, (uint32_t)slots[grp * S::WAVES + k]);
  }
  dot *= p.inv_cols;
  if (at >= p.rows) return;
  if (p.dres) place_row<DT, S, TAIL>(r, t, p.cols);
  raw* dx = reinterpret_cast<raw*>(p.dx) + row * p.lddx;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int left = p.cols - (t + i * G) * 8;
    Chunk<DT> c;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float v = s * __builtin_fmaf(-h[i].get(j) * s, dot, dy[i].get(j) * w[i][j]);
      c.put(j, p.dres ? v + r[i].get(j) : v);
    }
    if (left > 0) store_chunk<DT>(dx + (t + i * G) * 8, TAIL ? left : 8, c);
  }
}

// dw of a few rows with the bits that norm_dw_kernel gives: thread (run, column)
// makes the partial sums run, run + 32, ..., of the rows that one workgroup of
// rmsnorm_bwd_kernel takes (it has a single round of them at these sizes), eight
// rows at a time in flight, and adds both as the two kernels do.
template <int DT, int GROUPS>
SKG_DEV void norm_dw_columns(const NormBwdParams& p, int block, SKG_LDS float* part) {
  typedef typename Elem<DT>::raw raw;
  constexpr int MOST = kSmallRows / kRuns;
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5, c0 = block * 32 + lane, c = min(c0, p.cols - 1);
  const raw* dy = reinterpret_cast<const raw*>(p.dy) + c;
  const raw* h = reinterpret_cast<const raw*>(p.h) + c;
  auto row_of = [&](int i) { return (run + i / GROUPS * kRuns) * GROUPS + i % GROUPS; };
  float v[MOST];
#pragma unroll
  for (int k = 0; k < MOST; ++k) v[k] = 0.f;
#pragma unroll
  for (int i0 = 0; i0 < MOST; i0 += 8) {
    if (row_of(i0) < p.rows) {
      raw a[8], b[8];
      float s[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t r = min(row_of(i0 + i), p.rows - 1);
        a[i] = dy[r * p.lddy];
        b[i] = h[r * p.ldh];
        s[i] = p.rstd[r];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = (i0 + i) / GROUPS;
        const float t = __builtin_fmaf(Elem<DT>::get(a[i]), Elem<DT>::get(b[i]) * s[i], 0.f);
        v[k] = row_of(i0 + i) < p.rows ? v[k] + t : v[k];
      }
    }
  }
  part[run * 33 + lane] = tree_sum(v);
  __syncthreads();
  if (run == 0 && c0 < p.cols) {
    float total = 0.f;
#pragma unroll
    for (int k = 0; k < kRuns; ++k) total += part[k * 33 + lane];
    p.partial[c0] = total;
  }
}

template <int DT, class S>
__global__ __launch_bounds__(kSmallThreads) void rmsnorm_bwd_small_kernel(NormBwdParams p, int row_blocks) {
  __shared__ float lds[kRuns * 33];
  if ((int)blockIdx.x >= row_blocks) return norm_dw_columns<DT, S::GROUPS>(p, blockIdx.x - row_blocks, (SKG_LDS float*)lds);
  SKG_LDS uint32_t* slots = (SKG_LDS uint32_t*)(SKG_LDS float*)lds;
  if (!(p.cols & 7)) return norm_bwd_row<DT, S, 0>(p, slots);
  if constexpr (S::COLS == kSmallSpread) {
    if (p.cols < 8) return norm_bwd_row<DT, S, 2>(p, slots);
  }
  norm_bwd_row<DT, S, 1>(p, slots);
}

// dw[c] = sum of the groups' partial[g][c], in a fixed order: 32 columns by 32
// runs of groups a workgroup, then the runs.  A run's loads are in flight
// together, so the time is a few latencies however many groups there are
// (512 x 4096: 4 us; one column a thread over all groups took 32).
// Without groups (no rows) it writes zeros.
__global__ __launch_bounds__(1024) void norm_dw_kernel(const float* __restrict__ partial, float* __restrict__ dw, int groups, int cols) {
  constexpr int RUNS = kRuns, MOST = kMostGroups / RUNS;
  __shared__ float part[RUNS][33];
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int c = min((int)blockIdx.x * 32 + lane, cols - 1);
  float v[MOST];
#pragma unroll
  for (int k = 0; k < MOST; ++k) {
    const int g = run + k * RUNS;
    v[k] = g < groups ? partial[(int64_t)g * cols + c] : 0.f;
  }
  part[run][lane] = tree_sum(v);
  __syncthreads();
  if (run == 0 && (int)blockIdx.x * 32 + lane < cols) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < RUNS; ++k) sum += part[k][lane];
    dw[c] = sum;
  }
}

// --- host ------------------------------------------------------------------------

// The first spread of the list that holds the row.
template <class F, class... S>
void with_spread(int64_t cols, F&& f, S... spreads) {
  bool done = false;
  ((done || cols > decltype(spreads)::COLS ? (void)0 : (f(spreads), (void)(done = true))), ...);
}
template <class F>
void with_spread(int64_t cols, F&& f) {
  with_spread(cols, f, Spread<1, 8, 1>{}, Spread<1, 16, 1>{}, Spread<1, 32, 1>{}, Spread<1, 64, 1>{}, Spread<1, 64, 2>{},
              Spread<2, 64, 2>{}, Spread<4, 64, 2>{}, Spread<8, 64, 2>{}, Spread<16, 64, 2>{}, Spread<16, 64, 4>{});
}

template <int DT, class S>
void launch_norm(const NormParams& all, int out, hipStream_t st) {
  // Rows in launches of fewer than 2^32 threads.
  constexpr int64_t most = int64_t(kMostThreads / S::THREADS) * S::GROUPS, es = sizeof(typename Elem<DT>::raw);
  for (int64_t r0 = 0; r0 < all.rows; r0 += most) {
    NormParams p = all;
    p.rows = (int)std::min<int64_t>(most, all.rows - r0);
    p.x += r0 * p.ldx * es;
    if (p.r) p.r += r0 * p.ldr * es;
    if (p.h) p.h += r0 * p.ldh * es;
    if (p.rstd) p.rstd += r0;
    p.y += out == OUT_SAME ? r0 * p.ldy * es : out == OUT_E2M1_MX ? r0 * (p.ldy / 2) : r0 * p.ldy;
    if (out != OUT_SAME) p.scale = static_cast<char*>(p.scale) + r0 * (out == OUT_E4M3_ROW ? 4 : p.cols / 32);
    const dim3 grid((unsigned)ceil_div(p.rows, S::GROUPS)), block(S::THREADS);
    switch (out) {
      case OUT_SAME: hipLaunchKernelGGL((rmsnorm_kernel<DT, OUT_SAME, S>), grid, block, 0, st, p); break;
      case OUT_E4M3_ROW: hipLaunchKernelGGL((rmsnorm_kernel<DT, OUT_E4M3_ROW, S>), grid, block, 0, st, p); break;
      case OUT_E4M3_MX: hipLaunchKernelGGL((rmsnorm_kernel<DT, OUT_E4M3_MX, S>), grid, block, 0, st, p); break;
      default: hipLaunchKernelGGL((rmsnorm_kernel<DT, OUT_E2M1_MX, S>), grid, block, 0, st, p);
    }
  }
}
template <int DT>
void launch_norm(const NormParams& p, int out, hipStream_t st) {
  with_spread(p.cols, [&](auto s) { launch_norm<DT, decltype(s)>(p, out, st); });
}
template <int DT>
void launch_norm_bwd(const NormBwdParams& p, int groups, bool small, hipStream_t st) {
  with_spread(p.cols, [&](auto s) {
    typedef decltype(s) S;
    if constexpr (S::COLS <= kSmallCols) {
      if (small) {
        const int rows = p.dx ? (int)ceil_div(p.rows, kSmallThreads / S::SIZE) : 0;
        hipLaunchKernelGGL((rmsnorm_bwd_small_kernel<DT, S>), dim3((unsigned)(rows + ceil_div(p.cols, 32))),
                           dim3(kSmallThreads), 0, st, p, rows);
        return;
      }
    }
    hipLaunchKernelGGL((rmsnorm_bwd_kernel<DT, S>), dim3((unsigned)groups), dim3(S::THREADS), 0, st, p);
  });
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
  if (a->rows > kMostRows) return unsupported("too many rows");
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
  if (a->dtype == SKG_F16)
    launch_norm<DT_F16>(p, out, st);
  else if (a->dtype == SKG_BF16)
    launch_norm<DT_BF16>(p, out, st);
  else
    launch_norm<DT_F32>(p, out, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return hip_failure(std::string("launch: ") + hipGetErrorString(e));
  return SKG_OK;
}

int check_norm_bwd(const skg_norm_bwd_args_t* a) {
  if (!a) return unsupported("null arguments");
  if (!row_type(a->dtype)) return unsupported("the norm's rows are f16, bf16 or f32");
  if (a->dtype_w != a->dtype && a->dtype_w != SKG_F32) return unsupported("the weight has the rows' type or f32");
  if (a->rows < 0 || a->cols <= 0) return unsupported("rows must not be negative and cols must be positive");
  if (a->rows > kMostRows) return unsupported("too many rows");
  if (a->cols > SKG_NORM_MAX_COLS) return unsupported("rows longer than SKG_NORM_MAX_COLS");
  if (a->lddy < a->cols || a->ldh < a->cols || (a->dres && a->lddres < a->cols) || (a->dx && a->lddx < a->cols))
    return unsupported("leading dimension too small");
  return SKG_OK;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}
// Whether both gradients come from one launch without a workspace.  The
// columns' share reads dy and h a second time, which is cheaper than a second
// launch and the partial sums (509x1111 f32 5.9 us a call against 9.2,
// 1000x1024 bf16 6.7 against 9.7).  At 1024x4096 the two took the same time;
// the limit lies where one launch was well ahead.  Not where dx is written
// over what that share reads; dw has the same bits in both.
bool bwd_small(const skg_norm_bwd_args_t* a) {
  if (!a->dw || a->rows < 1 || a->rows > kSmallRows || a->cols > kSmallCols || a->rows * a->cols > kSmallElements) return false;
  if (!a->dx) return true;
  const size_t es = elem_bytes(a->dtype);
  auto bytes = [&](int64_t ld) { return ((a->rows - 1) * ld + a->cols) * es; };
  return !overlap(a->dx, bytes(a->lddx), a->dy, bytes(a->lddy)) && !overlap(a->dx, bytes(a->lddx), a->h, bytes(a->ldh));
}
// Workgroups, each with one row of partial dw sums.
int bwd_groups(const skg_norm_bwd_args_t* a) {
  int64_t groups = 0;
  with_spread(a->cols, [&](auto s) {
    typedef decltype(s) S;
    static_assert(S::MOST <= kMostGroups, "what norm_dw_kernel adds");
    static_assert(S::GROUPS * S::MOST >= kSmallRows || (S::COLS / 2 + 1) * (int64_t)S::GROUPS * S::MOST >= kSmallElements,
                  "norm_dw_columns: a single round of rows at its sizes");
    groups = ceil_div(a->rows, S::GROUPS);
    if (groups > S::MOST) groups = S::MOST;
  });
  return (int)groups;
}

size_t bwd_bytes(const skg_norm_bwd_args_t* a) { return a->dw ? size_t(bwd_groups(a)) * a->cols * 4 : 0; }

// out, launched: what the call takes is wanted, and a workspace too small for
// it is not an error but leaves the call undone.
int run_norm_bwd(const skg_norm_bwd_args_t* a, void* ws, size_t ws_bytes, hipStream_t st, size_t* out = nullptr,
                 int32_t* launched = nullptr) {
  int rc = check_norm_bwd(a);
  if (rc) return rc;
  if (a->rows > 0 && (!a->dy || !a->h || !a->rstd)) return unsupported("null dy, h or rstd");
  if (!a->dx && !a->dw) return unsupported("neither dx nor dw is asked for");
  const size_t es = elem_bytes(a->dtype);
  if (!aligned_to(a->dy, es) || !aligned_to(a->h, es) || !aligned_to(a->dres, es) || !aligned_to(a->dx, es) ||
      !aligned_to(a->weight, elem_bytes(a->dtype_w)) || !aligned_to(a->rstd, 4) || !aligned_to(a->dw, 4))
    return unsupported("pointers must be aligned to their elements");
  const int groups = bwd_groups(a);
  const bool small = bwd_small(a);
  const size_t need = small ? 0 : bwd_bytes(a);
  if (out) *out = need;
  if (launched) {
    *launched = need <= ws_bytes;
    if (!*launched) return SKG_OK;
  }
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
    p.partial = small ? a->dw : a->dw ? static_cast<float*>(ws) : nullptr;
    p.rows = (int)a->rows;
    p.cols = (int)a->cols;
    p.w_f32 = a->dtype_w == SKG_F32;
    p.lddy = a->lddy;
    p.ldh = a->ldh;
    p.ldr = a->lddres;
    p.lddx = a->lddx;
    p.inv_cols = 1.f / (float)a->cols;
    if (a->dtype == SKG_F16)
      launch_norm_bwd<DT_F16>(p, groups, small, st);
    else if (a->dtype == SKG_BF16)
      launch_norm_bwd<DT_BF16>(p, groups, small, st);
    else
      launch_norm_bwd<DT_F32>(p, groups, small, st);
    e = hipGetLastError();
    if (e != hipSuccess) return hip_failure(std::string("launch: ") + hipGetErrorString(e));
  }
  if (a->dw && !small) {
    hipLaunchKernelGGL(norm_dw_kernel, dim3((unsigned)ceil_div(a->cols, 32)), dim3(1024), 0, st,
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
    *out = bwd_bytes(a);
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

int skg_plan_run_rmsnorm_bwd(const skg_norm_bwd_args_t* a, void* ws, size_t ws_bytes, void* stream, size_t* need,
                             int32_t* launched) {
  try {
    clear_error();
    if (!need || !launched) return unsupported("null output");
    *launched = 0;
    return run_norm_bwd(a, ws, ws_bytes, static_cast<hipStream_t>(stream), need, launched);
  } catch (const std::exception& ex) {
    return hip_failure(std::string("exception: ") + ex.what());
  } catch (...) {
    return hip_failure("unknown exception");
  }
}

}  // extern "C"
