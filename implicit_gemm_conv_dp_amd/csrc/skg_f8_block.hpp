// 8-bit products with an fp32 scale for each block of 128 elements of K:
//   C[m][n] = round(sum_kb sa[kb][m] sb[kb][n] sum_{k in kb} a(m, k) b(n, k))
// (sb one value for 128 columns, or one a column).  A 16x16x128 matrix instruction
// is one block of K: it starts from zero, and its four results a lane are
// multiplied by the blocks' scales into the fp32 sums by vector instructions.
#pragma once

#include "skg_device.hpp"
#include "skg_kernels.hpp"
#include "skg_launch.hpp"
#include "skg_ring8.hpp"

namespace skg {

// Codes of 128 elements of 16 rows of B and of A: element e of lane l is row
// l % 16 (of A), column 4 (l / 16) + e (of B).
template <int FMT>
SKG_DEV f32x4 f8_block(const i32x8& b, const i32x8& a) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, f32x4{0.f, 0.f, 0.f, 0.f}, FMT, FMT, 0, 0, 0, 0);
}
SKG_DEV i32x8 f8_frag(const SKG_LDS char* rows, int row, int lane) {
  const i32x4 lo = *(const SKG_LDS i32x4*)(rows + lds_off<128>(row, 2 * (lane >> 4)));
  const i32x4 hi = *(const SKG_LDS i32x4*)(rows + lds_off<128>(row, 2 * (lane >> 4) + 1));
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}
// An operand's scales as a buffer; the host keeps them under 2^31 bytes.
SKG_DEV i32x4 f8_scales(const float* s, int64_t lines, int64_t width) {
  const uint64_t a = (uint64_t)(uintptr_t)s;
  return i32x4{__builtin_amdgcn_readfirstlane((int)(uint32_t)a), __builtin_amdgcn_readfirstlane((int)(a >> 32)),
               __builtin_amdgcn_readfirstlane((int)(lines * width * 4)), 0x00020000};
}

// --- few tiles -------------------------------------------------------------------
// The four waves of a workgroup split K; each streams its own blocks, without a
// barrier, through LDS of its own, D blocks ahead.  The four partial tiles meet
// once in LDS and are added in a fixed order: one launch, no workspace.
template <int FM, int FN, int D, int FMT, bool ROWS>
struct F8Direct {
  static constexpr int TM = 16 * FM, TN = 16 * FN, WAVES = 4, RB = 128;
  static constexpr int UA = TM / 8, UB = TN / 8, PER = UA + UB + 2;
  static constexpr int XOFF = (TM + TN) * RB, SLOT = XOFF + 512;
  static constexpr int WAVE_LDS = D * SLOT, RED = WAVES * FM * FN * 64 * 16;
  static constexpr int LDS = WAVES * WAVE_LDS > RED ? WAVES * WAVE_LDS : RED;
  static_assert(TM <= 64 && TN <= 64 && LDS <= 160 * 1024, "tile");

  struct Operand {
    i32x4 rows, scales;
    int n, sn;
    uint32_t off[2], pitch8;  // rows of even and odd DMAs, eight rows
    uint32_t soff, spitch;
  };
  SKG_DEV static Operand operand(const char* p, int row0, int rows, uint32_t pitch, uint32_t kbytes, int lane) {
    Operand o;
    o.rows = ring_rows(p, row0, rows, pitch, kbytes, o.n);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      int row, chunk;
      lds_slot<RB>(n * 64 + lane, row, chunk);
      o.off[n] = (uint32_t)(row - 8 * n) * pitch + chunk * 16;
    }
    o.pitch8 = 8 * pitch;
    return o;
  }

  Operand A, B;
  SKG_LDS char* lds;  // the wave's
  int lane, first, count;

  // Block s of the wave's; past the end it reads nothing.
  SKG_DEV void issue(int s, int at) const {
    const bool live = s < count;
    const uint32_t kb = live ? (uint32_t)(first + s) : 0;
    const uint32_t dst = lds_addr(lds) + at * SLOT;
    i32x4 ra = A.rows, rb = B.rows, sa = A.scales, sb = B.scales;
    ra[2] = live ? A.n : 0;
    rb[2] = live ? B.n : 0;
    sa[2] = live ? A.sn : 0;
    sb[2] = live ? B.sn : 0;
    static_for<0, UB>([&](auto n_) {
      constexpr int n = decltype(n_)::value;
      ring_dma16<TM * RB + n * 1024>(rb, dst, B.off[n & 1] + n * B.pitch8, kb * RB);
    });
    static_for<0, UA>([&](auto n_) {
      constexpr int n = decltype(n_)::value;
      ring_dma16<n * 1024>(ra, dst, A.off[n & 1] + n * A.pitch8, kb * RB);
    });
    ring_dma4(sa, dst + XOFF, A.soff, kb * A.spitch);
    ring_dma4(sb, dst + XOFF + 256, B.soff, kb * B.spitch);
  }

  typedef f32x4 Acc[FM][FN];
  SKG_DEV void compute(Acc& acc, int at) const {
    const SKG_LDS char* st = lds + at * SLOT;
    const int r = lane & 15, q = lane >> 4;
    const SKG_LDS float* sc = (const SKG_LDS float*)(st + XOFF);
    i32x8 a[FM], b[FN];
    float sa[FM];
    f32x4 sb[FN];
#pragma unroll
    for (int f = 0; f < FM; ++f) {
      a[f] = f8_frag(st, f * 16 + r, lane);
      sa[f] = sc[f * 16 + r];
    }
#pragma unroll
    for (int f = 0; f < FN; ++f) {
      b[f] = f8_frag(st + TM * RB, f * 16 + r, lane);
      sb[f] = *(const SKG_LDS f32x4*)(sc + 64 + f * 16 + 4 * q);
    }
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const f32x4 t = f8_block<FMT>(b[j], a[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(t[e], sa[i] * sb[j][ROWS ? e : 0], acc[i][j][e]);
      }
  }

  SKG_DEV void run(const GemmParams& g, const KPlan& p, SKG_LDS char* group_lds) {
    lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    lds = group_lds + wave * WAVE_LDS;
    // Each XCD takes a contiguous run of tiles, M fastest, so the tiles
    // that read the same columns of B share an L2.
    const int T = p.tiles_m * p.tiles_n, per = T >> 3, rem = T & 7, x = blockIdx.x & 7;
    const int tile = x * per + min(x, rem) + (int)(blockIdx.x >> 3);
    const int tn = tile / p.tiles_m, tm = tile - tn * p.tiles_m;
    const int m0 = tm * TM, n0 = tn * TN, stages = g.K / 128;
    A = operand(g.A, m0, g.M, g.lda_b, (uint32_t)g.K, lane);
    B = operand(g.B, n0, g.N, g.ldb_b, (uint32_t)g.K, lane);
    const int64_t nb = ROWS ? g.N : (g.N + 127) / 128;
    A.scales = f8_scales(g.sa, stages, g.M);
    B.scales = f8_scales(g.sb, stages, nb);
    A.sn = A.scales[2];
    B.sn = B.scales[2];
    A.spitch = (uint32_t)g.M * 4;
    B.spitch = (uint32_t)nb * 4;
    A.soff = lane < TM && m0 + lane < g.M ? (uint32_t)(m0 + lane) * 4 : kOOB;
    B.soff = lane < TN && n0 + lane < g.N ? (uint32_t)(ROWS ? n0 + lane : (n0 + lane) / 128) * 4 : kOOB;
    first = (int)((int64_t)stages * wave / WAVES);
    count = (int)((int64_t)stages * (wave + 1) / WAVES) - first;

    Acc acc;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (count > 0) {
      static_for<0, D>([&](auto s_) { issue(decltype(s_)::value, decltype(s_)::value); });
      for (int s = 0; s < count; s += D) {
        static_for<0, D>([&](auto d_) {
          constexpr int d = decltype(d_)::value;
          if (s + d < count) {
            wait_vm<(D - 1) * PER>();  // block s + d has landed: the younger ones have not
            compute(acc, d);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            issue(s + d + D, d);
          }
        });
      }
      wait_vm<0>();
    }
    __syncthreads();  // LDS becomes the partial tiles'
    SKG_LDS f32x4* red = (SKG_LDS f32x4*)group_lds;

    // Partial tiles: slot (wave, fragment, lane) of four consecutive columns.
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) red[(wave * FM * FN + i * FN + j) * 64 + lane] = acc[i][j];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < (FM * FN + WAVES - 1) / WAVES; ++k) {
      const int f = k * WAVES + wave;
      if (f >= FM * FN) break;
      f32x4 v = red[f * 64 + lane];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) v += red[(w * FM * FN + f) * 64 + lane];
      const int m = m0 + f / FN * 16 + (lane & 15), n = n0 + f % FN * 16 + 4 * (lane >> 4);
      if (m >= g.M || n >= g.N) continue;
      const size_t o = (size_t)m * g.ldc + n;
      if (g.dtype_c == DT_F32) {
        float* c = (float*)g.C + o;
        if (n + 4 <= g.N) {
          *(f32x4*)c = v;
        } else {
          for (int e = 0; e < g.N - n; ++e) c[e] = v[e];
        }
      } else {
        uint16_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = g.dtype_c == DT_F16 ? to_f16_bits(v[e]) : to_bf16_bits(v[e]);
        uint16_t* c = (uint16_t*)g.C + o;
        if (n + 4 <= g.N) {
          *(uint2*)c = make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
        } else {
          for (int e = 0; e < g.N - n; ++e) c[e] = h[e];
        }
      }
    }
  }
};

template <class T>
__global__ __launch_bounds__(256) void f8_direct_kernel(GemmParams g, KPlan p) {
  __shared__ __attribute__((aligned(128))) char lds[T::LDS];
  T d;
  d.run(g, p, (SKG_LDS char*)lds);
}

template <class T>
GemmInst f8_direct() {
  return {[](const GemmParams& g, const KPlan& p, const Scratch&, hipStream_t st, hipEvent_t ev0, hipEvent_t ev1) {
            hipError_t e;
            if (ev0 && (e = hipEventRecord(ev0, st)) != hipSuccess) return e;
            hipLaunchKernelGGL((f8_direct_kernel<T>), dim3(p.grid), dim3(256), 0, st, g, p);
            if ((e = hipGetLastError()) != hipSuccess) return e;
            return ev1 ? hipEventRecord(ev1, st) : hipSuccess;
          },
          [](int* out) { return hipOccupancyMaxActiveBlocksPerMultiprocessor(out, f8_direct_kernel<T>, 256, 0); }};
}

}  // namespace skg
