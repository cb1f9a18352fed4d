// fp4 (MX) products of few tiles: the four waves of a workgroup split the
// reduction and each streams its own part, without a barrier, through LDS of
// its own.
//
// C tile = sum over waves w of A[:, K_w] B[:, K_w]^T with K cut into stages of
// 256 elements dealt to the waves in contiguous runs.  A wave's partial tile
// stays in registers to its end; the four partials meet once in LDS and are
// added in a fixed order, so a call is deterministic, needs no workspace and
// is one launch.
//
// Used where the 128-row and 256-row tiles would leave most of the device
// idle: the time there is the latency of one tile's reduction, which this
// form cuts by four waves.  128-byte rows go straight to LDS (whole lines;
// loaded into the MFMA's register layout, 16 rows of 64 bytes an instruction,
// the same rows came in at half the rate).  With two stages a wave in flight a
// CU takes in 60 kB/us; the same loads with nothing else to do reach 135, so a
// deeper ring, for which the smaller tiles have the LDS, is what is left here.
#pragma once

#include "skg_device.hpp"
#include "skg_kernels.hpp"
#include "skg_launch.hpp"

namespace skg {

template <int FM, int FN>
struct F4Direct {
  static constexpr int TM = 16 * FM, TN = 16 * FN, WAVES = 4, THREADS = 64 * WAVES;
  static constexpr int D = 2, RB = 128;               // stages held, bytes of a row in one
  static constexpr int UA = TM / 8, UB = TN / 8;      // row DMAs of a stage
  static constexpr int CA = TM / 8, CB = TN / 8;      // scale DMAs of a chunk (four stages)
  static constexpr int UC = (CA + CB + 3) / 4;        // the share of one stage
  static constexpr int PER = UA + UB + UC;
  static constexpr int SLOT = (TM + TN) * RB, CH = (TM + TN) * 32;
  static constexpr int WAVE_LDS = D * SLOT + 2 * CH;
  static constexpr int RED = WAVES * FM * FN * 64 * 16;
  static constexpr int LDS = WAVES * WAVE_LDS > RED ? WAVES * WAVE_LDS : RED;
  static_assert(LDS <= 160 * 1024, "LDS");

  // An operand's rows and scales: buffer resources that end with its last
  // row's K elements, and this lane's offsets.
  struct Operand {
    i32x4 rows;
    __amdgpu_buffer_rsrc_t scales;
    uint32_t off[2], pitch8;  // rows of even and odd DMAs, eight rows
    uint32_t soff, spitch8;
  };
  SKG_DEV static Operand operand(const char* p, const char* s, int row0, int rows, uint32_t pitch, uint32_t kbytes,
                                 uint32_t kb32, int lane) {
    Operand o;
    const uint64_t a = (uint64_t)(uintptr_t)(p + (size_t)row0 * pitch);
    o.rows = i32x4{__builtin_amdgcn_readfirstlane((int)(uint32_t)a), __builtin_amdgcn_readfirstlane((int)(a >> 32)),
                   __builtin_amdgcn_readfirstlane((int)((uint32_t)(rows - 1) * pitch + kbytes)), 0x00020000};
    o.scales = make_rsrc_uniform(s + (size_t)row0 * kb32, (uint32_t)rows * kb32);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      int row, chunk;
      lds_slot<RB>(n * 64 + lane, row, chunk);
      o.off[n] = (uint32_t)(row - 8 * n) * pitch + chunk * 16;
    }
    o.pitch8 = 8 * pitch;
    o.soff = (uint32_t)(lane >> 3) * kb32 + (lane & 7) * 4;
    o.spitch8 = 8 * kb32;
    return o;
  }

  Operand A, B;
  SKG_LDS char* lds;  // the wave's
  int lane, first, count;  // the wave's stages
  uint32_t slim;

  // Row DMA n of the operand into a slot's part; kb: byte offset along K.
  template <int N>
  SKG_DEV static void dma_rows(const Operand& o, uint32_t dst, uint32_t kb) {
    asm volatile("s_add_u32 m0, %0, %4\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(dst), "v"(o.off[N & 1] + N * o.pitch8), "s"(o.rows), "s"(kb), "n"(N * 1024)
                 : "memory", "m0", "scc");
  }
  // Scale DMA n of chunk c (A's, then B's): eight rows of eight words of four
  // scales (K is a multiple of 128: whole words).  Words past K are zeros, so the
  // codes that were read past K, padding or another row's, are scaled by 2^-254
  // in all and vanish in fp32.
  template <int N>
  SKG_DEV void dma_scales(int c) const {
    if constexpr (N < CA + CB) {
      const uint32_t sk = (uint32_t)(first + 4 * c) * 8;
      const uint32_t dst = lds_addr(lds) + D * SLOT + (c & 1) * CH + N * 256;
      constexpr bool isa = N < CA;
      const Operand& o = isa ? A : B;
      constexpr int R = isa ? N : N - CA;
      dma4(o.scales, dst, (sk < slim ? o.soff + sk : kOOB) + R * o.spitch8);
    } else {
      dma_scales<CA + CB - 1>(c);  // evens out the stages
    }
  }
  // Stage s (Q = s mod 4) and its share of the scales: stages 4c-3 .. 4c carry
  // chunk c.  A stage past the end reads nothing.
  template <int Q>
  SKG_DEV void issue(int s, bool rows_only = false) {
    const bool live = s < count;
    const uint32_t kb = live ? (uint32_t)(first + s) * RB : 0;
    const uint32_t dst = lds_addr(lds) + (s & (D - 1)) * SLOT;
    Operand a = A, b = B;
    a.rows[2] = live ? A.rows[2] : 0;
    b.rows[2] = live ? B.rows[2] : 0;
    static_for<0, UB>([&](auto n_) { dma_rows<decltype(n_)::value>(b, dst + TM * RB, kb); });
    static_for<0, UA>([&](auto n_) { dma_rows<decltype(n_)::value>(a, dst, kb); });
    if (!rows_only)
      static_for<0, UC>([&](auto n_) { dma_scales<((Q + 3) & 3) * UC + decltype(n_)::value>((s + 3) >> 2); });
  }

  typedef f32x4 Acc[FM][FN];
  SKG_DEV void compute(Acc& acc, int s) const {
    const SKG_LDS char* st = lds + (s & (D - 1)) * SLOT;
    const SKG_LDS char* sc = lds + D * SLOT + ((s >> 2) & 1) * CH + (s & 3) * 8;
    const int r = lane & 15, q = lane >> 4, sh = 8 * q;
    i32x2 wa[FM], wb[FN];
    i32x4 a[2][FM], b[2][FN];
#pragma unroll
    for (int f = 0; f < FM; ++f) wa[f] = *(const SKG_LDS i32x2*)(sc + (f * 16 + r) * 32);
#pragma unroll
    for (int f = 0; f < FN; ++f) wb[f] = *(const SKG_LDS i32x2*)(sc + (TM + f * 16 + r) * 32);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int f = 0; f < FM; ++f) a[k][f] = *(const SKG_LDS i32x4*)(st + lds_off<RB>(f * 16 + r, k * 4 + q));
#pragma unroll
      for (int f = 0; f < FN; ++f) b[k][f] = *(const SKG_LDS i32x4*)(st + TM * RB + lds_off<RB>(f * 16 + r, k * 4 + q));
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              f4_operand(b[k][j]), f4_operand(a[k][i]), acc[i][j], 4, 4, 0, (int)((uint32_t)wb[j][k] >> sh), 0,
              (int)((uint32_t)wa[i][k] >> sh));
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
    const int m0 = tm * TM, n0 = tn * TN;
    const uint32_t kbytes = (uint32_t)g.K / 2, kb32 = (uint32_t)g.K / 32;
    A = operand(g.A, (const char*)g.sa, m0, min(TM, g.M - m0), g.lda_b, kbytes, kb32, lane);
    B = operand(g.B, (const char*)g.sb, n0, min(TN, g.N - n0), g.ldb_b, kbytes, kb32, lane);
    slim = (uint32_t)max((int)kb32 - (lane & 7) * 4, 0);
    const int stages = (g.K + 255) / 256;
    first = stages * wave / WAVES;
    count = stages * (wave + 1) / WAVES - first;

    Acc acc;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (count > 0) {
      static_for<0, CA + CB>([&](auto n_) { dma_scales<decltype(n_)::value>(0); });
      issue<0>(0, true);
      issue<1>(1);
      for (int s = 0; s < count; s += 4) {
        static_for<0, 4>([&](auto q_) {
          constexpr int q = decltype(q_)::value;
          if (s + q < count) {
            wait_vm<PER>();  // stage s + q has landed: the next one is younger
            compute(acc, s + q);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            issue<(q + 2) & 3>(s + q + 2);
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

template <int FM, int FN>
__global__ __launch_bounds__(256) void f4_direct_kernel(GemmParams g, KPlan p) {
  __shared__ __attribute__((aligned(128))) char lds[F4Direct<FM, FN>::LDS];
  F4Direct<FM, FN> d;
  d.run(g, p, (SKG_LDS char*)lds);
}

template <int FM, int FN>
GemmInst f4_direct() {
  return {[](const GemmParams& g, const KPlan& p, const Scratch&, hipStream_t st, hipEvent_t ev0, hipEvent_t ev1) {
            hipError_t e;
            if (ev0 && (e = hipEventRecord(ev0, st)) != hipSuccess) return e;
            hipLaunchKernelGGL((f4_direct_kernel<FM, FN>), dim3(p.grid), dim3(256), 0, st, g, p);
            if ((e = hipGetLastError()) != hipSuccess) return e;
            return ev1 ? hipEventRecord(ev1, st) : hipSuccess;
          },
          [](int* out) {
            return hipOccupancyMaxActiveBlocksPerMultiprocessor(out, f4_direct_kernel<FM, FN>, 256, 0);
          }};
}

}  // namespace skg
