// fp4 (MX) products of few tiles: operands go from memory straight into the
// MFMA's registers and the four waves of a workgroup split the reduction.
//
// C tile = sum over waves w of A[:, K_w] B[:, K_w]^T with K cut into units of
// 512 elements dealt to the waves in contiguous runs.  A wave's partial tile
// stays in registers to its end; the four partials meet once in LDS and are
// added in a fixed order, so a call is deterministic, needs no workspace and
// is one launch.
//
// Used where the 128-row and 256-row tiles would leave most of the device
// idle: the time there is the latency of one tile's reduction, which this
// form cuts by four waves and by having a whole unit (5 loads a fragment) in
// flight, without a barrier in the loop.  A workgroup reads each operand
// element of its tile once, as the shared-memory tiles do, because no two of its
// waves share a K range.
#pragma once

#include "skg_device.hpp"
#include "skg_kernels.hpp"
#include "skg_launch.hpp"

namespace skg {

template <int FM, int FN>
struct F4Direct {
  static constexpr int TM = 16 * FM, TN = 16 * FN, WAVES = 4, THREADS = 64 * WAVES;
  static constexpr int UNIT = 4;  // MFMA steps of 128 elements in a unit

  // One unit of an operand's fragment: lane l holds row l % 16, block l / 16
  // of each step, and the four words of four scales of the row's unit.
  struct Frag {
    i32x4 v[UNIT];
    i32x4 s;
  };
  struct Operand {
    __amdgpu_buffer_rsrc_t data, scales;
    uint32_t off, soff;  // this lane's row of fragment 0, bytes
    uint32_t pitch16, spitch16;
  };

  // Rows past the operand's end lie past the resource and read as zeros.
  SKG_DEV static Operand operand(const char* p, const char* s, int row0, int rows, uint32_t pitch, uint32_t kbytes,
                                 uint32_t sbytes, int lane) {
    Operand o;
    o.data = make_rsrc_uniform(p + (size_t)row0 * pitch, (uint32_t)(rows - 1) * pitch + kbytes);
    o.scales = make_rsrc_uniform(s + (size_t)row0 * sbytes, (uint32_t)rows * sbytes);
    o.off = (uint32_t)(lane & 15) * pitch + (uint32_t)(lane >> 4) * 16;
    o.soff = (uint32_t)(lane & 15) * sbytes;
    o.pitch16 = 16 * pitch;
    o.spitch16 = 16 * sbytes;
    return o;
  }
  // Unit u of fragment f; steps from `left` on lie past K and are zeros.
  SKG_DEV static void load(Frag& r, const Operand& o, int f, int u, int left) {
#pragma unroll
    for (int j = 0; j < UNIT; ++j)
      r.v[j] = buffer_load16(o.data, j < left ? o.off + f * o.pitch16 + (uint32_t)(u * UNIT + j) * 64 : kOOB);
    const uint32_t so = o.soff + f * o.spitch16 + (uint32_t)u * 16;
    if (left >= UNIT) {
      r.s = buffer_load16(o.scales, so);
    } else {
#pragma unroll
      for (int j = 0; j < UNIT; ++j)
        r.s[j] = (int)__builtin_amdgcn_raw_buffer_load_b32(o.scales, j < left ? so + 4 * j : kOOB, 0, 0);
    }
  }

  SKG_DEV static void run(const GemmParams& g, const KPlan& p, SKG_LDS f32x4* red) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // Each XCD takes a contiguous run of tiles, M fastest, so the tiles
    // that read the same columns of B share an L2.
    const int T = p.tiles_m * p.tiles_n, q = T >> 3, rem = T & 7, x = blockIdx.x & 7;
    const int tile = x * q + min(x, rem) + (int)(blockIdx.x >> 3);
    const int tn = tile / p.tiles_m, tm = tile - tn * p.tiles_m;
    const int m0 = tm * TM, n0 = tn * TN;
    const uint32_t kbytes = (uint32_t)g.K / 2, sbytes = (uint32_t)g.K / 32;
    const Operand A = operand(g.A, (const char*)g.sa, m0, min(TM, g.M - m0), g.lda_b, kbytes, sbytes, lane);
    const Operand B = operand(g.B, (const char*)g.sb, n0, min(TN, g.N - n0), g.ldb_b, kbytes, sbytes, lane);
    const int steps = g.K / 128, units = (steps + UNIT - 1) / UNIT;
    const int u0 = units * wave / WAVES, u1 = units * (wave + 1) / WAVES;
    const int sh = 8 * (lane >> 4);

    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    Frag a[2][FM], b[2][FN];
    auto fetch = [&](int buf, int u) {
      const int left = steps - u * UNIT;
#pragma unroll
      for (int i = 0; i < FN; ++i) load(b[buf][i], B, i, u, left);
#pragma unroll
      for (int i = 0; i < FM; ++i) load(a[buf][i], A, i, u, left);
    };
    auto math = [&](int buf) {
#pragma unroll
      for (int s = 0; s < UNIT; ++s)
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                f4_operand(b[buf][j].v[s]), f4_operand(a[buf][i].v[s]), acc[i][j], 4, 4, 0,
                (int)((uint32_t)b[buf][j].s[s] >> sh), 0, (int)((uint32_t)a[buf][i].s[s] >> sh));
    };
    if (u0 < u1) fetch(0, u0);
    for (int u = u0; u < u1; u += 2) {
      if (u + 1 < u1) fetch(1, u + 1);
      math(0);
      if (u + 1 < u1) {
        if (u + 2 < u1) fetch(0, u + 2);
        math(1);
      }
    }

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
  __shared__ f32x4 red[4 * FM * FN * 64];
  F4Direct<FM, FN>::run(g, p, (SKG_LDS f32x4*)red);
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
