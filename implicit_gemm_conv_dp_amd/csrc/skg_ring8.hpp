// Frame of the products that eight waves (WM x 8 / WM) of a workgroup compute on a
// ring of direct-to-LDS stages: the stages' loads and the copy-out.
//
// A stage is 128 bytes of K of the tile's TM rows of A, then of its TN rows of B,
// then EXTRA bytes that the product adds.  Two waves a SIMD: one issues vector
// arithmetic and LDS reads while the other's matrix instructions run.
#pragma once

#include "skg_device.hpp"
#include "skg_kernels.hpp"

namespace skg {

// Rows row0 .. rows-1 of an operand as a buffer that ends with the last one's
// kbytes, so nothing past the operand is read (nothing at all from row0 >= rows).
SKG_DEV i32x4 ring_rows(const char* p, int row0, int rows, uint32_t pitch, uint32_t kbytes, int& n) {
  const uint64_t a = (uint64_t)(uintptr_t)(p + (size_t)row0 * pitch);
  const int64_t bytes = row0 < rows ? (int64_t)(rows - row0 - 1) * pitch + kbytes : 0;
  n = __builtin_amdgcn_readfirstlane((int)min(bytes, (int64_t)0x7fffffff));
  return i32x4{__builtin_amdgcn_readfirstlane((int)(uint32_t)a), __builtin_amdgcn_readfirstlane((int)(a >> 32)), n, 0x00020000};
}
// 16 (or 4) bytes a lane to LDS address dst + IMM, from a scalar offset soff of
// the buffer.  The s_nop is the wait state that a write of M0 needs before such a
// load.
template <int IMM>
SKG_DEV void ring_dma16(const i32x4& r, uint32_t dst, uint32_t voff, uint32_t soff) {
  asm volatile("s_add_u32 m0, %0, %4\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(dst), "v"(voff), "s"(r), "s"(soff), "n"(IMM)
               : "memory", "m0", "scc");
}
SKG_DEV void ring_dma4(const i32x4& r, uint32_t dst, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
               :
               : "s"(dst), "v"(voff), "s"(r), "s"(soff)
               : "memory", "m0");
}

// NROWS rows of COLS elements of ES bytes in a wave's own LDS, in 16-byte pieces
// that are rotated within a row by the row's number.
template <int ES, int COLS>
SKG_DEV uint32_t strip_off(int row, int piece) {
  constexpr int P = COLS * ES, CPR = P / 16;
  return row * P + (uint32_t)(piece + row) % CPR * 16;
}
// Such a strip to rows m0 .. of C from column n0 on, whole 16-byte pieces where
// `vec` (C and its pitch are aligned to them); M, N: where C ends.
template <int ES, int COLS, int NROWS>
SKG_DEV void store_strip(const SKG_LDS char* st, char* C, int64_t ldc, int m0, int n0, int M, int N, bool vec) {
  constexpr int P = COLS * ES, CPR = P / 16, RPI = 64 / CPR < NROWS ? 64 / CPR : NROWS, EC = 16 / ES;
  constexpr bool EVEN = RPI * CPR == 64 && NROWS % RPI == 0;  // every lane has a piece each time
  const int lane = threadIdx.x & 63, cc = lane % CPR, r0 = lane / CPR, col = n0 + cc * EC;
  char* o = C + ((int64_t)(m0 + r0) * ldc + col) * ES;
  const int64_t step = RPI * ldc * ES;
  const bool fast = vec && m0 + NROWS <= M && n0 + COLS <= N;
  if (EVEN && fast) {
#pragma unroll
    for (int u = 0; u < NROWS / RPI; ++u)
      *(i32x4*)(o + u * step) = *(const SKG_LDS i32x4*)(st + strip_off<ES, COLS>(u * RPI + r0, cc));
  } else if (fast) {
#pragma unroll
    for (int u = 0; u < (NROWS + RPI - 1) / RPI; ++u)
      if (r0 < RPI && u * RPI + r0 < NROWS)
        *(i32x4*)(o + u * step) = *(const SKG_LDS i32x4*)(st + strip_off<ES, COLS>(u * RPI + r0, cc));
  } else {
#pragma unroll 1
    for (int u = 0; u < (NROWS + RPI - 1) / RPI; ++u) {
      const int row = u * RPI + r0;
      if (r0 >= RPI || row >= NROWS || m0 + row >= M || col >= N) continue;
      char* d = o + u * step;
      const SKG_LDS char* q = st + strip_off<ES, COLS>(row, cc);
      if (vec && col + EC <= N) {
        *(i32x4*)d = *(const SKG_LDS i32x4*)q;
      } else {
#pragma unroll 1
        for (int e = 0; e < min(EC, N - col); ++e) {
          if constexpr (ES == 4)
            ((int*)d)[e] = ((const SKG_LDS int*)q)[e];
          else
            ((uint16_t*)d)[e] = ((const SKG_LDS uint16_t*)q)[e];
        }
      }
    }
  }
}

template <int TM_, int TN_, int D_, int EXTRA_, int WM_ = 2>
struct Ring8 {
  static constexpr int TM = TM_, TN = TN_, D = D_, RB = 128, THREADS = 512;
  static constexpr int WM = WM_, WN = 8 / WM, WTM = TM / WM, WTN = TN / WN;
  static constexpr int UA = TM / 64, UB = TN / 64;  // row DMAs a wave and stage
  static constexpr int EXTRA = EXTRA_, SLOT = (TM + TN) * RB + EXTRA;
  static constexpr int LDS = D * SLOT;
  static constexpr int XOFF = (TM + TN) * RB;
  static_assert(LDS <= 160 * 1024, "LDS");

  SKG_LDS char* lds;
  int lane, wave, wm, wn, I;  // I: stages of a tile
  int at;                     // ring entry of the stage that runs
  uint32_t offa[UA], offb[UB];
  i32x4 ra, rb;
  int na, nb;

  SKG_DEV void init(SKG_LDS char* l, uint32_t lda_b, uint32_t ldb_b, int stages) {
    lds = l;
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wm = wave / WN;
    wn = wave % WN;
    I = stages;
    at = 0;
    int row, chunk;
    lds_slot<RB>(threadIdx.x, row, chunk);
#pragma unroll
    for (int u = 0; u < UA; ++u) offa[u] = (uint32_t)(row + 64 * u) * lda_b + chunk * 16;
#pragma unroll
    for (int u = 0; u < UB; ++u) offb[u] = (uint32_t)(row + 64 * u) * ldb_b + chunk * 16;
  }
  // Offset of the slot of the stage `ahead` (0 .. D) after the one that runs.
  SKG_DEV uint32_t slot(int ahead) const {
    const int s = at + ahead;
    return (s >= D ? s - D : s) * SLOT;
  }
  SKG_DEV void step() { at = at + 1 == D ? 0 : at + 1; }
  SKG_DEV uint32_t dst(int ahead) const { return lds_addr(lds) + slot(ahead); }
  // Row DMA N (0 .. UA+UB-1) of stage j into the slot at LDS address `to`; a stage
  // past the end reads nothing.
  template <int N>
  SKG_DEV void dma_rows(int j, uint32_t to) const {
    const bool live = j < I;
    const uint32_t kb = live ? (uint32_t)j * RB : 0;
    if constexpr (N < UB) {
      i32x4 r = rb;
      r[2] = live ? nb : 0;
      ring_dma16<TM * RB + N * 8192>(r, to + wave * 1024, offb[N], kb);
    } else {
      i32x4 r = ra;
      r[2] = live ? na : 0;
      ring_dma16<(N - UB) * 8192>(r, to + wave * 1024, offa[N - UB], kb);
    }
  }
};

// The tiles of a launch of at most a workgroup a CU: workgroup k of `per` on an
// XCD takes tiles k, k + per, ... of the XCD's contiguous run of the tile list.
struct TileRun {
  int first, count, per, k;
  SKG_DEV explicit TileRun(int total) {
    const int x = blockIdx.x & 7, q = total >> 3, rem = total & 7;
    first = x * q + min(x, rem);
    count = q + (x < rem);
    per = ((int)gridDim.x + 7 - x) >> 3;
    k = blockIdx.x >> 3;
  }
};

}  // namespace skg
