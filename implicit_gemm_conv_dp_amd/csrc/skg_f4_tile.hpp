// fp4 (MX) products of many tiles: a ring of direct-to-LDS stages, four waves
// of (TM/2) x (TN/2) each, as many workgroups as the device has CUs.
//
// A stage is one iteration of 256 elements of K: 128-byte rows of A, then of
// B.  Scales travel apart from it in chunks of four iterations (32 bytes a
// row), a quarter of the next chunk with each stage: read an iteration at a
// time they touch as many cache lines as the codes do, and the requests to the
// L2 double.
//
// One wave a SIMD issues everything, an instruction in four or five cycles,
// and a 32x32x64 MFMA takes 32: so addresses are kept in registers, the
// position along K is the scalar offset of the loads, and every fragment read
// and DMA has its place after an MFMA of the k-step before (left to itself the
// compiler moves the reads next to their uses, and the MFMAs wait for them).
//
// What bounds it: power.  An iteration's 64 MFMAs of a wave, with its reads and
// loads and operands that stay in the L2, take 0.90 us on an otherwise idle device
// (2.42 GHz, the matrix units 93 % busy).  On all CUs the clock falls: 1.25 to
// 1.36 us with constant operands and 1.59 to 1.73 with random ones (1.35 GHz, 88 %
// busy), by the device: 5.0 to 5.4 PFLOP/s.  This loop takes 1.74 where that
// takes 1.59.  8192x8192x8192 to bf16 256 to 275 us (4.0 to 4.3 PFLOP/s): 4 x (32 iterations,
// 4 us of copy-out, which writes 8 TB/s, 2 us of start).  Measured without
// gain: reading the next stages into the L2 ahead, strips of 2 or 8 tile rows,
// refills every second or third MFMA, streaming stores.
#pragma once

#include "skg_device.hpp"
#include "skg_kernels.hpp"
#include "skg_launch.hpp"

namespace skg {

template <int TM_, int TN_, int D_>
struct F4Tile {
  static constexpr int TM = TM_, TN = TN_, D = D_;
  static constexpr int WTM = TM / 2, WTN = TN / 2, FM = WTM / 32, FN = WTN / 32;
  static constexpr int KS = 4, RB = 128;
  static constexpr int UA = TM / 32, UB = TN / 32;    // data DMAs a wave and stage
  static constexpr int NA = TM / 128, NB = TN / 128;  // scale DMAs a wave and stage
  static constexpr int PER = UA + UB + NA + NB;
  static constexpr int NCH = D;  // scale chunks held
  static constexpr int SLOT = (TM + TN) * RB, CH = (TM + TN) * 32;
  static constexpr int LDS = D * SLOT + NCH * CH;
  static_assert(LDS <= 160 * 1024 && (D & (D - 1)) == 0, "LDS");
  // Iteration i frees its slot at a barrier after MFMA SYNC of its last
  // k-step; stage i + D is loaded into it from there on, a DMA after each
  // MFMA (reaching into iteration i + 1).
  static constexpr int NM = FM * FN, SYNC = NM / 4;
  static constexpr int PART1 = NM - SYNC < PER ? NM - SYNC : PER;

  static_assert(NM - SYNC + (KS - 1) * NM >= PER, "a refill ends before the next begins");

  typedef i32x4 Frag;
  const GemmParams& g;
  SKG_LDS char* lds;
  int lane, wave, wm, wn, I;
  uint32_t sbase, cbase;  // ring entries of the tile's stage 0 and scale chunk 0
  uint32_t kb32, slim;
  uint32_t offa[UA], offb[UB], sofa, sofb;
  uint32_t fra[KS], frb[KS], fsa, fsb;  // this lane's fragments and scales in a slot / chunk
  i32x4 ra, rb;  // buffer resources of the tile's rows
  int na, nb;    // their sizes
  __amdgpu_buffer_rsrc_t rsa, rsb;
  f32x16 acc[FM][FN];
  uint32_t msa[FM][2], msb[FN][2];

  SKG_DEV F4Tile(const GemmParams& g_, SKG_LDS char* lds_) : g(g_), lds(lds_) {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wm = wave >> 1;
    wn = wave & 1;
    I = (g.K + 255) / 256;
    sbase = cbase = 0;
    kb32 = (uint32_t)g.K / 32;
    int row, chunk;
    lds_slot<RB>(threadIdx.x, row, chunk);
#pragma unroll
    for (int u = 0; u < UA; ++u) offa[u] = (uint32_t)(row + 32 * u) * g.lda_b + chunk * 16;
#pragma unroll
    for (int u = 0; u < UB; ++u) offb[u] = (uint32_t)(row + 32 * u) * g.ldb_b + chunk * 16;
    slim = (uint32_t)max((int)kb32 - (lane & 7) * 4, 0);
    sofa = (uint32_t)(wave * NA * 8 + (lane >> 3)) * kb32 + (lane & 7) * 4;
    sofb = (uint32_t)(wave * NB * 8 + (lane >> 3)) * kb32 + (lane & 7) * 4;
    const int r = lane & 31;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      fra[ks] = lds_off<RB>(wm * WTM + r, ks * 2 + (lane >> 5));
      frb[ks] = TM * RB + lds_off<RB>(wn * WTN + r, ks * 2 + (lane >> 5));
    }
    fsa = (wm * WTM + r) * 32;
    fsb = (TM + wn * WTN + r) * 32;
  }
  // Rows from row0 on; the last ends with its K elements, so nothing past
  // the operand is read.
  SKG_DEV static i32x4 rows_rsrc(const char* p, int row0, int rows, uint32_t pitch, uint32_t kbytes, int& n) {
    const uint64_t a = (uint64_t)(uintptr_t)(p + (size_t)row0 * pitch);
    n = __builtin_amdgcn_readfirstlane((int)min((int64_t)(rows - row0 - 1) * pitch + kbytes, (int64_t)0x7fffffff));
    return i32x4{__builtin_amdgcn_readfirstlane((int)(uint32_t)a), __builtin_amdgcn_readfirstlane((int)(a >> 32)), n,
                 0x00020000};
  }
  SKG_DEV void open(int m0, int n0) {
    ra = rows_rsrc(g.A, m0, g.M, g.lda_b, (uint32_t)g.K / 2, na);
    rb = rows_rsrc(g.B, n0, g.N, g.ldb_b, (uint32_t)g.K / 2, nb);
    rsa = make_rsrc_uniform((const char*)g.sa + (size_t)m0 * kb32,
                            (uint32_t)min((int64_t)(g.M - m0) * kb32, (int64_t)0x7fffffff));
    rsb = make_rsrc_uniform((const char*)g.sb + (size_t)n0 * kb32,
                            (uint32_t)min((int64_t)(g.N - n0) * kb32, (int64_t)0x7fffffff));
  }
  SKG_DEV uint32_t slot(int j) const { return ((sbase + j) & (D - 1)) * SLOT; }
  SKG_DEV uint32_t chunk(int c) const { return D * SLOT + ((cbase + c) & (NCH - 1)) * CH; }

  // Stage j: its rows, and a share of the scales of the chunk after next.
  // Codes past K (half of the last stage) come from the next row and meet
  // scales that are zero bytes, 2^-127: such products vanish in fp32.
  struct Stage {
    uint32_t kb, dst;          // byte offset along K, LDS address
    uint32_t dsa, dsb, va, vb;  // LDS addresses and buffer offsets of the scales
  };
  SKG_DEV Stage stage(int j) {
    Stage s;
    const bool live = j < I;  // a stage past the end reads nothing
    s.kb = live ? (uint32_t)j * RB : 0;
    ra[2] = live ? na : 0;
    rb[2] = live ? nb : 0;
    s.dst = lds_addr(lds) + slot(j) + wave * 1024;
    const int q = j + 3, c = q >> 2, piece = q & 3;  // stages 4c-3 .. 4c carry chunk c
    const uint32_t sk = (uint32_t)c * 32;
    const uint32_t ch = lds_addr(lds) + chunk(c);
    s.dsa = ch + piece * (TM / 4 * 32) + wave * (NA * 256);
    s.dsb = ch + TM * 32 + piece * (TN / 4 * 32) + wave * (NB * 256);
    s.va = (sk < slim ? sofa + sk : kOOB) + piece * (TM / 4) * kb32;
    s.vb = (sk < slim ? sofb + sk : kOOB) + piece * (TN / 4) * kb32;
    return s;
  }
  // 16 bytes a lane to LDS address dst + IMM, from a scalar offset along the rows.
  template <int IMM>
  SKG_DEV static void dma_row(const i32x4& r, uint32_t dst, uint32_t voff, uint32_t kb) {
    asm volatile("s_add_u32 m0, %0, %4\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(dst), "v"(voff), "s"(r), "s"(kb), "n"(IMM)
                 : "memory", "m0", "scc");
  }
  // DMA n (0 .. PER-1) of a stage.
  template <int N>
  SKG_DEV void dma(const Stage& s) const {
    if constexpr (N < UB) {
      dma_row<TM * RB + N * 4096>(rb, s.dst, offb[N], s.kb);
    } else if constexpr (N < UA + UB) {
      dma_row<(N - UB) * 4096>(ra, s.dst, offa[N - UB], s.kb);
    } else if constexpr (N < UA + UB + NA) {
      constexpr int U = N - UA - UB;
      dma4(rsa, s.dsa + U * 256, s.va + U * 8 * kb32);
    } else {
      constexpr int U = N - UA - UB - NA;
      dma4(rsb, s.dsb + U * 256, s.vb + U * 8 * kb32);
    }
  }
  // Read n of a k-step's fragments from the slot at offset st, in the order
  // their MFMAs need them.
  template <int N, int KSTEP>
  SKG_DEV void read_frag(Frag (&a)[FM], Frag (&b)[FN], uint32_t st) const {
    const SKG_LDS char* l = lds + st;
    if constexpr (N == 0)
      a[0] = *(const SKG_LDS i32x4*)(l + fra[KSTEP]);
    else if constexpr (N <= FN)
      b[N - 1] = *(const SKG_LDS i32x4*)(l + frb[KSTEP] + (N - 1) * 32 * RB);
    else
      a[N - FN] = *(const SKG_LDS i32x4*)(l + fra[KSTEP] + (N - FN) * 32 * RB);
  }
  template <int N>
  SKG_DEV void read_scale(i32x2 (&w)[FM + FN], uint32_t ch) const {
    if constexpr (N < FM)
      w[N] = *(const SKG_LDS i32x2*)(lds + ch + fsa + N * 1024);
    else
      w[N] = *(const SKG_LDS i32x2*)(lds + ch + fsb + (N - FM) * 1024);
  }
  SKG_DEV uint32_t scales_of(int j) const { return chunk(j >> 2) + (j & 3) * 8; }
  // The lane's block of each k-step: byte 0 (even k-steps) or 2 of its word.
  SKG_DEV void set_scales(const i32x2 (&w)[FM + FN]) {
    const int sh = 8 * (lane >> 5);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int f = 0; f < FM; ++f) msa[f][k] = (uint32_t)w[f][k] >> sh;
#pragma unroll
      for (int f = 0; f < FN; ++f) msb[f][k] = (uint32_t)w[FM + f][k] >> sh;
    }
  }

  // MFMAs [M0, M1) of a k-step, each followed by after(its number): the
  // order is kept, or the compiler moves reads next to their uses.
  template <int M0, int M1, int KSTEP, class F>
  SKG_DEV void mma(const Frag (&a)[FM], const Frag (&b)[FN], F&& after) {
    static_for<M0, M1>([&](auto m_) {
      constexpr int m = decltype(m_)::value, f = m / FN, n = m % FN;
      Mfma<DT_F4, 32>::run_scaled<(KSTEP & 1) * 2>(acc[f][n], b[n], a[f], msb[n][KSTEP >> 1], msa[f][KSTEP >> 1]);
      after(m_);
      __builtin_amdgcn_sched_barrier(0);
    });
  }
  // The k-step's fragments, read during the one before, are there: one wait
  // instead of one before each first use.
  SKG_DEV static void reads_done() {
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    __builtin_amdgcn_sched_barrier(0);
  }
  // DMA of the refill after MFMA m counted from its start, if one is due.
  template <int M, int END>
  SKG_DEV void refill(const Stage& s) const {
    if constexpr (M < END) dma<M>(s);
  }

  // Iteration i: its MFMAs, the reads of the next k-step's fragments among
  // them, the rest of the refill begun in iteration i - 1 (stage i - 1 + D)
  // and, once the slot is free, the beginning of the next (stage i + D).
  // The same for every iteration: past the tile's end the refills read
  // nothing and the fragments read are not used.
  SKG_DEV void iteration(Frag (&a)[2][FM], Frag (&b)[2][FN], Stage& s, int i) {
    constexpr int R = (FM + FN + NM - 1) / NM;  // reads after each MFMA
    const uint32_t cur = slot(i);
    static_for<0, KS - 1>([&](auto ks_) {
      constexpr int ks = decltype(ks_)::value;
      reads_done();
      mma<0, NM, ks>(a[ks & 1], b[ks & 1], [&](auto m_) {
        constexpr int m = decltype(m_)::value;
        static_for<m * R, (m + 1) * R>([&](auto n_) {
          if constexpr (decltype(n_)::value < FM + FN)
            read_frag<decltype(n_)::value, ks + 1>(a[(ks + 1) & 1], b[(ks + 1) & 1], cur);
        });
        constexpr int M = NM - SYNC + ks * NM + m;
        if constexpr (M >= PART1) refill<M, PER>(s);
      });
    });
    reads_done();
    mma<0, SYNC, KS - 1>(a[1], b[1], [](auto) {});
    // Stage i + 1 has landed once only younger ones are in flight.
    wait_vm<(D - 2) * PER>();
    lds_barrier();
    s = stage(i + D);
    i32x2 w[FM + FN];
    const uint32_t nxt = slot(i + 1), ch = scales_of(i + 1);
    constexpr int R2 = (2 * (FM + FN) + NM - SYNC - 1) / (NM - SYNC);
    mma<SYNC, NM, KS - 1>(a[1], b[1], [&](auto m_) {
      constexpr int m = decltype(m_)::value - SYNC;
      static_for<m * R2, (m + 1) * R2>([&](auto n_) {
        constexpr int n = decltype(n_)::value;
        if constexpr (n < FM + FN)
          read_scale<n>(w, ch);
        else if constexpr (n < 2 * (FM + FN))
          read_frag<n - FM - FN, 0>(a[0], b[0], nxt);
      });
      refill<m, PART1>(s);
    });
    set_scales(w);
    __builtin_amdgcn_sched_barrier(0);
  }

  SKG_DEV void advance() {
    sbase += I;
    cbase += (I + 3) >> 2;
  }
  // Chunk 0 and the stages that do not need the previous tile's last slot.
  SKG_DEV void ahead() {
    static_for<0, 4>([&](auto p_) {
      const Stage s = stage(decltype(p_)::value - 3);
      static_for<UA + UB, PER>([&](auto n_) { dma<decltype(n_)::value>(s); });
    });
    static_for<0, D - 1>([&](auto j_) {
      constexpr int j = decltype(j_)::value;
      const Stage s = stage(j);
      static_for<0, j == 0 ? UA + UB : PER>([&](auto n_) { dma<decltype(n_)::value>(s); });
    });
  }

  SKG_DEV void mainloop() {
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
      for (int n = 0; n < FN; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[f][n][e] = 0.f;
    Stage s = stage(D - 1);
    static_for<0, PART1>([&](auto n_) { dma<decltype(n_)::value>(s); });
    wait_vm<PART1 + (D - 2) * PER>();
    lds_barrier();
    Frag a[2][FM], b[2][FN];
    static_for<0, FM + FN>([&](auto n_) { read_frag<decltype(n_)::value, 0>(a[0], b[0], slot(0)); });
    i32x2 w[FM + FN];
    static_for<0, FM + FN>([&](auto n_) { read_scale<decltype(n_)::value>(w, scales_of(0)); });
    set_scales(w);
#pragma unroll 1
    for (int i = 0; i < I; ++i) iteration(a, b, s, i);
    wait_vm<0>();  // the refills past the end
    lds_barrier();
  }

  // The wave's part of the tile, a strip of 32 rows at a time through its
  // share of the last stage's slot, so that memory sees whole rows.
  template <int DTC>
  SKG_DEV void pack_strip(const f32x16 (&v)[FN], SKG_LDS char* st) const {
    constexpr int ES = DTC == DT_F32 ? 4 : 2, P = WTN * ES, CPR = P / 16;
    const int r = lane & 31, h = lane >> 5;
#pragma unroll
    for (int n = 0; n < FN; ++n) {
      if constexpr (DTC == DT_F32) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *(SKG_LDS f32x4*)(st + r * P + (((n * 8 + 2 * e + h) ^ r) % CPR) * 16) =
              f32x4{v[n][4 * e], v[n][4 * e + 1], v[n][4 * e + 2], v[n][4 * e + 3]};
      } else {
        // Lane l holds columns 8j + 4 (l / 32) + 0..3; exchanging halves gives
        // it eight consecutive ones.
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t p[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            p[k] = DTC == DT_F16 ? pack_f16x2(v[n][8 * e + 2 * k], v[n][8 * e + 2 * k + 1])
                                 : pack_bf16x2(v[n][8 * e + 2 * k], v[n][8 * e + 2 * k + 1]);
          const auto x = __builtin_amdgcn_permlane32_swap(p[0], p[2], false, false);
          const auto y = __builtin_amdgcn_permlane32_swap(p[1], p[3], false, false);
          *(SKG_LDS i32x4*)(st + r * P + (((n * 4 + 2 * e + h) ^ r) % CPR) * 16) =
              i32x4{(int)x[0], (int)y[0], (int)x[1], (int)y[1]};
        }
      }
    }
  }
  template <int ES>
  SKG_DEV void store_strip(const SKG_LDS char* st, int m0, int n0, bool whole) const {
    constexpr int P = WTN * ES, CPR = P / 16, RPI = 64 / CPR, EC = 16 / ES;
    const int cc = lane % CPR, r0 = lane / CPR, m = m0 + r0, col = n0 + cc * EC;
    char* o = g.C + ((size_t)m * g.ldc + col) * ES;
    const size_t step = (size_t)RPI * g.ldc * ES;
    if (whole) {
#pragma unroll
      for (int u = 0; u < 32 / RPI; ++u)
        *(i32x4*)(o + u * step) = *(const SKG_LDS i32x4*)(st + (u * RPI + r0) * P + ((cc ^ (u * RPI + r0)) % CPR) * 16);
    } else {
#pragma unroll 1
      for (int u = 0; u < 32 / RPI; ++u) {
        if (m + u * RPI >= g.M || col >= g.N) continue;
        char* d = o + u * step;
        const SKG_LDS char* q = st + (u * RPI + r0) * P + ((cc ^ (u * RPI + r0)) % CPR) * 16;
        if (col + EC <= g.N) {
          *(i32x4*)d = *(const SKG_LDS i32x4*)q;
        } else {
#pragma unroll 1
          for (int e = 0; e < g.N - col; ++e) {
            if constexpr (ES == 4)
              ((int*)d)[e] = ((const SKG_LDS int*)q)[e];
            else
              ((uint16_t*)d)[e] = ((const SKG_LDS uint16_t*)q)[e];
          }
        }
      }
    }
  }
  SKG_DEV void store_tile(int m0, int n0, SKG_LDS char* strips) const {
    static_assert(4 * 32 * WTN * 4 <= SLOT, "strips fit the slot");
    const bool whole = m0 + TM <= g.M && n0 + TN <= g.N;
    SKG_LDS char* st = strips + wave * 32 * WTN * 4;
    static_for<0, FM>([&](auto f_) {
      constexpr int f = decltype(f_)::value;
      const int m = m0 + wm * WTM + f * 32, n = n0 + wn * WTN;
      if (g.dtype_c == DT_F32) {
        pack_strip<DT_F32>(acc[f], st);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        store_strip<4>(st, m, n, whole);
      } else {
        if (g.dtype_c == DT_F16)
          pack_strip<DT_F16>(acc[f], st);
        else
          pack_strip<DT_BF16>(acc[f], st);
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        store_strip<2>(st, m, n, whole);
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    });
  }
};

// Workgroup k of `per` on XCD x takes tiles k, k + per, ... of the XCD's
// contiguous run of the tile list, which walks strips of GROUP tile rows column
// by column: the tiles in flight on an XCD form a block that shares its rows
// and columns in the XCD's L2.
template <class T>
__global__ __launch_bounds__(256, 1) void f4_tile_kernel(GemmParams g, KPlan p) {
  __shared__ __attribute__((aligned(128))) char lds[T::LDS];
  T t(g, (SKG_LDS char*)lds);
  const int total = p.tiles_m * p.tiles_n, x = blockIdx.x & 7;
  const int q = total >> 3, rem = total & 7;
  const int first = x * q + min(x, rem), count = q + (x < rem);
  const int per = ((int)gridDim.x + 7 - x) >> 3;
  constexpr int GROUP = 4;
  auto origin = [&](int k, int& m0, int& n0) {
    const int id = first + k, strip = id / (GROUP * p.tiles_n), in = id - strip * GROUP * p.tiles_n;
    const int rows = min(GROUP, p.tiles_m - strip * GROUP);
    const int tn = in / rows;
    m0 = (strip * GROUP + in - tn * rows) * T::TM;
    n0 = tn * T::TN;
    t.open(m0, n0);
  };
  int k = blockIdx.x >> 3, m0, n0;
  if (k >= count) return;
  origin(k, m0, n0);
  t.ahead();
  for (;;) {
    t.mainloop();
    // The next tile's first stages travel during this one's copy-out.
    const int m = m0, n = n0;
    k += per;
    SKG_LDS char* last = (SKG_LDS char*)lds + t.slot(t.I - 1);
    if (k < count) {
      origin(k, m0, n0);
      t.advance();
      t.ahead();
    }
    t.store_tile(m, n, last);
    if (k >= count) return;
    lds_barrier();  // every wave is done with the slot the strips went through
  }
}

template <class T>
hipError_t f4_tile_launch(const GemmParams& g, const KPlan& p, hipStream_t st) {
  const int total = p.tiles_m * p.tiles_n;
  hipLaunchKernelGGL((f4_tile_kernel<T>), dim3(total < p.cus ? total : p.cus), dim3(256), 0, st, g, p);
  return hipGetLastError();
}

}  // namespace skg
