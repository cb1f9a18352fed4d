// Orthogonalisation of an update by Newton-Schulz products (as the Muon optimiser
// does): X = G / (|G|_F + eps), then steps times
//   S = X X^T,   P = b S + c S^2,   X <- a X + P X.
//
// X is m x n with m <= n (G, or G transposed).  It is kept both ways in the
// workspace, X (m x n) and Y = X^T (n x m): S reduces over n, where X's rows are
// contiguous, and Y <- a Y + Y P over m, where Y's and the symmetric P's are; so
// every product is of two operands whose rows run along K, and a tile is written
// as it is and transposed.  S and P are symmetric: only tiles on and below the
// diagonal are computed, and written twice.
//
// Between the products everything is fp16 times a power of two (X 2^13, S 2^12,
// P 2^11): eleven bits against bf16's eight at the same rate of the matrix
// instructions, and S of a large matrix, whose entries are around 1/m, stays clear
// of fp16's subnormals.  Sums, the polynomial and the update are fp32, each
// rounded once when it is stored; the norm's sum is fp64.  P's diagonal is kept apart
// in fp32: where X is nearly orthogonal it is near -2.7, and a X + P X what is left of
// 3.4 X, so its rounding to eleven bits was most of the result's error (64 x 4096
// 0.0018 of its norm, 0.0008 so; one row 0.0043 and 0.0007).
//
// 4864 x 4096 takes 1.63 to 1.69 ms, five steps of three products at 0.87 to 0.96
// PFLOP/s (S 88 us, P 79, Y 170), the norm and first forms 65 us.  The matrix units are
// busy 48 % of the time: a product is one round of tiles, so a seventh of it is filling
// the ring and writing both forms with nothing behind it (40 MB each, at once), and
// the main loop waits for its loads.  300 x 1111 takes 84 us, seventeen launches of
// 3.5 to 6 us.  Where X is flat, S has few tiles over a long K, which nothing splits
// further than a workgroup's four waves: 64 x 4096 (three tiles of 32 x 32) takes 84 us,
// 256 x 16384 212, and 2048 x 2048 (136 tiles of 128 x 128 on 256 CUs) 348.
//
// Rows in the workspace are padded to whole 128 bytes with zeros: a product of
// padded operands is zero there, so the copy-out keeps the padding zero by writing
// it like the rest.
#include <algorithm>
#include <cmath>
#include <exception>
#include <string>

#include "skg_internal.hpp"
#include "skg_lowp.hpp"
#include "skg_ring8.hpp"

namespace skg {
namespace {

constexpr float kScaleX = 0x1p+13f, kScaleS = 0x1p+12f, kScaleP = 0x1p+11f;

// C = alpha A B^T + beta D: A M x K, B N x K, D and C M x N, Ct N x M, fp16 with
// rows of whole 128 bytes (the last step's C or Ct: the caller's type).
struct NsParams {
  const char *A, *B;
  const char* D;  // or nullptr; C's layout
  char *C, *Ct;   // either may be nullptr
  int M, N, K;
  int cn, ctn;               // columns of C and Ct that are written
  uint32_t lda_b, ldb_b;     // bytes
  int64_t ldd, ldc, ldct;    // elements
  float alpha, beta;
  // The diagonal of a symmetric product apart from it: ctn floats, and zeros in C.  And
  // of B: C = alpha A (B + diag) + beta D where D is A, so D's column n counts
  // beta + alpha diag[n] times.
  float* diag_out;
  const float* diag_in;
  int dt;                    // of C and Ct: DT_F16, DT_BF16 or DT_F32
  int vec;                   // C and Ct are aligned to 16 bytes
  int sym;                   // M == N: tiles on and below the diagonal; Ct is C
  int tiles_m, tiles_n, tiles;
};

// Tile `id` of the list: rows and columns in tiles.  Full grids are walked in
// strips of four tile rows, column by column, so that neighbours share operands.
SKG_DEV void ns_tile(const NsParams& p, int id, int& tm, int& tn) {
  if (p.sym) {
    tm = (int)((__builtin_sqrtf(8.f * (float)id + 1.f) - 1.f) * 0.5f);
    while (tm * (tm + 1) / 2 > id) --tm;
    while ((tm + 1) * (tm + 2) / 2 <= id) ++tm;
    tn = id - tm * (tm + 1) / 2;
  } else {
    constexpr int G = 4;
    const int strip = id / (G * p.tiles_n), in = id - strip * G * p.tiles_n, rows = min(G, p.tiles_m - strip * G);
    tn = in / rows;
    tm = strip * G + in - tn * rows;
  }
}

template <int DT>
SKG_DEV uint32_t ns_pack(float a, float b) {
  return DT == DT_F16 ? pack_f16x2(a, b) : pack_bf16x2(a, b);
}
SKG_DEV float half_at(const i32x4& v, int i) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)((uint32_t)v[i >> 1] >> (16 * (i & 1))));
}

// --- few tiles -------------------------------------------------------------------
// Four waves split K, each streaming its part through LDS of its own, D stages of
// 64 elements ahead; the partial tiles are added in a fixed order.
template <int FM, int FN, int D>
struct NsDirect {
  static constexpr int TM = 16 * FM, TN = 16 * FN, WAVES = 4, RB = 128;
  static constexpr int UA = TM / 8, UB = TN / 8, PER = UA + UB, SLOT = (TM + TN) * RB;
  static constexpr int WAVE_LDS = D * SLOT, RED = WAVES * FM * FN * 64 * 16;
  static constexpr int LDS = WAVES * WAVE_LDS > RED ? WAVES * WAVE_LDS : RED;
  static_assert(LDS <= 160 * 1024, "tile");

  SKG_DEV static void run(const NsParams& g, SKG_LDS char* group_lds) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    SKG_LDS char* lds = group_lds + wave * WAVE_LDS;
    const TileRun run(g.tiles);
    int tm, tn;
    ns_tile(g, run.first + run.k, tm, tn);
    const int m0 = tm * TM, n0 = tn * TN, stages = (g.K + 63) / 64;
    int na, nb;
    const i32x4 ra = ring_rows(g.A, m0, g.M, g.lda_b, g.lda_b, na), rb = ring_rows(g.B, n0, g.N, g.ldb_b, g.ldb_b, nb);
    uint32_t offa[2], offb[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      int row, chunk;
      lds_slot<RB>(n * 64 + lane, row, chunk);
      offa[n] = (uint32_t)(row - 8 * n) * g.lda_b + chunk * 16;
      offb[n] = (uint32_t)(row - 8 * n) * g.ldb_b + chunk * 16;
    }
    const int first = (int)((int64_t)stages * wave / WAVES), count = (int)((int64_t)stages * (wave + 1) / WAVES) - first;
    auto issue = [&](int s, int at) {
      const bool live = s < count;
      const uint32_t kb = live ? (uint32_t)(first + s) * RB : 0, dst = lds_addr(lds) + at * SLOT;
      i32x4 a = ra, b = rb;
      a[2] = live ? na : 0;
      b[2] = live ? nb : 0;
      static_for<0, UB>([&](auto n_) {
        constexpr int n = decltype(n_)::value;
        ring_dma16<TM * RB + n * 1024>(b, dst, offb[n & 1] + n * 8 * g.ldb_b, kb);
      });
      static_for<0, UA>([&](auto n_) {
        constexpr int n = decltype(n_)::value;
        ring_dma16<n * 1024>(a, dst, offa[n & 1] + n * 8 * g.lda_b, kb);
      });
    };
    // The wave's fragments of the joined tile, and D there, which travels with the
    // first stages (its rows are padded: whole fours).
    constexpr int PART = (FM * FN + WAVES - 1) / WAVES;
    auto place = [&](int k, int& m, int& n) {
      const int f = k * WAVES + wave;
      m = m0 + f / FN * 16 + (lane & 15);
      n = n0 + f % FN * 16 + 4 * (lane >> 4);
      return f < FM * FN;
    };
    uint2 d[PART];
    f32x4 more[PART];
#pragma unroll
    for (int k = 0; k < PART; ++k) {
      int m, n;
      d[k] = make_uint2(0, 0);
      more[k] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (place(k, m, n) && g.D && m < g.M && n < g.cn) {
        d[k] = *(const uint2*)(g.D + ((int64_t)m * g.ldd + n) * 2);
        if (g.diag_in) more[k] = *(const f32x4*)(g.diag_in + n);
      }
    }
    f32x4 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto compute = [&](int at) {
      const SKG_LDS char* st = lds + at * SLOT;
      const int r = lane & 15, q = lane >> 4;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        i32x4 a[FM], b[FN];
#pragma unroll
        for (int f = 0; f < FM; ++f) a[f] = *(const SKG_LDS i32x4*)(st + lds_off<RB>(f * 16 + r, 2 * q + k));
#pragma unroll
        for (int f = 0; f < FN; ++f) b[f] = *(const SKG_LDS i32x4*)(st + TM * RB + lds_off<RB>(f * 16 + r, 2 * q + k));
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j) Mfma<DT_F16, 16>::run(acc[i][j], b[j], a[i]);
      }
    };
    if (count > 0) {
      static_for<0, D>([&](auto s_) { issue(decltype(s_)::value, decltype(s_)::value); });
      for (int s = 0; s < count; s += D) {
        static_for<0, D>([&](auto d_) {
          constexpr int d = decltype(d_)::value;
          if (s + d < count) {
            wait_vm<(D - 1) * PER>();
            compute(d);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            issue(s + d + D, d);
          }
        });
      }
      wait_vm<0>();
    }
    __syncthreads();  // LDS becomes the partial tiles'
    SKG_LDS f32x4* red = (SKG_LDS f32x4*)group_lds;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) red[(wave * FM * FN + i * FN + j) * 64 + lane] = acc[i][j];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PART; ++k) {
      int m, n;
      if (!place(k, m, n)) break;
      const int f = k * WAVES + wave;
      f32x4 v = red[f * 64 + lane];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) v += red[(w * FM * FN + f) * 64 + lane];
      const i32x4 w = {(int)d[k].x, (int)d[k].y, 0, 0};
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[e] = __builtin_fmaf(v[e], g.alpha, half_at(w, e) * __builtin_fmaf(g.alpha, more[k][e], g.beta));
      if (g.diag_out) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (m == n + e) {
            if (m < g.ctn) g.diag_out[m] = x[e];
            x[e] = 0.f;
          }
        }
      }
      auto put = [&](char* base, int64_t at, float y) {
        if (g.dt == DT_F32)
          ((float*)base)[at] = y;
        else
          ((uint16_t*)base)[at] = g.dt == DT_F16 ? to_f16_bits(y) : to_bf16_bits(y);
      };
      if (g.C && m < g.M) {
        if (g.vec && n + 4 <= g.cn) {
          const int64_t at = (int64_t)m * g.ldc + n;
          if (g.dt == DT_F32)
            *(f32x4*)((float*)g.C + at) = f32x4{x[0], x[1], x[2], x[3]};
          else
            *(uint2*)((uint16_t*)g.C + at) = g.dt == DT_F16 ? make_uint2(pack_f16x2(x[0], x[1]), pack_f16x2(x[2], x[3]))
                                                            : make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n + e < g.cn) put(g.C, (int64_t)m * g.ldc + n + e, x[e]);
        }
      }
      if (g.Ct && m < g.ctn && !(g.sym && tm == tn)) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < g.N) put(g.Ct, (int64_t)(n + e) * g.ldct + m, x[e]);
      }
    }
  }
};
template <class T>
__global__ __launch_bounds__(256) void ns_direct_kernel(NsParams g) {
  __shared__ __attribute__((aligned(128))) char lds[T::LDS];
  T::run(g, (SKG_LDS char*)lds);
}

// --- many tiles ------------------------------------------------------------------
// Eight waves on a ring of D stages of 64 elements of K, a wave's part of the tile in
// 16 x 16 pieces.  A stage is 2 FM rows of FN instructions (two k-steps of 32); a row's
// fragment of A is read AHEAD rows before it, a k-step's fragments of B in the rows
// before.  AHEAD rows before its end a stage has been read: the barrier there frees
// its slot, which stage i + D is loaded into, and the next stage's reads begin.
template <int TM_, int TN_, int D_>
struct NsRing : Ring8<TM_, TN_, D_, 0> {
  typedef Ring8<TM_, TN_, D_, 0> R;
  using R::dst, R::I, R::lane, R::lds, R::na, R::nb, R::ra, R::rb, R::slot, R::step, R::wave, R::wm, R::wn;
  static constexpr int TM = TM_, TN = TN_, D = D_, WTM = R::WTM, WTN = R::WTN, RB = 128;
  static constexpr int FM = WTM / 16, FN = WTN / 16, ROWS = 2 * FM, AHEAD = 3, NA = AHEAD + 1, PER = R::UA + R::UB;
  static constexpr int STRIP = R::SLOT / 8;  // bytes of LDS of a wave's copy-out
  static_assert(STRIP >= 32 * WTN * 4, "strips fit the slot");
  static_assert(FM % 2 == 0 && ROWS % NA == 0 && FM > AHEAD, "rows");

  uint32_t fra, frb;
  f32x4 acc[FM][FN];

  SKG_DEV NsRing(const NsParams& g, SKG_LDS char* l) {
    R::init(l, g.lda_b, g.ldb_b, (g.K + 63) / 64);
    const int r = lane & 15, q = lane >> 4;
    fra = lds_off<RB>(wm * WTM + r, 2 * q);
    frb = TM * RB + lds_off<RB>(wn * WTN + r, 2 * q);
  }
  SKG_DEV void open(const NsParams& g, int m0, int n0) {
    ra = ring_rows(g.A, m0, g.M, g.lda_b, g.lda_b, na);
    rb = ring_rows(g.B, n0, g.N, g.ldb_b, g.ldb_b, nb);
  }
  typedef i32x4 Frag;
  // A lane's place in a slot at both k-steps: chunks 2q and 2q + 1 of a row, neighbours
  // in the permuted row.  (Any split of a row's chunks serves, A's and B's alike.  The
  // LDS serves a 16-byte read to 16 lanes at once, and not those of one q: with chunks q
  // and 4 + q they met in its banks by twos: 2048 x 2048 346 us, 321 so.)
  struct At {
    const SKG_LDS char* k[2];
  };
  SKG_DEV At at_k(uint32_t st, uint32_t first) const { return {{lds + (st + first), lds + ((st + first) ^ 16)}}; }
  template <int ROW>
  SKG_DEV static Frag read_a(const At& p) {
    return *(const SKG_LDS Frag*)(p.k[ROW / FM] + ROW % FM * 16 * RB);
  }
  template <int N, int KSTEP>
  SKG_DEV static Frag read_b(const At& p) {
    return *(const SKG_LDS Frag*)(p.k[KSTEP] + N * 16 * RB);
  }
  SKG_DEV void iteration(Frag (&a)[NA], Frag (&b)[2][FN], int i) {
    const uint32_t to = dst(0);
    const At ca = at_k(slot(0), fra), cb = at_k(slot(0), frb);
    At xa, xb;  // the next stage's
    static_for<0, ROWS>([&](auto r_) {
      constexpr int r = decltype(r_)::value, f = r % FM, ks = r / FM;
      constexpr bool late = r >= ROWS - AHEAD;  // reads belong to the next stage
      if constexpr (r == ROWS - AHEAD) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        wait_vm<(D - 2) * PER>();  // stage i + 1 has landed: the younger ones have not
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        xa = at_k(slot(1), fra);
        xb = at_k(slot(1), frb);
      }
      static_for<0, FN>([&](auto n_) {
        constexpr int n = decltype(n_)::value;
        Mfma<DT_F16, 16>::run(acc[f][n], b[ks][n], a[r % NA]);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (n == 0) {
          // Row r + AHEAD goes where row r - 1 was.
          if constexpr (late)
            a[(r + AHEAD) % NA] = read_a<r + AHEAD - ROWS>(xa);
          else
            a[(r + AHEAD) % NA] = read_a<r + AHEAD>(ca);
        }
        // B of the second k-step in the first rows, of the next stage in the last.
        if constexpr (late) {
          constexpr int s = (r - (ROWS - AHEAD)) * FN + n;  // 0 .. AHEAD FN - 1
          static_for<s * FN / (AHEAD * FN), (s + 1) * FN / (AHEAD * FN)>([&](auto m_) {
            b[0][decltype(m_)::value] = read_b<decltype(m_)::value, 0>(xb);
          });
          static_for<s * PER / (AHEAD * FN), (s + 1) * PER / (AHEAD * FN)>([&](auto d_) {
            R::template dma_rows<decltype(d_)::value>(i + D, to);
          });
        } else if constexpr (r >= 1 && r < 1 + FN && n == 1 % FN) {
          b[1][r - 1] = read_b<r - 1, 1>(cb);
        }
        __builtin_amdgcn_sched_barrier(0);
      });
    });
    step();
  }
  SKG_DEV void ahead() {
    static_for<0, D - 1>([&](auto j_) {
      constexpr int j = decltype(j_)::value;
      static_for<0, PER>([&](auto n_) { R::template dma_rows<decltype(n_)::value>(j, dst(j)); });
    });
  }
  // acc = D (beta / alpha + diag), so that alpha acc is all of C at the end: D's
  // loads travel with the first stages; behind a tile's stores they were waited for
  // (40 us of a 4096 x 4096 product).  (D's rows are whole 128 bytes: columns come in
  // fours.)
  SKG_DEV void begin(const NsParams& g, int m0, int n0) {
    const float ratio = g.beta / g.alpha;
    const __amdgpu_buffer_rsrc_t rd =
        make_rsrc_uniform(g.D + (int64_t)m0 * g.ldd * 2, (uint32_t)min((int64_t)max(g.M - m0, 0) * g.ldd * 2, (int64_t)0x7fffffff));
    f32x4 by[FN];
#pragma unroll
    for (int n = 0; n < FN; ++n) {
      const int c = n0 + wn * WTN + n * 16 + 4 * (lane >> 4);
      by[n] = f32x4{ratio, ratio, ratio, ratio};
      if (g.diag_in && c < g.cn) by[n] += *(const f32x4*)(g.diag_in + c);
    }
#pragma unroll
    for (int f = 0; f < FM; ++f) {
      i32x2 d[FN];
      const uint32_t row = (uint32_t)(wm * WTM + f * 16 + (lane & 15)) * (uint32_t)g.ldd;
#pragma unroll
      for (int n = 0; n < FN; ++n) {
        const int c = n0 + wn * WTN + n * 16 + 4 * (lane >> 4);
        d[n] = __builtin_bit_cast(i32x2, __builtin_amdgcn_raw_buffer_load_b64(rd, c < g.cn ? (row + c) * 2 : kOOB, 0, 0));
      }
#pragma unroll
      for (int n = 0; n < FN; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[f][n][e] = half_at(i32x4{d[n][0], d[n][1], 0, 0}, e) * by[n][e];
    }
  }
  SKG_DEV void zero() {
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
      for (int n = 0; n < FN; ++n) acc[f][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  SKG_DEV void mainloop() {
    static_for<0, PER>([&](auto n_) { R::template dma_rows<decltype(n_)::value>(D - 1, dst(D - 1)); });
    wait_vm<(D - 1) * PER>();
    lds_barrier();
    Frag a[NA], b[2][FN];
    const At pa = at_k(slot(0), fra), pb = at_k(slot(0), frb);
    static_for<0, AHEAD>([&](auto r_) { a[decltype(r_)::value] = read_a<decltype(r_)::value>(pa); });
    static_for<0, FN>([&](auto n_) { b[0][decltype(n_)::value] = read_b<decltype(n_)::value, 0>(pb); });
#pragma unroll 1
    for (int i = 0; i < I; ++i) iteration(a, b, i);
    wait_vm<0>();  // the refills past the end
    lds_barrier();
  }
  // The wave's part of the tile, 32 rows at a time through LDS of its own, as they are
  // and transposed.
  template <int DT>
  SKG_DEV void store_tile(const NsParams& g, int m0, int n0, bool diagonal, SKG_LDS char* strips) const {
    constexpr int ES = DT == DT_F32 ? 4 : 2;
    SKG_LDS char* st = strips + wave * STRIP;
    SKG_LDS char* tr = st + (DT == DT_F32 ? 0 : 32 * WTN * 2);  // fp32 (the last step's): one form only
    const int r = lane & 15, q = lane >> 4, c0 = n0 + wn * WTN;
    const bool transposed = g.Ct && !diagonal;
    static_for<0, FM / 2>([&](auto h_) {
      constexpr int h = decltype(h_)::value;
      const int m = m0 + wm * WTM + h * 32;
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int n = 0; n < FN; ++n) {
          f32x4 v = acc[2 * h + k][n] * g.alpha;
          const int row = k * 16 + r;
          if (diagonal && g.diag_out) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (m + row == c0 + n * 16 + 4 * q + e) {
                if (m + row < g.ctn) g.diag_out[m + row] = v[e];
                v[e] = 0.f;
              }
            }
          }
          if constexpr (DT == DT_F32) {
            if (g.C) {
              *(SKG_LDS f32x4*)(st + strip_off<4, WTN>(row, n * 4 + q)) = v;
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                *(SKG_LDS float*)(tr + strip_off<4, 32>(n * 16 + 4 * q + e, row / 4) + (row & 3) * 4) = v[e];
            }
          } else {
            const uint32_t p0 = ns_pack<DT>(v[0], v[1]), p1 = ns_pack<DT>(v[2], v[3]);
            if (g.C) *(SKG_LDS i32x2*)(st + strip_off<2, WTN>(row, n * 2 + (q >> 1)) + (q & 1) * 8) = i32x2{(int)p0, (int)p1};
            if (transposed) {
              // Neighbouring lanes hold neighbouring rows: each takes one column's pair.
              const uint32_t q0 = (uint32_t)__builtin_amdgcn_mov_dpp((int)p0, 0xB1, 0xf, 0xf, true);
              const uint32_t q1 = (uint32_t)__builtin_amdgcn_mov_dpp((int)p1, 0xB1, 0xf, 0xf, true);
              const uint32_t w0 = r & 1 ? __builtin_amdgcn_perm(p0, q0, 0x07060302) : __builtin_amdgcn_perm(q0, p0, 0x05040100);
              const uint32_t w1 = r & 1 ? __builtin_amdgcn_perm(p1, q1, 0x07060302) : __builtin_amdgcn_perm(q1, p1, 0x05040100);
              const int col = n * 16 + 4 * q + (r & 1);
              *(SKG_LDS uint32_t*)(tr + strip_off<2, 32>(col, row / 8) + (row % 8 / 2) * 4) = w0;
              *(SKG_LDS uint32_t*)(tr + strip_off<2, 32>(col + 2, row / 8) + (row % 8 / 2) * 4) = w1;
            }
          }
        }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (g.C) store_strip<ES, WTN, 32>(st, g.C, g.ldc, m, c0, g.M, g.cn, g.vec);
      if (transposed) store_strip<ES, 32, WTN>(tr, g.Ct, g.ldct, c0, m, g.N, g.ctn, g.vec);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    });
  }
};

// The kernel's arguments, read again from memory where they are used between main
// loops: kept in scalar registers through those, they would be spilled, along with
// the resources of the direct-to-LDS loads.
typedef const NsParams __attribute__((address_space(4))) * NsArgs;
SKG_DEV const NsParams& ns_args() {
  NsArgs p = (NsArgs)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const NsParams*)p;
}

template <class T>
__global__ __launch_bounds__(512, 1) void ns_ring_kernel(NsParams first) {
  __shared__ __attribute__((aligned(128))) char lds[T::LDS];
  T t(first, (SKG_LDS char*)lds);
  TileRun run(first.tiles);
  int k = run.k, tm, tn;
  if (k >= run.count) return;
  ns_tile(first, run.first + k, tm, tn);
  t.open(first, tm * T::TM, tn * T::TN);
  t.ahead();
  for (;;) {
    {
      const NsParams& g = ns_args();
      if (g.D)
        t.begin(g, tm * T::TM, tn * T::TN);
      else
        t.zero();
    }
    t.mainloop();
    // The next tile's first stages travel during this one's copy-out.
    const NsParams& g = ns_args();
    const int m = tm, n = tn;
    k += run.per;
    SKG_LDS char* last = (SKG_LDS char*)lds + t.slot(T::D - 1);  // the stage that ran last
    if (k < run.count) {
      ns_tile(g, run.first + k, tm, tn);
      t.open(g, tm * T::TM, tn * T::TN);
      t.ahead();
    }
    const bool diagonal = g.sym && m == n;
    if (g.dt == DT_F16)
      t.template store_tile<DT_F16>(g, m * T::TM, n * T::TN, diagonal, last);
    else if (g.dt == DT_BF16)
      t.template store_tile<DT_BF16>(g, m * T::TM, n * T::TN, diagonal, last);
    else
      t.template store_tile<DT_F32>(g, m * T::TM, n * T::TN, diagonal, last);
    if (k >= run.count) return;
    lds_barrier();  // every wave is done with the slot the strips went through
  }
}

// --- the norm and the operands' first form ---------------------------------------
constexpr int kSumBlocks = 1024;
struct NsInput {
  const char* g;
  int64_t rows, cols, ldg;
  double* partial;
  char *x, *xt;      // G / norm as it lies (rows x cols) and transposed
  int64_t px, pxt;   // their pitches in elements
  uint32_t chunks;   // of eight elements: rows x per
  FastDiv per;
  FastDiv across;    // tiles of 64 columns
  float eps;
  int blocks;
};
// Elements c .. c + 7 of a row, zeros past its end.
template <int DT>
SKG_DEV Chunk<DT> ns_load(const NsInput& a, int64_t row, int64_t c) {
  const typename Elem<DT>::raw* p = reinterpret_cast<const typename Elem<DT>::raw*>(a.g) + row * a.ldg + c;
  if (c + 8 <= a.cols) return reinterpret_cast<const Loose<Chunk<DT>>*>(p)->c;
  Chunk<DT> v{};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c + j < a.cols) v.v[j] = p[j];
  return v;
}
// Four chunks of a thread's are on their way at once.
template <int DT>
__global__ __launch_bounds__(256) void ns_sum_kernel(NsInput a) {
  constexpr int U = 4;
  __shared__ double part[4];
  double sum = 0;
  const uint32_t step = gridDim.x * 256;
  for (uint64_t i = blockIdx.x * 256 + threadIdx.x; i < a.chunks; i += (uint64_t)U * step) {
    Chunk<DT> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t k = (uint32_t)min(i + (uint64_t)u * step, (uint64_t)a.chunks - 1), r = fdiv(k, a.per);
      v[u] = ns_load<DT>(a, r, (int64_t)(k - r * a.per.d) * 8);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + (uint64_t)u * step >= a.chunks) break;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = __builtin_fma((double)v[u].get(j), (double)v[u].get(j), sum);
    }
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) a.partial[blockIdx.x] = part[0] + part[1] + part[2] + part[3];
}
// Tiles of 64 x 64: both forms, their padding with zeros, in whole 128-byte rows.
template <int DT>
__global__ __launch_bounds__(256) void ns_first_kernel(NsInput a) {
  __shared__ double part[4];
  __shared__ uint32_t tile[64][33];
  const uint32_t down = fdiv(blockIdx.x, a.across);
  const int64_t r0 = (int64_t)down * 64, c0 = (int64_t)(blockIdx.x - down * a.across.d) * 64;
  const int chunk = threadIdx.x & 7, line = threadIdx.x >> 3;  // of 32 lines
  Chunk<DT> v[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int64_t r = r0 + u * 32 + line;
    v[u] = ns_load<DT>(a, min(r, a.rows - 1), c0 + chunk * 8);
  }
  double sum = 0;
  for (int i = threadIdx.x; i < a.blocks; i += 256) sum += a.partial[i];
#pragma unroll
  for (int o = 32; o; o >>= 1) sum += __shfl_xor(sum, o);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
  __syncthreads();
  const double f = (double)kScaleX / (__builtin_sqrt(part[0] + part[1] + part[2] + part[3]) + (double)a.eps);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int64_t r = r0 + u * 32 + line;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = to_f16_bits((float)((double)v[u].get(2 * j) * f)), hi = to_f16_bits((float)((double)v[u].get(2 * j + 1) * f));
      w[j] = lo | hi << 16;
      // Zeros where nothing is read (a zero times an infinite factor is none).
      if (r >= a.rows || c0 + chunk * 8 + 2 * j >= a.cols)
        w[j] = 0;
      else if (c0 + chunk * 8 + 2 * j + 1 >= a.cols)
        w[j] &= 0xffff;
      tile[u * 32 + line][chunk * 4 + j] = w[j];
    }
    if (r < a.rows) *(uint4*)(a.x + (r * a.px + c0 + chunk * 8) * 2) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int c = u * 32 + line;
    if (c0 + c >= a.cols) continue;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = tile[chunk * 8 + 2 * j][c >> 1] >> (c & 1) * 16, hi = tile[chunk * 8 + 2 * j + 1][c >> 1] >> (c & 1) * 16;
      w[j] = (lo & 0xffff) | hi << 16;
    }
    *(uint4*)(a.xt + ((c0 + c) * a.pxt + r0 + chunk * 8) * 2) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// --- host ------------------------------------------------------------------------
bool row_type(int dt) { return dt == SKG_F16 || dt == SKG_BF16 || dt == SKG_F32; }
bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int64_t pitch_of(int64_t n) { return ceil_div(n, 64) * 64; }

// The workspace: partial sums, X and Y twice (a step reads one pair and writes the
// other), S, P and P's diagonal.
struct NsSpace {
  int64_t m, n, pm, pn;
  size_t x[2], y[2], s, p, diag, bytes;
};
NsSpace ns_space(const skg_newton_schulz_args_t* a) {
  NsSpace w;
  w.m = std::min(a->rows, a->cols);
  w.n = std::max(a->rows, a->cols);
  w.pm = pitch_of(w.m);
  w.pn = pitch_of(w.n);
  size_t at = kSumBlocks * sizeof(double);
  auto take = [&](int64_t rows, int64_t pitch) {
    const size_t r = at;
    at += (size_t)rows * pitch * 2;  // whole 128-byte rows
    return r;
  };
  for (int i = 0; i < 2; ++i) {
    w.x[i] = take(w.m, w.pn);
    w.y[i] = take(w.n, w.pm);
  }
  w.s = take(w.m, w.pm);
  w.p = take(w.m, w.pm);
  w.diag = take(2, w.pm);  // P's diagonal, fp32
  w.bytes = at;
  return w;
}

int check_newton(const skg_newton_schulz_args_t* a) {
  if (!a) return unsupported("null arguments");
  if (!row_type(a->dtype) || !row_type(a->dtype_out)) return unsupported("the update is f16, bf16 or f32");
  if (a->rows < 0 || a->cols < 0) return unsupported("rows and cols must not be negative");
  // Rows of the fp16 operands within 32-bit offsets of a tile of 256.
  constexpr int64_t most = (int64_t(INT32_MAX) / 256) / 2 - 64;
  if (a->rows > most || a->cols > most) return unsupported("dimension too large");
  // Tiles of every kernel, and the threads of their launches, within 32 bits.
  if (a->rows && a->cols > (int64_t(1) << 33) / a->rows) return unsupported("rows x cols must be at most 2^33");
  if (a->steps < 1 || a->steps > SKG_NEWTON_SCHULZ_MAX_STEPS) return unsupported("steps must be 1 to SKG_NEWTON_SCHULZ_MAX_STEPS");
  if (a->ldg < a->cols || a->ldo < a->cols) return unsupported("leading dimension too small");
  if (!(a->eps >= 0.f)) return unsupported("eps must not be negative");
  if (a->tile < SKG_NS_TILE_AUTO || a->tile >= SKG_NS_TILE_COUNT) return unsupported("unknown tile");
  // The last step's factors are scale times 2^-24 and less: normal numbers of fp32.
  if (!std::isfinite(a->scale) || (a->scale != 0.f && std::fabs(a->scale) < 0x1p-100f))
    return unsupported("scale must be finite, and 0 or at least 2^-100 in magnitude");
  return SKG_OK;
}

// Tiles of a product, over what is written of C and Ct (padding too); -1 where this
// kernel does not take it: a symmetric one needs square tiles.
int ns_tiles_m(const NsParams& p, int tm) { return (int)ceil_div(p.Ct ? std::max(p.M, p.ctn) : p.M, tm); }
int ns_tiles_n(const NsParams& p, int tn) { return (int)ceil_div(p.C ? std::max(p.N, p.cn) : p.N, tn); }
int ns_count(const NsParams& p, int tm, int tn) {
  const int m = ns_tiles_m(p, tm), n = ns_tiles_n(p, tn);
  return p.sym ? (tm == tn ? m * (m + 1) / 2 : -1) : m * n;
}
template <class T>
void ns_launch(const NsParams& q, int cus, int threads, hipStream_t st, void (*kernel)(NsParams), bool walk) {
  NsParams p = q;
  p.tiles_m = ns_tiles_m(p, T::TM);
  p.tiles_n = ns_tiles_n(p, T::TN);
  p.tiles = ns_count(p, T::TM, T::TN);
  hipLaunchKernelGGL(kernel, dim3((unsigned)(walk ? std::min(p.tiles, cus) : p.tiles)), dim3(threads), 0, st, p);
}
template <class T>
void ns_ring(const NsParams& p, int cus, hipStream_t st) {
  ns_launch<T>(p, cus, 512, st, ns_ring_kernel<T>, true);
}
template <class T>
void ns_direct(const NsParams& p, int cus, hipStream_t st) {
  ns_launch<T>(p, cus, 256, st, ns_direct_kernel<T>, false);
}

// The kernel and tile of a product: the least of the times that these models give, in
// us, rounds x (start + stages x stage) of a workgroup a CU and the launch.  They are
// rough: set by the sizes named here on the first forms of the ring kernels, some 10 %
// over what 256 x 256 and 128 x 128 take now, and for one workgroup of 32 x 32 a CU
// where two fit.  But on thirteen sizes from 64 x 4096 to 5120 x 5120 the update they
// choose took at most 7 % longer than the best with one tile for all its products
// (2048 x 2048 348 us, 325 on 128 x 128), and up to 28 % less.  What counts
// most for a large one is how full the last round is: 4096 x 4096 symmetric over 4864
// 88 us on 192 x 192 (253 tiles; 105 on 256 x 256, 136 tiles; 123 on 128 x 128, 528
// tiles), 4864 x 4096 over 4096 170 on 320 x 256 (256 tiles; 211 on 256 x 256, 304
// tiles; 197 on 128 x 128).  The direct kernels' waves split K, which a small one
// needs: fifteen products of 300 x 1111 and the norm take 83 us on 32 x 32 (two stages
// ahead, two workgroups a CU; 97 with four and one), 143 on 64 x 64 and 166 on
// 128 x 128.
struct NsKernel {
  int tm, tn, square;  // square: the kernel that takes this one's symmetric products
  double launch, start, stage;
  void (*run)(const NsParams&, int, hipStream_t);
};
const NsKernel kNsKernels[SKG_NS_TILE_COUNT] = {
    /* 32x32   */ {32, 32, 0, 2, 1.2, 0.16, ns_direct<NsDirect<2, 2, 2>>},
    /* 64x64   */ {64, 64, 1, 2, 3.3, 0.3, ns_direct<NsDirect<4, 4, 2>>},
    /* 128x128 */ {128, 128, 2, 1, 5, 0.52, ns_ring<NsRing<128, 128, 4>>},
    /* 192x192 */ {192, 192, 3, 1, 12, 0.97, ns_ring<NsRing<192, 192, 3>>},
    /* 256x192 */ {256, 192, 3, 1, 16, 1.15, ns_ring<NsRing<256, 192, 2>>},
    /* 256x256 */ {256, 256, 5, 1, 18, 1.3, ns_ring<NsRing<256, 256, 2>>},
    /* 320x256 */ {320, 256, 5, 1, 26, 2.25, ns_ring<NsRing<320, 256, 2>>},
};

hipError_t ns_product(const NsParams& p, int tile, int cus, hipStream_t st) {
  // A ring kernel divides D by alpha.
  const bool rings = !p.D || std::fabs(p.alpha) > 1e-20f * std::fabs(p.beta);
  if (tile == SKG_NS_TILE_AUTO) {
    double best = 1e300;
    for (int i = 0; i < SKG_NS_TILE_COUNT; ++i) {
      const NsKernel& k = kNsKernels[i];
      const int tiles = ns_count(p, k.tm, k.tn);
      if (tiles <= 0 || (k.tm >= 128 && !rings)) continue;
      const double us = k.launch + std::ceil((double)tiles / cus) * (k.start + (double)ceil_div(p.K, 64) * k.stage);
      if (us < best) {
        best = us;
        tile = i;
      }
    }
  } else {
    if (p.sym) tile = kNsKernels[tile].square;
    if (!rings && kNsKernels[tile].tm >= 128) tile = SKG_NS_TILE_64x64;
  }
  kNsKernels[tile].run(p, cus, st);
  return hipGetLastError();
}

int run_newton(const skg_newton_schulz_args_t* a, void* ws, size_t ws_bytes, hipStream_t st) {
  int rc = check_newton(a);
  if (rc) return rc;
  if (a->rows == 0 || a->cols == 0) return SKG_OK;
  if (!a->g || !a->out || !a->coefficients) return unsupported("null g, out or coefficients");
  for (int i = 0; i < 3 * a->steps; ++i)
    if (!std::isfinite(a->coefficients[i])) return unsupported("coefficients must be finite");
  if (!aligned_to(a->g, elem_bytes(a->dtype)) || !aligned_to(a->out, elem_bytes(a->dtype_out)))
    return unsupported("pointers must be aligned to their elements");
  const NsSpace w = ns_space(a);
  if (w.bytes > ws_bytes) return unsupported("workspace too small for this call");
  if (!ws || !aligned_to(ws, 256)) return unsupported("workspace must be 256-byte aligned device memory");
  int cus = 0;
  rc = check_device(&cus);
  if (rc) return rc;
  char* base = static_cast<char*>(ws);
  const bool wide = a->rows <= a->cols;
  NsInput in;
  in.g = static_cast<const char*>(a->g);
  in.rows = a->rows;
  in.cols = a->cols;
  in.ldg = a->ldg;
  in.partial = reinterpret_cast<double*>(base);
  in.x = base + (wide ? w.x[0] : w.y[0]);
  in.xt = base + (wide ? w.y[0] : w.x[0]);
  in.px = wide ? w.pn : w.pm;
  in.pxt = wide ? w.pm : w.pn;
  in.eps = a->eps;
  in.chunks = (uint32_t)(a->rows * ceil_div(a->cols, 8));
  in.per = make_fastdiv((uint32_t)ceil_div(a->cols, 8));
  in.across = make_fastdiv((uint32_t)ceil_div(a->cols, 64));
  in.blocks = (int)std::min<int64_t>(kSumBlocks, ceil_div(in.chunks, 256));
  auto first = [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    hipLaunchKernelGGL((ns_sum_kernel<DT>), dim3((unsigned)in.blocks), dim3(256), 0, st, in);
    hipLaunchKernelGGL((ns_first_kernel<DT>), dim3((unsigned)(ceil_div(a->cols, 64) * ceil_div(a->rows, 64))), dim3(256), 0, st, in);
  };
  if (a->dtype == SKG_F16)
    first(std::integral_constant<int, DT_F16>{});
  else if (a->dtype == SKG_BF16)
    first(std::integral_constant<int, DT_BF16>{});
  else
    first(std::integral_constant<int, DT_F32>{});
  hipError_t e = hipGetLastError();
  const int m = (int)w.m, n = (int)w.n;
  for (int i = 0; i < a->steps && e == hipSuccess; ++i) {
    const float ca = a->coefficients[3 * i], cb = a->coefficients[3 * i + 1], cc = a->coefficients[3 * i + 2];
    char *x = base + w.x[i & 1], *y = base + w.y[i & 1], *s = base + w.s, *poly = base + w.p;
    NsParams p{};
    p.dt = DT_F16;
    p.vec = 1;
    // S = X X^T
    p.A = p.B = x;
    p.lda_b = p.ldb_b = (uint32_t)w.pn * 2;
    p.M = p.N = m;
    p.K = n;
    p.C = p.Ct = s;
    p.ldc = p.ldct = w.pm;
    p.cn = p.ctn = (int)w.pm;
    p.alpha = kScaleS / (kScaleX * kScaleX);
    p.sym = 1;
    e = ns_product(p, a->tile, cus, st);
    // P = b S + c S S
    p.A = p.B = p.D = s;
    p.lda_b = p.ldb_b = (uint32_t)w.pm * 2;
    p.ldd = w.pm;
    p.K = m;
    p.C = p.Ct = poly;
    p.alpha = cc * (kScaleP / (kScaleS * kScaleS));
    p.beta = cb * (kScaleP / kScaleS);
    p.diag_out = reinterpret_cast<float*>(base + w.diag);
    if (e == hipSuccess) e = ns_product(p, a->tile, cus, st);
    // Y <- a Y + Y P, and X
    const bool last = i + 1 == a->steps;
    p.A = p.D = y;
    p.B = poly;
    p.diag_out = nullptr;
    p.diag_in = reinterpret_cast<const float*>(base + w.diag);
    p.M = n;
    p.N = m;
    p.sym = 0;
    p.ldd = w.pm;
    p.C = base + w.y[1 - (i & 1)];
    p.ldc = w.pm;
    p.cn = (int)w.pm;
    p.Ct = base + w.x[1 - (i & 1)];
    p.ldct = w.pn;
    p.ctn = (int)w.pn;
    p.alpha = 1.f / kScaleP;
    p.beta = ca;
    if (last) {
      p.dt = a->dtype_out == SKG_F32 ? DT_F32 : a->dtype_out == SKG_F16 ? DT_F16 : DT_BF16;
      const int64_t es = elem_bytes(a->dtype_out);
      p.vec = aligned_to(a->out, 16) && a->ldo * es % 16 == 0;
      char* out = static_cast<char*>(a->out);
      p.C = wide ? nullptr : out;
      p.Ct = wide ? out : nullptr;
      p.ldc = p.ldct = a->ldo;
      p.cn = m;
      p.ctn = n;
      p.alpha *= a->scale / kScaleX;
      p.beta *= a->scale / kScaleX;
    }
    if (e == hipSuccess) e = ns_product(p, a->tile, cus, st);
  }
  if (e != hipSuccess) return hip_failure(std::string("launch: ") + hipGetErrorString(e));
  return SKG_OK;
}

}  // namespace
}  // namespace skg

using namespace skg;

extern "C" {

int skg_newton_schulz_workspace_bytes(const skg_newton_schulz_args_t* a, size_t* out) {
  try {
    clear_error();
    const int rc = check_newton(a);
    if (rc) return rc;
    if (!out) return unsupported("null output");
    *out = a->rows == 0 || a->cols == 0 ? 0 : ns_space(a).bytes;
    return SKG_OK;
  } catch (...) {
    return hip_failure("exception in skg_newton_schulz_workspace_bytes");
  }
}

int skg_run_newton_schulz(const skg_newton_schulz_args_t* a, void* ws, size_t ws_bytes, void* stream) {
  try {
    clear_error();
    return run_newton(a, ws, ws_bytes, static_cast<hipStream_t>(stream));
  } catch (const std::exception& ex) {
    return hip_failure(std::string("exception: ") + ex.what());
  } catch (...) {
    return hip_failure("unknown exception");
  }
}

}  // extern "C"
