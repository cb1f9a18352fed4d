// Root-mean-square norms of queries and keys for each head with the position's
// rotation in the same pass, and their gradient.
//
// Forward, one head of D elements of one token:
//   s = 1 / sqrt(mean(x^2) + eps)                                  (fp32)
//   n = x s w
//   y = n with its first R elements turned in pairs (i, i + R/2), or with
//   neighbouring pairs (2i, 2i + 1), by the angle of pair i at the token's
//   position: (a, b) -> (a cos - b sin, b cos + a sin).
// Backward, g = dy turned back by the same angles:
//   dx = s (g w - x s^2 mean(g w x)),   dw = sum over tokens and heads g x s.
// Everything between the loads and the one rounding of y or dx is fp32.
//
// A group of 8 to 64 lanes takes a head, eight elements a lane, and keeps it in
// registers, so each operand is read once; the two elements of a pair (i, i + R/2)
// meet through LDS.  A group takes several heads of one token with the same
// cosines and sines, which come from the caches.  Bound by memory traffic: 16384
// tokens of 32 + 8 heads of 128 in bf16 take 72 us forward, 4.8 TB/s, and 106 us
// back, 4.8 TB/s (a large copy: 5.4); for a few tokens by the latency of the position,
// its table row, one reduction and a store (one token: 3.3 us).
#include <algorithm>
#include <exception>
#include <string>

#include "skg_internal.hpp"
#include "skg_lowp.hpp"

namespace skg {
namespace {

constexpr int kHeadThreads = 256;
// Most workgroups of the gradient of queries and of keys, each with a row of
// partial sums of dw.
constexpr int kHeadRuns = 32, kHeadMost = 1024;

struct Strides {
  int64_t b, t, h;  // elements between batches, tokens, heads
};
// Queries or keys.
struct HeadSet {
  const char *x, *w, *dy;
  char* y;         // backward: dx, or nullptr
  float* partial;  // backward: [blocks][D], or nullptr
  Strides sx, sy, sdy;
  int heads;
  uint32_t items, blocks;  // groups' shares; workgroups
  FastDiv div;             // by shares a token
};
struct HeadsParams {
  HeadSet set[2];
  const float *cos, *sin;  // table x half
  const void* pos;         // or nullptr
  int64_t pos0;
  int pos64, table, half, D, pairs, w_f32, seq;
  FastDiv div_seq;
  float eps, inv_d;
};

template <int DT, int TAIL>
SKG_DEV void head_weights(float (&w)[8], const HeadSet& s, const HeadsParams& p, int e0) {
  if (!s.w) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 1.f;
  } else if (DT == DT_F32 || p.w_f32) {
    Chunk<DT_F32> c = load_within<DT_F32, TAIL>(reinterpret_cast<const uint32_t*>(s.w), e0, p.D);
    place_chunk<DT_F32, TAIL>(c, e0, p.D);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = c.get(j);
  } else {
    Chunk<DT> c = load_within<DT, TAIL>(reinterpret_cast<const typename Elem<DT>::raw*>(s.w), e0, p.D);
    place_chunk<DT, TAIL>(c, e0, p.D);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = c.get(j);
  }
}

template <int N>
SKG_DEV void load_floats(float (&v)[N], const float* p) {
  struct __attribute__((packed, aligned(4))) L {
    float v[N];
  };
  const L l = *reinterpret_cast<const L*>(p);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = l.v[i];
}

// What element e0 + j of a token's heads is turned by: y = n c + m s, m the
// other element of its pair; c = 1 and s = 0 past the rotated ones.  A position
// outside the table reads row 0 in its place and gives NaN.
struct Turn {
  float c[8], s[8];
};
// PLAIN: see heads_bwd_kernel.
template <bool PLAIN>
SKG_DEV Turn load_turn(const HeadsParams& p, uint32_t token, int e0) {
  Turn r;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    r.c[j] = 1.f;
    r.s[j] = 0.f;
  }
  if (p.half == 0) return r;
  int64_t pos;
  if (!p.pos)
    pos = p.pos0 + (token - fdiv(token, p.div_seq) * (uint32_t)p.seq);
  else if (p.pos64)
    pos = static_cast<const int64_t*>(p.pos)[token];
  else
    pos = static_cast<const int32_t*>(p.pos)[token];
  const bool known = pos >= 0 && pos < p.table;
  const float* cs = p.cos + (known ? pos : 0) * p.half;
  const float* sn = p.sin + (known ? pos : 0) * p.half;
  if (p.pairs) {
    if (PLAIN || (p.half & 3) == 0) {  // a lane's four pairs all are, or none is, turned
      if (e0 < 2 * p.half) {
        float c[4], s[4];
        load_floats<4>(c, cs + e0 / 2);
        load_floats<4>(s, sn + e0 / 2);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          r.c[j] = c[j / 2];
          r.s[j] = j & 1 ? s[j / 2] : -s[j / 2];
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (e0 + j < 2 * p.half) {
          r.c[j] = cs[(e0 + j) / 2];
          r.s[j] = j & 1 ? sn[(e0 + j) / 2] : -sn[(e0 + j) / 2];
        }
    }
  } else {
    if (PLAIN || (p.half & 7) == 0) {  // a lane's eight elements lie on one side
      if (e0 < 2 * p.half) {
        const bool low = e0 < p.half;
        load_floats<8>(r.c, cs + (low ? e0 : e0 - p.half));
        load_floats<8>(r.s, sn + (low ? e0 : e0 - p.half));
#pragma unroll
        for (int j = 0; j < 8; ++j) r.s[j] = low ? -r.s[j] : r.s[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = e0 + j;
        if (e < 2 * p.half) {
          r.c[j] = cs[e < p.half ? e : e - p.half];
          r.s[j] = e < p.half ? -sn[e] : sn[e - p.half];
        }
      }
    }
  }
  if (!known) {
#pragma unroll
    for (int j = 0; j < 8; ++j) r.c[j] = e0 + j < 2 * p.half ? __builtin_nanf("") : 1.f;
  }
  return r;
}

// Turns a lane's elements; `row` is LDS of the group, a float for each element.
// Only the group's own wave touches it, so the wave's order of its LDS accesses
// is enough; the fences keep the compiler to it.
template <bool PLAIN>
SKG_DEV void turn(float (&v)[8], const Turn& r, const HeadsParams& p, int e0, SKG_LDS float* row) {
  float m[8];
  if (p.pairs) {
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = v[j ^ 1];
  } else {
    asm volatile("" ::: "memory");
    *(SKG_LDS f32x4*)(row + e0) = f32x4{v[0], v[1], v[2], v[3]};
    *(SKG_LDS f32x4*)(row + e0 + 4) = f32x4{v[4], v[5], v[6], v[7]};
    asm volatile("" ::: "memory");
    if (PLAIN || (p.half & 7) == 0) {
      const int o = e0 < p.half ? e0 + p.half : e0 < 2 * p.half ? e0 - p.half : e0;
      const f32x4 a = *(const SKG_LDS f32x4*)(row + o), b = *(const SKG_LDS f32x4*)(row + o + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        m[j] = a[j];
        m[j + 4] = b[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = e0 + j;
        m[j] = row[e < p.half ? e + p.half : e < 2 * p.half ? e - p.half : e];
      }
    }
    asm volatile("" ::: "memory");
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    v[j] = (PLAIN ? e0 : e0 + j) < 2 * p.half ? __builtin_fmaf(m[j], r.s[j], v[j] * r.c[j]) : v[j];
}

template <class C>
SKG_DEV C* head_at(C* base, const Strides& s, int64_t b, int64_t t, int h, int es) {
  return base + (b * s.b + t * s.t + h * s.h) * es;
}

// --- forward -------------------------------------------------------------------
template <int DT, int LANES, int U, int TAIL>
SKG_DEV void heads_rows(const HeadsParams& p, SKG_LDS float* lds) {
  typedef typename Elem<DT>::raw raw;
  constexpr int GROUPS = kHeadThreads / LANES, ES = sizeof(raw);
  const bool keys = blockIdx.x >= p.set[0].blocks;
  const HeadSet& s = p.set[keys];
  const int lane = threadIdx.x % LANES, sub = threadIdx.x / LANES, e0 = lane * 8;
  const uint32_t at = (blockIdx.x - (keys ? p.set[0].blocks : 0)) * GROUPS + sub;
  const uint32_t item = min(at, s.items - 1), token = fdiv(item, s.div);
  const int h0 = (int)(item - token * s.div.d) * U;
  const uint32_t b = fdiv(token, p.div_seq), t = token - b * (uint32_t)p.seq;
  Chunk<DT> x[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    x[u] = load_within<DT, TAIL>(reinterpret_cast<const raw*>(head_at(s.x, s.sx, b, t, min(h0 + u, s.heads - 1), ES)), e0, p.D);
  const Turn r = load_turn<false>(p, token, e0);
  float w[8];
  head_weights<DT, TAIL>(w, s, p, e0);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    place_chunk<DT, TAIL>(x[u], e0, p.D);
    float v[8], sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = x[u].get(j);
      sum = __builtin_fmaf(v[j], v[j], sum);
    }
    const float f = rsqrt_refined(lanes_reduce<OpSum, LANES>(sum) * p.inv_d + p.eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] * f * w[j];
    turn<false>(v, r, p, e0, lds + sub * LANES * 8);
    Chunk<DT> c;
#pragma unroll
    for (int j = 0; j < 8; ++j) c.put(j, v[j]);
    const int left = p.D - e0;
    if (at < s.items && h0 + u < s.heads && left > 0)
      store_chunk<DT>(reinterpret_cast<raw*>(head_at(s.y, s.sy, b, t, h0 + u, ES)) + e0, TAIL ? left : 8, c);
  }
}
template <int DT, int LANES, int U>
__global__ __launch_bounds__(kHeadThreads) void heads_kernel(HeadsParams p) {
  __shared__ __attribute__((aligned(16))) float lds[kHeadThreads * 8];
  if (!(p.D & 7)) return heads_rows<DT, LANES, U, 0>(p, (SKG_LDS float*)lds);
  if (p.D >= 8) return heads_rows<DT, LANES, U, 1>(p, (SKG_LDS float*)lds);
  if constexpr (LANES == 8) heads_rows<DT, LANES, U, 2>(p, (SKG_LDS float*)lds);
}

// --- backward ------------------------------------------------------------------
// The groups of a workgroup walk their shares in steps of the whole launch and
// add up dw of their elements; at the end the groups' sums are added in a fixed
// order through LDS.
template <int DT, int LANES, int U, int TAIL, bool PLAIN>
SKG_DEV void heads_bwd_rows(const HeadsParams& p, SKG_LDS float* lds) {
  typedef typename Elem<DT>::raw raw;
  constexpr int GROUPS = kHeadThreads / LANES, ES = sizeof(raw);
  const bool keys = blockIdx.x >= p.set[0].blocks;
  const HeadSet& s = p.set[keys];
  const uint32_t block = blockIdx.x - (keys ? p.set[0].blocks : 0);
  const int lane = threadIdx.x % LANES, sub = threadIdx.x / LANES, e0 = lane * 8;
  float w[8], dw[8];
  head_weights<DT, TAIL>(w, s, p, e0);
#pragma unroll
  for (int j = 0; j < 8; ++j) dw[j] = 0.f;
  for (uint32_t base = block * GROUPS; base < s.items; base += s.blocks * GROUPS) {
    const uint32_t at = base + sub, item = min(at, s.items - 1), token = fdiv(item, s.div);
    const int h0 = (int)(item - token * s.div.d) * U;
    const uint32_t b = fdiv(token, p.div_seq), t = token - b * (uint32_t)p.seq;
    Chunk<DT> x[U], dy[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = min(h0 + u, s.heads - 1);
      x[u] = load_within<DT, TAIL>(reinterpret_cast<const raw*>(head_at(s.x, s.sx, b, t, h, ES)), e0, p.D);
      dy[u] = load_within<DT, TAIL>(reinterpret_cast<const raw*>(head_at(s.dy, s.sdy, b, t, h, ES)), e0, p.D);
    }
    Turn r = load_turn<PLAIN>(p, token, e0);
#pragma unroll
    for (int j = 0; j < 8; ++j) r.s[j] = -r.s[j];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool live = at < s.items && h0 + u < s.heads;
      place_chunk<DT, TAIL>(x[u], e0, p.D);
      place_chunk<DT, TAIL>(dy[u], e0, p.D);
      float g[8], sum = 0.f, dot = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = dy[u].get(j);
      turn<PLAIN>(g, r, p, e0, lds + sub * LANES * 8);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float v = x[u].get(j);
        sum = __builtin_fmaf(v, v, sum);
        dot = __builtin_fmaf(g[j] * w[j], v, dot);
      }
      const float f = rsqrt_refined(lanes_reduce<OpSum, LANES>(sum) * p.inv_d + p.eps);
      const float k = lanes_reduce<OpSum, LANES>(dot) * p.inv_d * f;
      Chunk<DT> c;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = x[u].get(j) * f;
        dw[j] = live ? __builtin_fmaf(g[j], n, dw[j]) : dw[j];
        c.put(j, f * __builtin_fmaf(-n, k, g[j] * w[j]));
      }
      const int left = p.D - e0;
      if (s.y && live && left > 0)
        store_chunk<DT>(reinterpret_cast<raw*>(head_at(s.y, s.sy, b, t, h0 + u, ES)) + e0, TAIL ? left : 8, c);
    }
  }
  if (!s.partial) return;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 8; ++j) lds[sub * LANES * 8 + e0 + j] = dw[j];
  __syncthreads();
  for (int e = threadIdx.x; e < p.D; e += kHeadThreads) {
    float sum = 0.f;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) sum += lds[g * LANES * 8 + e];
    s.partial[(int64_t)block * p.D + e] = sum;
  }
}
// PLAIN: whole chunks of eight elements, each of which is turned as one or not at
// all, by eight (or, of neighbours, four) table entries in a row.  A kernel of its
// own, so that its four workgroups a CU, with two heads a group, stay resident:
// 16384 x (32 + 8) x 128 bf16 106 us, 119 with the others' registers and four heads.
// (The forward pass is not faster for it.)
template <int DT, int LANES, int U, bool PLAIN>
__global__ __launch_bounds__(kHeadThreads, PLAIN ? 4 : 1) void heads_bwd_kernel(HeadsParams p) {
  __shared__ __attribute__((aligned(16))) float lds[kHeadThreads * 8];
  if constexpr (PLAIN) {
    heads_bwd_rows<DT, LANES, U, 0, true>(p, (SKG_LDS float*)lds);
  } else {
    if (!(p.D & 7)) return heads_bwd_rows<DT, LANES, U, 0, false>(p, (SKG_LDS float*)lds);
    if (p.D >= 8) return heads_bwd_rows<DT, LANES, U, 1, false>(p, (SKG_LDS float*)lds);
    if constexpr (LANES == 8) heads_bwd_rows<DT, LANES, U, 2, false>(p, (SKG_LDS float*)lds);
  }
}

// dw of queries (blockIdx.y 0) and keys: the workgroups' partial sums in a fixed
// order, 32 elements by 32 runs of workgroups, a run's loads in flight together.
// Without workgroups (no rows) it writes zeros.
struct HeadDw {
  const float* partial[2];
  float* dw[2];
  int blocks[2];
};
__global__ __launch_bounds__(32 * kHeadRuns) void heads_dw_kernel(HeadDw a, int D) {
  constexpr int MOST = kHeadMost / kHeadRuns;
  __shared__ float part[kHeadRuns][33];
  const int y = blockIdx.y, lane = threadIdx.x & 31, run = threadIdx.x >> 5, e0 = blockIdx.x * 32 + lane;
  if (!a.dw[y]) return;
  const int e = min(e0, D - 1);
  float v[MOST];
#pragma unroll
  for (int k = 0; k < MOST; ++k) {
    const int g = run + k * kHeadRuns;
    v[k] = g < a.blocks[y] ? a.partial[y][(int64_t)g * D + e] : 0.f;
  }
#pragma unroll
  for (int n = MOST / 2; n; n >>= 1)
#pragma unroll
    for (int k = 0; k < n; ++k) v[k] += v[k + n];
  part[run][lane] = v[0];
  __syncthreads();
  if (run == 0 && e0 < D) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < kHeadRuns; ++k) sum += part[k][lane];
    a.dw[y][e0] = sum;
  }
}

// --- host ------------------------------------------------------------------------
bool row_type(int dt) { return dt == SKG_F16 || dt == SKG_BF16 || dt == SKG_F32; }
bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int lanes_of(int64_t D) { return D <= 64 ? 8 : D <= 128 ? 16 : D <= 256 ? 32 : 64; }

// Heads of one token that a group takes, of queries and of keys alike: `most` where
// that leaves enough groups to fill the device.  (A set of fewer heads than that takes
// its last one again, and drops the result.)
int heads_a_group(int64_t tokens, int heads, int lanes, int most) {
  return tokens * ceil_div(heads, most) * lanes >= int64_t(64) * 4096 ? most : 1;
}
// Shares of queries or keys: heads in fours (the gradient: twos) or one by one for
// each token.
int64_t shares(int64_t tokens, int heads, int u) { return tokens * ceil_div(heads, u); }

struct HeadPlan {
  int lanes, u;
  int64_t items[2], blocks[2];
};
HeadPlan plan_heads(const skg_heads_args_t* a, bool bwd) {
  HeadPlan p;
  p.lanes = lanes_of(a->head_dim);
  const int64_t tokens = a->batch * a->seq;
  p.u = heads_a_group(tokens, std::max(a->heads_q, a->heads_k), p.lanes, bwd ? 2 : 4);
  const int groups = kHeadThreads / p.lanes;
  for (int i = 0; i < 2; ++i) {
    p.items[i] = shares(tokens, i ? a->heads_k : a->heads_q, p.u);
    p.blocks[i] = ceil_div(p.items[i], groups);
  }
  if (bwd) {
    // As many workgroups as stay resident, shared out by the work.
    const int64_t all = p.blocks[0] + p.blocks[1];
    for (int i = 0; i < 2; ++i)
      if (all > kHeadMost && p.blocks[i])
        p.blocks[i] = std::max<int64_t>(1, std::min<int64_t>(p.blocks[i], kHeadMost * p.blocks[i] / all));
  }
  return p;
}

int check_heads(const skg_heads_args_t* a) {
  if (!a) return unsupported("null arguments");
  if (!row_type(a->dtype)) return unsupported("heads are f16, bf16 or f32");
  if (a->dtype_w != a->dtype && a->dtype_w != SKG_F32) return unsupported("the weight has the heads' type or f32");
  if (a->batch < 0 || a->seq < 0 || a->heads_q < 0 || a->heads_k < 0) return unsupported("sizes must not be negative");
  if (a->head_dim <= 0 || a->head_dim > SKG_HEADS_MAX_DIM) return unsupported("head_dim must be 1 to SKG_HEADS_MAX_DIM");
  if (a->rope_dim < 0 || a->rope_dim > a->head_dim || a->rope_dim % 2)
    return unsupported("rope_dim must be even and within head_dim");
  if (a->style != SKG_ROPE_HALF && a->style != SKG_ROPE_PAIRS) return unsupported("unknown rotation style");
  if (!(a->eps >= 0.f)) return unsupported("eps must not be negative");
  if (a->pos_bits != 32 && a->pos_bits != 64) return unsupported("positions have 32 or 64 bits");
  constexpr int64_t most = INT32_MAX - 65536;
  const int64_t heads = std::max<int64_t>(1, std::max(a->heads_q, a->heads_k));
  if (a->seq > most || a->batch > most || (a->seq && a->batch > most / a->seq) ||
      (a->seq && a->batch && heads > most / (a->batch * a->seq)))
    return unsupported("too many heads for 32-bit counts");
  return SKG_OK;
}

int fill_heads(const skg_heads_args_t* a, const HeadPlan& pl, HeadsParams& p) {
  const int64_t tokens = a->batch * a->seq;
  auto set = [&](int i, const void* x, const void* w, int heads, const skg_head_strides_t& sx) {
    HeadSet& s = p.set[i];
    s = HeadSet{};
    s.x = static_cast<const char*>(x);
    s.w = static_cast<const char*>(w);
    s.sx = {sx.batch, sx.token, sx.head};
    s.heads = heads;
    s.items = (uint32_t)pl.items[i];
    s.blocks = (uint32_t)pl.blocks[i];
    s.div = make_fastdiv((uint32_t)std::max<int64_t>(1, ceil_div(heads, pl.u)));
  };
  set(0, a->q, a->weight_q, a->heads_q, a->q_strides);
  set(1, a->k, a->weight_k, a->heads_k, a->k_strides);
  p.cos = a->cos;
  p.sin = a->sin;
  p.pos = a->positions;
  p.pos0 = a->pos0;
  p.pos64 = a->pos_bits == 64;
  p.table = (int)a->table_rows;
  p.half = a->rope_dim / 2;
  p.D = a->head_dim;
  p.pairs = a->style == SKG_ROPE_PAIRS;
  p.w_f32 = a->dtype_w == SKG_F32;
  p.seq = (int)a->seq;
  p.div_seq = make_fastdiv((uint32_t)std::max<int64_t>(1, a->seq));
  p.eps = a->eps;
  p.inv_d = 1.f / (float)a->head_dim;
  if (tokens == 0) p.seq = 1;
  const size_t es = elem_bytes(a->dtype), ws = elem_bytes(a->dtype_w);
  for (int i = 0; i < 2; ++i) {
    if (!pl.items[i]) continue;
    if (!p.set[i].x) return unsupported("null q or k");
    if (!aligned_to(p.set[i].x, es) || !aligned_to(p.set[i].w, ws)) return unsupported("pointers must be aligned to their elements");
  }
  if (a->rope_dim && (pl.items[0] || pl.items[1])) {
    if (!a->cos || !a->sin) return unsupported("a rotation needs its cos and sin tables");
    if (a->table_rows <= 0 || a->table_rows > INT32_MAX) return unsupported("table_rows must be positive and within 32 bits");
    if (!aligned_to(a->cos, 4) || !aligned_to(a->sin, 4) || !aligned_to(a->positions, a->pos_bits / 8))
      return unsupported("pointers must be aligned to their elements");
  }
  return SKG_OK;
}

template <int U, class F>
void by_heads(const skg_heads_args_t* a, const HeadPlan& pl, F&& f) {
  const int dtype = a->dtype;
  const bool plain = a->head_dim % 8 == 0 && a->rope_dim % (a->style == SKG_ROPE_PAIRS ? 8 : 16) == 0;
  auto by_plain = [&](auto dt, auto lanes, auto u) {
    if (plain)
      f(dt, lanes, u, std::true_type{});
    else
      f(dt, lanes, u, std::false_type{});
  };
  auto by_u = [&](auto dt, auto lanes) {
    if (pl.u == U)
      by_plain(dt, lanes, std::integral_constant<int, U>{});
    else
      by_plain(dt, lanes, std::integral_constant<int, 1>{});
  };
  auto by_lanes = [&](auto dt) {
    if (pl.lanes == 8)
      by_u(dt, std::integral_constant<int, 8>{});
    else if (pl.lanes == 16)
      by_u(dt, std::integral_constant<int, 16>{});
    else if (pl.lanes == 32)
      by_u(dt, std::integral_constant<int, 32>{});
    else
      by_u(dt, std::integral_constant<int, 64>{});
  };
  if (dtype == SKG_F16)
    by_lanes(std::integral_constant<int, DT_F16>{});
  else if (dtype == SKG_BF16)
    by_lanes(std::integral_constant<int, DT_BF16>{});
  else
    by_lanes(std::integral_constant<int, DT_F32>{});
}

int run_heads(const skg_heads_args_t* a, hipStream_t st) {
  int rc = check_heads(a);
  if (rc) return rc;
  const HeadPlan pl = plan_heads(a, false);
  HeadsParams p;
  rc = fill_heads(a, pl, p);
  if (rc) return rc;
  const int64_t blocks = pl.blocks[0] + pl.blocks[1];
  if (blocks == 0) return SKG_OK;
  const size_t es = elem_bytes(a->dtype);
  if ((pl.items[0] && !a->yq) || (pl.items[1] && !a->yk)) return unsupported("null yq or yk");
  if (!aligned_to(a->yq, es) || !aligned_to(a->yk, es)) return unsupported("pointers must be aligned to their elements");
  if (blocks * kHeadThreads > int64_t(kMostThreads)) return unsupported("too many heads for one launch");
  int cus = 0;
  rc = check_device(&cus);
  if (rc) return rc;
  p.set[0].y = static_cast<char*>(a->yq);
  p.set[0].sy = {a->yq_strides.batch, a->yq_strides.token, a->yq_strides.head};
  p.set[1].y = static_cast<char*>(a->yk);
  p.set[1].sy = {a->yk_strides.batch, a->yk_strides.token, a->yk_strides.head};
  by_heads<4>(a, pl, [&](auto dt, auto lanes, auto u, auto) {
    hipLaunchKernelGGL((heads_kernel<decltype(dt)::value, decltype(lanes)::value, decltype(u)::value>),
                       dim3((unsigned)blocks), dim3(kHeadThreads), 0, st, p);
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return hip_failure(std::string("launch: ") + hipGetErrorString(e));
  return SKG_OK;
}

size_t heads_bwd_bytes(const skg_heads_args_t* a, const HeadPlan& pl) {
  return ((a->dwq ? pl.blocks[0] : 0) + (a->dwk ? pl.blocks[1] : 0)) * size_t(a->head_dim) * 4;
}

// out, launched: what the call takes is wanted, and a workspace too small for
// it is not an error but leaves the call undone.
int run_heads_bwd(const skg_heads_args_t* a, void* ws, size_t ws_bytes, hipStream_t st, size_t* out = nullptr,
                  int32_t* launched = nullptr) {
  int rc = check_heads(a);
  if (rc) return rc;
  const HeadPlan pl = plan_heads(a, true);
  HeadsParams p;
  rc = fill_heads(a, pl, p);
  if (rc) return rc;
  const size_t es = elem_bytes(a->dtype);
  if ((pl.items[0] && !a->dyq) || (pl.items[1] && !a->dyk)) return unsupported("null dyq or dyk");
  if (!aligned_to(a->yq, es) || !aligned_to(a->yk, es) || !aligned_to(a->dyq, es) || !aligned_to(a->dyk, es) ||
      !aligned_to(a->dwq, 4) || !aligned_to(a->dwk, 4))
    return unsupported("pointers must be aligned to their elements");
  const size_t need = heads_bwd_bytes(a, pl);
  if (out) *out = need;
  if (launched) {
    *launched = need <= ws_bytes;
    if (!*launched) return SKG_OK;
  }
  if (need > ws_bytes) return unsupported("workspace too small for this call");
  if (need && (!ws || !aligned_to(ws, 16))) return unsupported("workspace must be 16-byte aligned device memory");
  HeadDw d{};
  float* part = static_cast<float*>(ws);
  for (int i = 0; i < 2; ++i) {
    HeadSet& s = p.set[i];
    const skg_head_strides_t &sy = i ? a->yk_strides : a->yq_strides, &sd = i ? a->dyk_strides : a->dyq_strides;
    s.y = static_cast<char*>(i ? a->yk : a->yq);
    s.dy = static_cast<const char*>(i ? a->dyk : a->dyq);
    s.sy = {sy.batch, sy.token, sy.head};
    s.sdy = {sd.batch, sd.token, sd.head};
    d.dw[i] = i ? a->dwk : a->dwq;
    if (!d.dw[i]) {
      // Without dw or dx there is nothing to do.
      if (!s.y) s.blocks = s.items = 0;
      continue;
    }
    s.partial = part;
    d.partial[i] = part;
    d.blocks[i] = (int)s.blocks;
    part += (size_t)s.blocks * a->head_dim;
  }
  const unsigned blocks = p.set[0].blocks + p.set[1].blocks;
  if (!blocks && !d.dw[0] && !d.dw[1]) return SKG_OK;
  int cus = 0;
  rc = check_device(&cus);
  if (rc) return rc;
  hipError_t e;
  if (blocks) {
    by_heads<2>(a, pl, [&](auto dt, auto lanes, auto u, auto plain) {
      hipLaunchKernelGGL((heads_bwd_kernel<decltype(dt)::value, decltype(lanes)::value, decltype(u)::value, decltype(plain)::value>), dim3(blocks),
                         dim3(kHeadThreads), 0, st, p);
    });
    e = hipGetLastError();
    if (e != hipSuccess) return hip_failure(std::string("launch: ") + hipGetErrorString(e));
  }
  if (d.dw[0] || d.dw[1]) {
    hipLaunchKernelGGL(heads_dw_kernel, dim3((unsigned)ceil_div(a->head_dim, 32), 2), dim3(32 * kHeadRuns), 0, st, d, (int)a->head_dim);
    e = hipGetLastError();
    if (e != hipSuccess) return hip_failure(std::string("launch: ") + hipGetErrorString(e));
  }
  return SKG_OK;
}

template <class F>
int guarded(F&& f) {
  try {
    clear_error();
    return f();
  } catch (const std::exception& ex) {
    return hip_failure(std::string("exception: ") + ex.what());
  } catch (...) {
    return hip_failure("unknown exception");
  }
}

}  // namespace
}  // namespace skg

using namespace skg;

extern "C" {

int skg_run_qknorm_rope(const skg_heads_args_t* a, void* stream) {
  return guarded([&] { return run_heads(a, static_cast<hipStream_t>(stream)); });
}

int skg_qknorm_rope_bwd_workspace_bytes(const skg_heads_args_t* a, size_t* out) {
  return guarded([&] {
    const int rc = check_heads(a);
    if (rc) return rc;
    if (!out) return unsupported("null output");
    *out = heads_bwd_bytes(a, plan_heads(a, true));
    return SKG_OK;
  });
}

int skg_run_qknorm_rope_bwd(const skg_heads_args_t* a, void* ws, size_t ws_bytes, void* stream) {
  return guarded([&] { return run_heads_bwd(a, ws, ws_bytes, static_cast<hipStream_t>(stream)); });
}

int skg_plan_run_qknorm_rope_bwd(const skg_heads_args_t* a, void* ws, size_t ws_bytes, void* stream, size_t* need,
                                 int32_t* launched) {
  return guarded([&] {
    if (!need || !launched) return unsupported("null output");
    *launched = 0;
    return run_heads_bwd(a, ws, ws_bytes, static_cast<hipStream_t>(stream), need, launched);
  });
}

}  // extern "C"
