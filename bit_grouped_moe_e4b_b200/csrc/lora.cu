// Low-rank adapters of many groups of rows beside a shared projection, and
// their gradients. Positions p of group g (offsets[g] <= p < offsets[g+1]) with
// rows i = row ? row[p] : p, adapters A_g [r, K], B_g [N, r], weight w_g:
//   forward    s[p] = A_g x_i,  y_i = base_i + w_g B_g s[p]   (h_i = act(y_i))
//   backward   t[p] = w_g B_g^T dy_i,  dx_i = dx_base_i + A_g^T t[p]
//              dA_g = sum_p t[p] x_i^T,  dB_g = w_g sum_p dy_i s[p]^T
// With r <= 64 every product has far fewer operations than its rows have bytes
// to move (2 r FLOP per bf16 value of x, y, dy or dx), so the kernels are built
// around reading and writing those rows once, straight between HBM and the
// registers of mma.sync.m16n8k16 fragments: a fragment's place in the
// contracted (or output) dimension is free as long as both operands agree, so
// each lane's eight consecutive bf16 values (one 16-byte access) are dealt to
// the fragment slots that the lane owns, and no tile passes through shared
// memory on its way to the tensor cores.
//
// Numbers: x, y, dy, A and B enter the MMAs as they are (bf16); sums are fp32.
// The fp32 intermediates s and t enter a second MMA as two bf16 terms hi + lo
// (hi = bf16(v), lo = bf16(v - hi)), i.e. with 16 bits and more of mantissa,
// so that fp32 gradients keep a relative error near 2^-17 per term. All
// reductions run in an order that depends on the sizes alone.
#include "adapters.h"
#include "common.cuh"

namespace e4b {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// ------------------------------------------------------------ small helpers
E4B_DEV void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

E4B_DEV float2 unpack2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// (a, b) as bf16 pairs hi + lo; an infinite or NaN value has no second term.
E4B_DEV void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(a, b);
  const float2 h = unpack2(hi);
  const float la = fabsf(h.x) < INFINITY ? a - h.x : 0.f;
  const float lb = fabsf(h.y) < INFINITY ? b - h.y : 0.f;
  lo = pack_bf16x2(la, lb);
}

E4B_DEV uint4 ldg16(const uint16_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }
E4B_DEV uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Pieces of up to `piece` positions that the groups' rows are cut into, in
// group order. Of groups with several pieces each piece also has a slot, in
// the same order: at most 2 * (R_max / piece) slots, unless the offsets are no
// prefix sums (pieces past that bound are left out).
struct Piece {
  int g;          // -1: no such piece
  int32_t row0;   // first position
  int32_t n;      // positions
  int32_t pieces; // of the group
  int32_t slot;   // of this piece (pieces > 1)
};

// By one warp; the same answer in every lane. offsets outside [0, R_max] are
// clamped, so that no position outside the row buffers is ever formed.
E4B_DEV Piece find_piece(const int64_t* __restrict__ offsets, int G, int64_t R_max, int piece, int index) {
  const int lane = threadIdx.x & 31;
  int run = 0, slots = 0;
  for (int base = 0; base < G; base += 32) {
    const int g = base + lane;
    int64_t beg = 0, end = 0;
    if (g < G) {
      beg = min(max(__ldg(offsets + g), int64_t(0)), R_max);
      end = min(max(__ldg(offsets + g + 1), int64_t(0)), R_max);
    }
    const int n = end > beg ? int(end - beg) : 0;
    const int np = (n + piece - 1) / piece;
    const int ns = np > 1 ? np : 0;
    int incl = np, sincl = ns;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d), w = __shfl_up_sync(0xffffffffu, sincl, d);
      if (lane >= d) {
        incl += v;
        sincl += w;
      }
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, run + incl > index);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const int k = index - (run + incl - np);  // in the source lane: which of the group's pieces
      Piece t;
      t.g = base + src;
      t.row0 = __shfl_sync(0xffffffffu, int(beg) + k * piece, src);
      t.n = __shfl_sync(0xffffffffu, min(piece, n - k * piece), src);
      t.pieces = __shfl_sync(0xffffffffu, np, src);
      t.slot = __shfl_sync(0xffffffffu, slots + sincl - ns + k, src);
      return t;
    }
    run += __shfl_sync(0xffffffffu, incl, 31);
    slots += __shfl_sync(0xffffffffu, sincl, 31);
  }
  return Piece{-1, 0, 0, 0, 0};
}

// The row of position p, or -1 where the map points outside the rows.
E4B_DEV int32_t row_of(const int32_t* __restrict__ row, int64_t rows, int32_t p) {
  if (!row) return p;
  const int32_t i = __ldg(row + p);
  return i >= 0 && i < rows ? i : -1;
}

// CTA b of a flat grid: column block b % blocks of piece b / blocks (the
// pieces may pass the 65535 that the grid's second dimension holds).
struct FlatBlock {
  int col, piece;
};
E4B_DEV FlatBlock flat_block(int blocks) {
  const int p = int(blockIdx.x) / blocks;
  return FlatBlock{int(blockIdx.x) - p * blocks, p};
}

struct Adapters {
  const uint16_t* a;  // [G, r, K]
  const uint16_t* b;  // [G, N, r]
  const float* scale;
  const int64_t* offsets;
  const int32_t* row;
  int64_t rows;
  int64_t N, K, R_max;
  int G, r;
};

E4B_DEV float weight(const Adapters& d, int g) { return d.scale ? __ldg(d.scale + g) : 1.f; }

// -------------------------------------------------------- forward: s = x A^T
// A CTA takes 32 positions of a group and a slice of K; its warps split the
// slice in 32-wide chunks (together 512 bytes of every row at a time) and
// their sums meet in shared memory. A lane reads eight consecutive k of rows
// lane / 4 and lane / 4 + 8 (+ 16 ...) and the same k of A's rows: two MMA
// k-steps. JT: 8-row tiles of A (r <= 8 JT).
constexpr int kShrinkRows = 32;

template <int JT>
__global__ void __launch_bounds__(kThreads, 2)
shrink_kernel(Adapters d, const uint16_t* __restrict__ x, int64_t ld_x, int kslices, float* __restrict__ out) {
  constexpr int MT = kShrinkRows / 16;
  constexpr int JR = JT > 2 ? 2 : JT;  // A tiles that are reduced together
  __shared__ float red[kWarps][kShrinkRows][8 * JR];
  grid_dependency_wait();
  grid_launch_dependents();
  const Piece t = find_piece(d.offsets, d.G, d.R_max, kShrinkRows, blockIdx.x);
  if (t.g < 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q = lane & 3, rr = lane >> 2;
  const uint16_t* xr[2 * MT];
#pragma unroll
  for (int i = 0; i < 2 * MT; ++i) {
    const int m = rr + 8 * i;
    const int32_t at = m < t.n ? row_of(d.row, d.rows, t.row0 + m) : -1;
    xr[i] = at >= 0 ? x + int64_t(at) * ld_x : nullptr;
  }
  const uint16_t* ag = d.a + int64_t(t.g) * d.r * d.K;
  float acc[MT][JT][4] = {};
  const int64_t chunks = (d.K + 31) / 32;
#pragma unroll 2
  for (int64_t c = int64_t(blockIdx.y) * kWarps + warp; c < chunks; c += int64_t(kslices) * kWarps) {
    const int64_t k = c * 32 + 8 * q;
    const bool in = k < d.K;
    uint4 xv[2 * MT], av[JT];
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) xv[i] = in && xr[i] ? ldg16(xr[i] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < JT; ++j) {
      const int jr = 8 * j + rr;
      av[j] = in && jr < d.r ? ldg16(ag + int64_t(jr) * d.K + k) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < JT; ++j)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        mma_bf16(acc[m][j], xv[2 * m].x, xv[2 * m + 1].x, xv[2 * m].y, xv[2 * m + 1].y, av[j].x, av[j].y);
        mma_bf16(acc[m][j], xv[2 * m].z, xv[2 * m + 1].z, xv[2 * m].w, xv[2 * m + 1].w, av[j].z, av[j].w);
      }
  }
  float* dst = out + int64_t(blockIdx.y) * d.R_max * d.r;
#pragma unroll
  for (int j0 = 0; j0 < JT; j0 += JR) {
    if (j0) __syncthreads();
#pragma unroll
    for (int j = 0; j < JR; ++j)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        float* w0 = &red[warp][16 * m + rr][8 * j + 2 * q];
        float* w1 = &red[warp][16 * m + rr + 8][8 * j + 2 * q];
        w0[0] = acc[m][j0 + j][0];
        w0[1] = acc[m][j0 + j][1];
        w1[0] = acc[m][j0 + j][2];
        w1[1] = acc[m][j0 + j][3];
      }
    __syncthreads();
    for (int i = threadIdx.x; i < kShrinkRows * 8 * JR; i += kThreads) {
      const int m = i / (8 * JR), j = 8 * j0 + i % (8 * JR);
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += red[w][m][i % (8 * JR)];
      if (m < t.n && j < d.r) dst[int64_t(t.row0 + m) * d.r + j] = sum;
    }
  }
}

// ------------------------------------------- forward: y = base + w s B^T
// A warp owns two strips of 32 columns (adjacent, or a gate and an up strip),
// keeps its columns of B in registers and walks the 16-position tiles of a
// piece. Column c of n8-tile i of a strip is the strip's column
// 8 (c / 2) + 2 i + c % 2, so that a lane's results are eight consecutive
// columns: one 16-byte access to base, y and h.
struct Expand {
  const uint16_t* base;
  int64_t ld_base;
  uint16_t* y;
  int64_t ld_y;
  uint16_t* h;
  int64_t ld_h;
  const float* s;  // [kslices][R_max][r]
  int kslices;
  float* s_out;    // the slices' sum, written by the first columns' warps; or null
  int col_blocks;
  int act;
  float alpha, limit;
};

constexpr int kExpandRows = 128;  // positions of a piece

enum { kGluNone = 0, kGluHalves = 1, kGluInterleaved = 2 };

E4B_DEV void add8(float (&v)[8], uint4 w) {
  const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2(q[i]);
    v[2 * i] += f.x;
    v[2 * i + 1] += f.y;
  }
}

E4B_DEV uint4 pack8(const float (&a)[8]) {
  return make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]),
                    pack_bf16x2(a[6], a[7]));
}

template <int JT, int GLU>
__global__ void __launch_bounds__(kThreads, JT > 4 ? 1 : 2)
expand_kernel(Adapters d, Expand e) {
  constexpr int KS = (JT + 1) / 2;  // MMA k-steps over the rank
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q = lane & 3, rr = lane >> 2;
  const FlatBlock fb = flat_block(e.col_blocks);
  const int64_t block_col = (int64_t(fb.col) * kWarps + warp) * (GLU == kGluHalves ? 32 : 64);
  const int64_t half = d.N / 2;
  int64_t col0[2];  // first column of the strips
  col0[0] = block_col;
  col0[1] = GLU == kGluHalves ? half + block_col : block_col + 32;
  const int64_t limit[2] = {GLU == kGluHalves ? half : d.N, d.N};
  grid_launch_dependents();
  const Piece t = find_piece(d.offsets, d.G, d.R_max, kExpandRows, fb.piece);
  if (t.g < 0) return;

  // B does not come from the launch before this one, which has itself waited
  // for all earlier work
  uint32_t bf[2][4][KS][2];
  const uint16_t* bg = d.b + int64_t(t.g) * d.N * d.r;
#pragma unroll
  for (int st = 0; st < 2; ++st)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t n = col0[st] + 8 * (rr >> 1) + 2 * i + (rr & 1);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int j = 16 * ks + 4 * q;
        uint2 v = make_uint2(0, 0);
        if (n < limit[st] && j < d.r) v = __ldg(reinterpret_cast<const uint2*>(bg + n * d.r + j));
        bf[st][i][ks][0] = v.x;
        bf[st][i][ks][1] = v.y;
      }
    }
  const float w = weight(d, t.g);
  grid_dependency_wait();

  const int64_t c[2] = {col0[0] + 8 * q, col0[1] + 8 * q};
  const bool in[2] = {c[0] < limit[0], c[1] < limit[1]};
  const bool writes_s = e.s_out && fb.col == 0 && warp == 0;
  for (int m0 = 0; m0 < t.n; m0 += 16) {
    int32_t pos[2], at[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int m = m0 + rr + 8 * i;
      pos[i] = m < t.n ? t.row0 + m : -1;
      at[i] = pos[i] >= 0 ? row_of(d.row, d.rows, pos[i]) : -1;
    }
    uint4 bv[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int st = 0; st < 2; ++st)
        bv[i][st] = e.base && at[i] >= 0 && in[st]
                        ? *reinterpret_cast<const uint4*>(e.base + int64_t(at[i]) * e.ld_base + c[st])
                        : make_uint4(0, 0, 0, 0);
    float acc[2][4][4] = {};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int j = 16 * ks + 4 * q;
      uint32_t hi[2][2], lo[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (pos[i] >= 0 && j < d.r) {
          const float* sp = e.s + int64_t(pos[i]) * d.r + j;
          for (int k = 0; k < e.kslices; ++k) {
            const float4 z = *reinterpret_cast<const float4*>(sp + int64_t(k) * d.R_max * d.r);
            v.x += z.x;
            v.y += z.y;
            v.z += z.z;
            v.w += z.w;
          }
          if (writes_s) *reinterpret_cast<float4*>(e.s_out + int64_t(pos[i]) * d.r + j) = v;
        }
        split2(w * v.x, w * v.y, hi[i][0], lo[i][0]);
        split2(w * v.z, w * v.w, hi[i][1], lo[i][1]);
      }
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          mma_bf16(acc[st][i], hi[0][0], hi[1][0], hi[0][1], hi[1][1], bf[st][i][ks][0], bf[st][i][ks][1]);
          mma_bf16(acc[st][i], lo[0][0], lo[1][0], lo[0][1], lo[1][1], bf[st][i][ks][0], bf[st][i][ks][1]);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (at[i] < 0) continue;
      float v[2][8];
#pragma unroll
      for (int st = 0; st < 2; ++st) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[st][2 * k] = acc[st][k][2 * i];
          v[st][2 * k + 1] = acc[st][k][2 * i + 1];
        }
        if (e.base) add8(v[st], bv[i][st]);
        if (e.y && in[st]) *reinterpret_cast<uint4*>(e.y + int64_t(at[i]) * e.ld_y + c[st]) = pack8(v[st]);
      }
      if constexpr (GLU == kGluHalves) {
        float h[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) h[k] = glu_act(e.act, v[0][k], v[1][k], e.alpha, e.limit);
        if (in[0]) *reinterpret_cast<uint4*>(e.h + int64_t(at[i]) * e.ld_h + c[0]) = pack8(h);
      } else if constexpr (GLU == kGluInterleaved) {
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          float h[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) h[k] = glu_act(e.act, v[st][2 * k], v[st][2 * k + 1], e.alpha, e.limit);
          if (in[st])
            *reinterpret_cast<uint2*>(e.h + int64_t(at[i]) * e.ld_h + c[st] / 2) =
                make_uint2(pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3]));
        }
      }
    }
  }
}

// ------------------------------------------------------------- backward
// Both passes walk a piece of a group's positions 16 at a time, a warp owning
// WC columns of the rows it reads (dy, or x and dx). The weight gradients
// contract over positions: a lane reads 8 (WC / 8) consecutive columns of
// positions 4 q .. 4 q + 3 and deals them, two positions a register, to the B
// operands of WC / 8 MMAs; the A operand is s or t transposed. CTAs stage
// s or t of 64 positions in shared memory in the order of the MMA fragments.
constexpr int kStage = 64;
constexpr int kStageTiles = kStage / 16;

// A operand of the weight gradient: element (j, position), j = 16 mt + lane / 4
// (+ 8), positions 4 q .. 4 q + 3; hi and lo terms.
template <int JT>
struct GradFrags {
  static constexpr int MT = (JT + 1) / 2;
  uint4 f[kStageTiles][MT][2][32];
};
// A operand of the expansion: element (position, j), position = lane / 4 (+ 8),
// j = 16 ks + 4 q .. + 3; hi and lo terms.
template <int JT>
struct RowFrags {
  static constexpr int KS = (JT + 1) / 2;
  uint4 f[kStageTiles][KS][2][32];
};

// v[m][j] of 64 positions: the fp32 value of position m0 + m, zero past the
// piece or the rank.
E4B_DEV float value_at(const float* __restrict__ v, int r, const Piece& t, const int32_t* at, int m0, int m, int j) {
  return at[m] >= 0 && j < r ? v[int64_t(t.row0 + m0 + m) * r + j] : 0.f;
}

template <int JT>
E4B_DEV void stage_grad(GradFrags<JT>& out, const float* __restrict__ v, int r, float w, const Piece& t,
                        const int32_t* at, int m0) {
  constexpr int MT = GradFrags<JT>::MT;
  for (int i = threadIdx.x; i < kStageTiles * MT * 32; i += kThreads) {
    const int lane = i & 31, mt = (i >> 5) % MT, tile = (i >> 5) / MT;
    const int j = 16 * mt + (lane >> 2), m = 16 * tile + 4 * (lane & 3);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // a0..a3: (j, m), (j + 8, m), (j, m + 2), (j + 8, m + 2)
      const int jj = j + 8 * (k & 1), mm = m + 2 * (k >> 1);
      split2(w * value_at(v, r, t, at, m0, mm, jj), w * value_at(v, r, t, at, m0, mm + 1, jj), hi[k], lo[k]);
    }
    out.f[tile][mt][0][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    out.f[tile][mt][1][lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

template <int JT>
E4B_DEV void stage_rows(RowFrags<JT>& out, const float* __restrict__ v, int r, const Piece& t, const int32_t* at,
                        int m0) {
  constexpr int KS = RowFrags<JT>::KS;
  for (int i = threadIdx.x; i < kStageTiles * KS * 32; i += kThreads) {
    const int lane = i & 31, ks = (i >> 5) % KS, tile = (i >> 5) / KS;
    const int m = 16 * tile + (lane >> 2), j = 16 * ks + 4 * (lane & 3);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // a0..a3: (m, j), (m + 8, j), (m, j + 2), (m + 8, j + 2)
      const int mm = m + 8 * (k & 1), jj = j + 2 * (k >> 1);
      split2(value_at(v, r, t, at, m0, mm, jj), value_at(v, r, t, at, m0, mm, jj + 1), hi[k], lo[k]);
    }
    out.f[tile][ks][0][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    out.f[tile][ks][1][lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

// The lane's columns of positions 4 q .. 4 q + 3, as 32-bit words of two
// columns (WC / 16 words a position).
template <int WC>
struct GradLoad {
  uint32_t w[4][WC / 16];
};

template <int WC>
E4B_DEV void load_grad(GradLoad<WC>& v, const uint16_t* __restrict__ p, int64_t ld, const int32_t* at, int m, int64_t c,
                       bool in) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int32_t i = at[m + k];
    const bool on = in && i >= 0;
    const uint16_t* src = p + (on ? int64_t(i) * ld + c : 0);
    if constexpr (WC == 64) {
      const uint4 z = on ? ldg16(src) : make_uint4(0, 0, 0, 0);
      v.w[k][0] = z.x;
      v.w[k][1] = z.y;
      v.w[k][2] = z.z;
      v.w[k][3] = z.w;
    } else {
      const uint2 z = on ? __ldg(reinterpret_cast<const uint2*>(src)) : make_uint2(0, 0);
      v.w[k][0] = z.x;
      v.w[k][1] = z.y;
    }
  }
}

// acc[mt][i] += (values of 16 positions)^T (rows): columns i + (WC / 8) n of
// the warp's strip, n = the MMA's column.
template <int JT, int WC>
E4B_DEV void grad_mma(float (&acc)[(JT + 1) / 2][WC / 8][4], const GradFrags<JT>& frags, int tile,
                      const GradLoad<WC>& v) {
  const int lane = threadIdx.x & 31;
  uint32_t b[WC / 8][2];
#pragma unroll
  for (int i = 0; i < WC / 8; ++i) {
    const uint32_t sel = i & 1 ? 0x7632 : 0x5410;
    b[i][0] = prmt(v.w[0][i / 2], v.w[1][i / 2], sel);
    b[i][1] = prmt(v.w[2][i / 2], v.w[3][i / 2], sel);
  }
#pragma unroll
  for (int mt = 0; mt < (JT + 1) / 2; ++mt)
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const uint4 f = frags.f[tile][mt][part][lane];
#pragma unroll
      for (int i = 0; i < WC / 8; ++i) mma_bf16(acc[mt][i], f.x, f.y, f.z, f.w, b[i][0], b[i][1]);
    }
}

E4B_DEV void stage_positions(int32_t* at, const Adapters& d, const Piece& t, int m0) {
  for (int i = threadIdx.x; i < kStage; i += kThreads)
    at[i] = m0 + i < t.n ? row_of(d.row, d.rows, t.row0 + m0 + i) : -1;
}

struct BackDy {
  const uint16_t* dy;
  int64_t ld_dy;
  const float* s;   // [R_max, r]
  float* db;        // [G, N, r] or null
  float* db_part;   // [slots][N][r]
  float* t_part;    // [column blocks][R_max][r] or null
  int col_blocks;
  int piece;
  int slots;  // of the parts
  int accumulate;
};

// Pass over dy: dB of the piece, and the column block's part of t. The rank's
// index j of tile jt is JT n + jt (n the MMA's column), so that a lane's t of
// a position is 2 JT consecutive values.
template <int JT, int WC>
__global__ void __launch_bounds__(kThreads, JT > 2 ? 1 : 2)
back_dy_kernel(Adapters d, BackDy e) {
  constexpr int KC = WC / 16;  // MMA k-steps over the warp's columns
  extern __shared__ __align__(16) uint8_t smem[];
  GradFrags<JT>& frags = *reinterpret_cast<GradFrags<JT>*>(smem);
  float* red = reinterpret_cast<float*>(smem + sizeof(GradFrags<JT>));  // [2][kWarps][16][8 JT]
  __shared__ int32_t at[kStage];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q = lane & 3, rr = lane >> 2;
  grid_dependency_wait();
  grid_launch_dependents();
  const FlatBlock fb = flat_block(e.col_blocks);
  const Piece t = find_piece(d.offsets, d.G, d.R_max, e.piece, fb.piece);
  if (t.g < 0 || (t.pieces > 1 && t.slot >= e.slots)) return;
  const int64_t col0 = (int64_t(fb.col) * kWarps + warp) * WC;
  const float w = weight(d, t.g);

  // B operand of t: columns (k) 8 q .. 8 q + 7 of each 32, j = JT rr + jt
  uint32_t bf[KC][JT][2];
  const uint16_t* bg = d.b + int64_t(t.g) * d.N * d.r;
#pragma unroll
  for (int ks = 0; ks < KC; ++ks)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int64_t n = col0 + 32 * (ks / 2) + 8 * q + 4 * (ks % 2) + 2 * half;
#pragma unroll
      for (int jt = 0; jt < JT; ++jt) {
        const int j = JT * rr + jt;
        uint32_t lo = 0, hi = 0;
        if (e.t_part && n < d.N && j < d.r) {  // N is a multiple of 8: n and n + 1 are in together
          lo = __ldg(bg + n * d.r + j);
          hi = __ldg(bg + (n + 1) * d.r + j);
        }
        bf[ks][jt][half] = lo | (hi << 16);
      }
    }

  const int64_t cg = col0 + (WC / 8) * rr;  // the lane's columns for dB
  const bool in_g = cg < d.N;
  float acc[(JT + 1) / 2][WC / 8][4] = {};
  int buf = 0;
  for (int m0 = 0; m0 < t.n; m0 += kStage) {
    __syncthreads();
    stage_positions(at, d, t, m0);
    __syncthreads();
    if (e.db) stage_grad<JT>(frags, e.s, d.r, w, t, at, m0);  // s may be null without db
    __syncthreads();
    const int tiles = min(kStageTiles, (t.n - m0 + 15) / 16);
    for (int tile = 0; tile < tiles; ++tile) {
      GradLoad<WC> v;
      if (e.db) load_grad<WC>(v, e.dy, e.ld_dy, at, 16 * tile + 4 * q, cg, in_g);
      uint4 x[2][KC / 2];
      if (e.t_part) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int32_t row = at[16 * tile + rr + 8 * i];
#pragma unroll
          for (int k = 0; k < KC / 2; ++k) {
            const int64_t c = col0 + 32 * k + 8 * q;
            x[i][k] = row >= 0 && c < d.N ? ldg16(e.dy + int64_t(row) * e.ld_dy + c) : make_uint4(0, 0, 0, 0);
          }
        }
      }
      if (e.db) grad_mma<JT, WC>(acc, frags, tile, v);
      if (e.t_part) {
        float ta[JT][4] = {};
#pragma unroll
        for (int k = 0; k < KC / 2; ++k)
#pragma unroll
          for (int jt = 0; jt < JT; ++jt) {
            mma_bf16(ta[jt], x[0][k].x, x[1][k].x, x[0][k].y, x[1][k].y, bf[2 * k][jt][0], bf[2 * k][jt][1]);
            mma_bf16(ta[jt], x[0][k].z, x[1][k].z, x[0][k].w, x[1][k].w, bf[2 * k + 1][jt][0], bf[2 * k + 1][jt][1]);
          }
        float* mine = red + ((buf * kWarps + warp) * 16) * (8 * JT);
#pragma unroll
        for (int jt = 0; jt < JT; ++jt)
#pragma unroll
          for (int k = 0; k < 4; ++k) mine[(rr + 8 * (k >> 1)) * (8 * JT) + (2 * q + (k & 1)) * JT + jt] = ta[jt][k];
        __syncthreads();
        for (int i = threadIdx.x; i < 16 * 8 * JT; i += kThreads) {
          const int m = i / (8 * JT), j = i % (8 * JT);
          float sum = 0.f;
#pragma unroll
          for (int k = 0; k < kWarps; ++k) sum += red[(buf * kWarps + k) * 16 * 8 * JT + i];
          const int mm = m0 + 16 * tile + m;
          if (mm < t.n && j < d.r) e.t_part[(int64_t(fb.col) * d.R_max + t.row0 + mm) * d.r + j] = w * sum;
        }
        buf ^= 1;
      }
    }
  }
  if (!e.db) return;
  const bool direct = t.pieces == 1;
  float* dst = direct ? e.db + int64_t(t.g) * d.N * d.r : e.db_part + int64_t(t.slot) * d.N * d.r;
  const bool add = direct && e.accumulate;
#pragma unroll
  for (int mt = 0; mt < (JT + 1) / 2; ++mt)
#pragma unroll
    for (int i = 0; i < WC / 8; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = 16 * mt + rr + 8 * (k >> 1);
        const int64_t n = col0 + (WC / 8) * (2 * q + (k & 1)) + i;
        if (j < d.r && n < d.N) {
          float* at_ = dst + n * d.r + j;
          *at_ = add ? *at_ + acc[mt][i][k] : acc[mt][i][k];
        }
      }
}

// t[p] = the column blocks' parts, in block order.
__global__ void __launch_bounds__(kThreads)
sum_parts_kernel(const float* __restrict__ part, int parts, int64_t n4, float* __restrict__ out) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t stride = int64_t(gridDim.x) * kThreads;
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < n4; i += stride) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int k = 0; k < parts; ++k) {
      const float4 v = reinterpret_cast<const float4*>(part)[int64_t(k) * n4 + i];
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    reinterpret_cast<float4*>(out)[i] = s;
  }
}

struct BackX {
  const uint16_t* x;
  int64_t ld_x;
  const float* t;   // [R_max, r]
  float* da;        // [G, r, K] or null
  float* da_part;   // [slots][r][K]
  const uint16_t* dx_base;
  int64_t ld_dx_base;
  uint16_t* dx;     // or null
  int64_t ld_dx;
  int col_blocks;
  int piece;
  int slots;  // of the parts
  int accumulate;
};

// Pass over x and dx: dA of the piece, and the rows of dx.
template <int JT, int WC>
__global__ void __launch_bounds__(kThreads, JT > 2 ? 1 : 2)
back_x_kernel(Adapters d, BackX e) {
  constexpr int KS = (JT + 1) / 2;
  constexpr int ST = WC / 32;  // strips of 32 columns
  extern __shared__ __align__(16) uint8_t smem[];
  GradFrags<JT>& gf = *reinterpret_cast<GradFrags<JT>*>(smem);
  RowFrags<JT>& rf = *reinterpret_cast<RowFrags<JT>*>(smem + sizeof(GradFrags<JT>));
  __shared__ int32_t at[kStage];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q = lane & 3, rr = lane >> 2;
  grid_dependency_wait();
  grid_launch_dependents();
  const FlatBlock fb = flat_block(e.col_blocks);
  const Piece t = find_piece(d.offsets, d.G, d.R_max, e.piece, fb.piece);
  if (t.g < 0 || (t.pieces > 1 && t.slot >= e.slots)) return;
  const int64_t col0 = (int64_t(fb.col) * kWarps + warp) * WC;

  // B operand of dx: j = 16 ks + 4 q .. + 3, the strips' columns as in expand_kernel
  uint32_t bf[ST][4][KS][2];
  const uint16_t* ag = d.a + int64_t(t.g) * d.r * d.K;
#pragma unroll
  for (int st = 0; st < ST; ++st) {
    const int64_t n = col0 + 32 * st + 8 * (rr >> 1);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int j = 16 * ks + 4 * q;
      uint4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        v[k] = e.dx && n < d.K && j + k < d.r ? ldg16(ag + int64_t(j + k) * d.K + n) : make_uint4(0, 0, 0, 0);
      const uint32_t sel = rr & 1 ? 0x7632 : 0x5410;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        bf[st][i][ks][0] = prmt(word(v[0], i), word(v[1], i), sel);
        bf[st][i][ks][1] = prmt(word(v[2], i), word(v[3], i), sel);
      }
    }
  }

  const int64_t cg = col0 + (WC / 8) * rr;
  const bool in_g = cg < d.K;
  float acc[(JT + 1) / 2][WC / 8][4] = {};
  for (int m0 = 0; m0 < t.n; m0 += kStage) {
    __syncthreads();
    stage_positions(at, d, t, m0);
    __syncthreads();
    if (e.da) stage_grad<JT>(gf, e.t, d.r, 1.f, t, at, m0);
    if (e.dx) stage_rows<JT>(rf, e.t, d.r, t, at, m0);
    __syncthreads();
    const int tiles = min(kStageTiles, (t.n - m0 + 15) / 16);
    for (int tile = 0; tile < tiles; ++tile) {
      GradLoad<WC> v;
      if (e.da) load_grad<WC>(v, e.x, e.ld_x, at, 16 * tile + 4 * q, cg, in_g);
      if (e.dx) {
        int32_t row[2];
        uint4 bv[2][ST];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          row[i] = at[16 * tile + rr + 8 * i];
#pragma unroll
          for (int st = 0; st < ST; ++st) {
            const int64_t c = col0 + 32 * st + 8 * q;
            bv[i][st] = e.dx_base && row[i] >= 0 && c < d.K
                            ? *reinterpret_cast<const uint4*>(e.dx_base + int64_t(row[i]) * e.ld_dx_base + c)
                            : make_uint4(0, 0, 0, 0);
          }
        }
        float o[ST][4][4] = {};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            const uint4 f = rf.f[tile][ks][part][lane];
#pragma unroll
            for (int st = 0; st < ST; ++st)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                mma_bf16(o[st][i], f.x, f.y, f.z, f.w, bf[st][i][ks][0], bf[st][i][ks][1]);
          }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int st = 0; st < ST; ++st) {
            const int64_t c = col0 + 32 * st + 8 * q;
            if (row[i] < 0 || c >= d.K) continue;
            float z[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              z[2 * k] = o[st][k][2 * i];
              z[2 * k + 1] = o[st][k][2 * i + 1];
            }
            if (e.dx_base) add8(z, bv[i][st]);
            *reinterpret_cast<uint4*>(e.dx + int64_t(row[i]) * e.ld_dx + c) = pack8(z);
          }
      }
      if (e.da) grad_mma<JT, WC>(acc, gf, tile, v);
    }
  }
  if (!e.da) return;
  const bool direct = t.pieces == 1;
  float* dst = direct ? e.da + int64_t(t.g) * d.r * d.K : e.da_part + int64_t(t.slot) * d.r * d.K;
  const bool add = direct && e.accumulate;
#pragma unroll
  for (int mt = 0; mt < (JT + 1) / 2; ++mt)
#pragma unroll
    for (int i = 0; i < WC / 8; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = 16 * mt + rr + 8 * (k >> 1);
        const int64_t n = col0 + (WC / 8) * (2 * q + (k & 1)) + i;
        if (j < d.r && n < d.K) {
          float* at_ = dst + int64_t(j) * d.K + n;
          *at_ = add ? *at_ + acc[mt][i][k] : acc[mt][i][k];
        }
      }
}

// The gradients of groups whose rows were cut into several pieces (the parts'
// sum, in piece order) and of groups without rows (zero). n: values of a
// group's gradient.
__global__ void __launch_bounds__(kThreads)
finish_grads_kernel(const int64_t* __restrict__ offsets, int G, int64_t R_max, int piece_b, int piece_a,
                    int slots_b, int slots_a, const float* __restrict__ db_part, int64_t nb4, float* __restrict__ db,
                    const float* __restrict__ da_part, int64_t na4, float* __restrict__ da, int accumulate) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int g = blockIdx.y;
  // the slots of the groups before g, and g's pieces
  for (int side = 0; side < 2; ++side) {
    const int piece = side ? piece_a : piece_b;
    float* out = side ? da : db;
    const float* part = side ? da_part : db_part;
    const int64_t n4 = side ? na4 : nb4;
    if (!out) continue;
    int slots = 0, mine = 0;
    for (int base = 0; base <= g; base += 32) {
      const int k = base + lane;
      int np = 0;
      if (k <= g) {
        const int64_t beg = min(max(__ldg(offsets + k), int64_t(0)), R_max);
        const int64_t end = min(max(__ldg(offsets + k + 1), int64_t(0)), R_max);
        np = end > beg ? int((end - beg + piece - 1) / piece) : 0;
      }
      int before = k < g && np > 1 ? np : 0;
      int own = k == g ? np : 0;
#pragma unroll
      for (int m = 16; m; m >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, m);
        own += __shfl_xor_sync(0xffffffffu, own, m);
      }
      slots += before;
      mine += own;
    }
    if (mine == 1 || (mine == 0 && accumulate)) continue;
    mine = min(mine, (side ? slots_a : slots_b) - slots);
    float4* dst = reinterpret_cast<float4*>(out) + int64_t(g) * n4;
    const float4* src = reinterpret_cast<const float4*>(part) + int64_t(slots) * n4;
    const int64_t stride = int64_t(gridDim.x) * kThreads;
    for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < n4; i += stride) {
      float4 s = accumulate ? dst[i] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int k = 0; k < mine; ++k) {
        const float4 v = src[int64_t(k) * n4 + i];
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
      dst[i] = s;
    }
  }
}

// --------------------------------------------------------------- launches
int tiles_of_rank(int r) { return r <= 8 ? 1 : r <= 16 ? 2 : r <= 32 ? 4 : 8; }
int warp_cols(int jt) { return jt > 4 ? 32 : 64; }

int64_t pieces_bound(int64_t G, int64_t R_max, int64_t piece) {
  const int64_t full = R_max / piece;
  return full + (G < R_max ? G : R_max);
}

// K slices of the forward contraction: enough CTAs to fill the GPU when there
// are few rows, each with at least one 32-wide chunk a warp.
int forward_slices(int64_t G, int64_t K, int64_t R_max, int sms) {
  const int64_t tiles = pieces_bound(G, R_max, kShrinkRows);
  const int64_t most = (K + 32 * kWarps - 1) / (32 * kWarps);
  int64_t want = sms / (tiles > 0 ? tiles : 1);
  if (want > 16) want = 16;
  if (want > most) want = most;
  return int(want < 1 ? 1 : want);
}

struct BackPlan {
  int jt, wc;
  int64_t cb_n, cb_k;      // column blocks of dy and of x
  int piece_n, piece_k;    // positions of a piece, per pass
  int64_t slots_n, slots_k;
  size_t t_part, t, db_part, da_part, total;
};

// Positions of a piece: a few waves of CTAs over (pieces, column blocks), but
// no fewer than 16 r, so that the parts a piece writes and the last kernel
// reads (8 r bytes a column) stay below a quarter of the 2 bytes a position
// and column that it reads.
int back_piece(int64_t R_max, int64_t blocks, int r, int sms) {
  int64_t p = R_max * blocks / (int64_t(sms) * 8);
  if (p < 16 * r) p = 16 * r;
  if (p < 256) p = 256;
  if (p > 4096) p = 4096;
  return int((p + kStage - 1) / kStage * kStage);
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

BackPlan plan_backward(int64_t G, int r, int64_t N, int64_t K, int64_t R_max, int sms) {
  BackPlan p;
  p.jt = tiles_of_rank(r);
  p.wc = warp_cols(p.jt);
  p.cb_n = (N + kWarps * p.wc - 1) / (kWarps * p.wc);
  p.cb_k = (K + kWarps * p.wc - 1) / (kWarps * p.wc);
  p.piece_n = back_piece(R_max, p.cb_n, r, sms);
  p.piece_k = back_piece(R_max, p.cb_k, r, sms);
  p.slots_n = 2 * (R_max / p.piece_n);
  p.slots_k = 2 * (R_max / p.piece_k);
  size_t o = 0;
  p.t_part = o;  o = align256(o + size_t(p.cb_n) * R_max * r * 4);
  p.t = o;       o = align256(o + size_t(R_max) * r * 4);
  p.db_part = o; o = align256(o + size_t(p.slots_n) * N * r * 4);
  p.da_part = o; o = align256(o + size_t(p.slots_k) * K * r * 4);
  p.total = o;
  return p;
}

Adapters adapters_of(const e4b_lora_args& a) {
  return Adapters{a.a, a.b, a.scale, a.offsets, a.row, a.rows, a.N, a.K, a.R_max, a.G, a.r};
}

template <int JT>
cudaError_t forward(const e4b_lora_args& a, void* ws, cudaStream_t st, int sms, int* launches) {
  const Adapters d = adapters_of(a);
  const int slices = forward_slices(a.G, a.K, a.R_max, sms);
  float* s = a.s && slices == 1 ? a.s : static_cast<float*>(ws);
  const int tiles = int(pieces_bound(a.G, a.R_max, kShrinkRows));
  cudaError_t err = launch_dependent(shrink_kernel<JT>, dim3(tiles, slices), dim3(kThreads), 0, st, d, a.x, a.ld_x,
                                     slices, s);
  if (err != cudaSuccess) return err;
  *launches = 1;
  if (!a.y && !a.h && slices == 1) return cudaSuccess;  // s alone was asked for
  Expand e{a.base, a.ld_base, a.y, a.ld_y, a.h, a.ld_h, s, slices, slices > 1 ? a.s : nullptr, 0, a.activation,
           a.glu_alpha, a.glu_limit};
  const int glu = !a.h ? kGluNone : a.gate_up_layout == E4B_GATE_UP_INTERLEAVED ? kGluInterleaved : kGluHalves;
  const int64_t cols = glu == kGluHalves ? a.N / 2 : a.N, per = kWarps * (glu == kGluHalves ? 32 : 64);
  e.col_blocks = int((cols + per - 1) / per);
  const dim3 grid(unsigned(e.col_blocks * pieces_bound(a.G, a.R_max, kExpandRows)));
  auto kernel = glu == kGluNone ? expand_kernel<JT, kGluNone>
                : glu == kGluHalves ? expand_kernel<JT, kGluHalves> : expand_kernel<JT, kGluInterleaved>;
  *launches = 2;
  return launch_dependent(kernel, grid, dim3(kThreads), 0, st, d, e);
}

template <int JT, int WC>
cudaError_t backward(const e4b_lora_args& a, bool accumulate, void* ws, cudaStream_t st, int sms, int* launches) {
  const Adapters d = adapters_of(a);
  const BackPlan p = plan_backward(a.G, a.r, a.N, a.K, a.R_max, sms);
  uint8_t* base = static_cast<uint8_t*>(ws);
  const size_t smem_dy = sizeof(GradFrags<JT>) + size_t(2) * kWarps * 16 * 8 * JT * 4;
  const size_t smem_x = sizeof(GradFrags<JT>) + sizeof(RowFrags<JT>);
  // set on every call: the attribute belongs to the device that is current
  cudaError_t err = cudaFuncSetAttribute(back_dy_kernel<JT, WC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(smem_dy));
  if (err == cudaSuccess)
    err = cudaFuncSetAttribute(back_x_kernel<JT, WC>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem_x));
  if (err != cudaSuccess) return err;
  const bool wants_t = a.da || a.dx;
  float* t_part = reinterpret_cast<float*>(base + p.t_part);
  float* t = p.cb_n == 1 ? t_part : reinterpret_cast<float*>(base + p.t);
  float* db_part = reinterpret_cast<float*>(base + p.db_part);
  float* da_part = reinterpret_cast<float*>(base + p.da_part);
  const int acc = accumulate ? 1 : 0;
  *launches = 0;
  if (a.R_max > 0) {
    BackDy e{a.dy, a.ld_dy, a.s, a.db, db_part, wants_t ? t_part : nullptr, int(p.cb_n), p.piece_n, int(p.slots_n), acc};
    const dim3 grid(unsigned(p.cb_n * pieces_bound(a.G, a.R_max, p.piece_n)));
    err = launch_dependent(back_dy_kernel<JT, WC>, grid, dim3(kThreads), smem_dy, st, d, e);
    if (err != cudaSuccess) return err;
    ++*launches;
  }
  if (a.R_max > 0 && wants_t) {
    if (p.cb_n > 1) {
      const int64_t n4 = a.R_max * a.r / 4;
      int64_t g = (n4 + kThreads - 1) / kThreads;
      if (g > int64_t(sms) * 8) g = int64_t(sms) * 8;
      err = launch_dependent(sum_parts_kernel, dim3(unsigned(g)), dim3(kThreads), 0, st,
                             const_cast<const float*>(t_part), int(p.cb_n), n4, t);
      if (err != cudaSuccess) return err;
      ++*launches;
    }
    BackX e{a.x, a.ld_x, t, a.da, da_part, a.dx_base, a.ld_dx_base, a.dx, a.ld_dx, int(p.cb_k), p.piece_k, int(p.slots_k), acc};
    const dim3 grid(unsigned(p.cb_k * pieces_bound(a.G, a.R_max, p.piece_k)));
    err = launch_dependent(back_x_kernel<JT, WC>, grid, dim3(kThreads), smem_x, st, d, e);
    if (err != cudaSuccess) return err;
    ++*launches;
  }
  if (a.da || a.db) {
    const int64_t nb4 = a.N * a.r / 4, na4 = a.K * a.r / 4;
    const int64_t most = nb4 > na4 ? nb4 : na4;
    int64_t g = (most + kThreads * 4 - 1) / (kThreads * 4);
    if (g > 64) g = 64;
    err = launch_dependent(finish_grads_kernel, dim3(unsigned(g), unsigned(a.G)), dim3(kThreads), 0, st, a.offsets,
                           a.G, a.R_max, p.piece_n, p.piece_k, int(p.slots_n), int(p.slots_k),
                           const_cast<const float*>(db_part), nb4, a.db,
                           const_cast<const float*>(da_part), na4, a.da, acc);
    if (err != cudaSuccess) return err;
    ++*launches;
  }
  return cudaSuccess;
}

}  // namespace

size_t lora_workspace_bytes(int64_t G, int r, int64_t N, int64_t K, int64_t R_max, bool back, int sms) {
  if (back) return plan_backward(G, r, N, K, R_max, sms).total + 256;
  return align256(size_t(forward_slices(G, K, R_max, sms)) * size_t(R_max) * r * 4) + 256;
}

cudaError_t launch_lora(const e4b_lora_args& a, void* ws, cudaStream_t st, int sms, int* launches) {
  switch (tiles_of_rank(a.r)) {
    case 1: return forward<1>(a, ws, st, sms, launches);
    case 2: return forward<2>(a, ws, st, sms, launches);
    case 4: return forward<4>(a, ws, st, sms, launches);
    default: return forward<8>(a, ws, st, sms, launches);
  }
}

cudaError_t launch_lora_backward(const e4b_lora_args& a, bool accumulate, void* ws, cudaStream_t st, int sms,
                                 int* launches) {
  switch (tiles_of_rank(a.r)) {
    case 1: return backward<1, 64>(a, accumulate, ws, st, sms, launches);
    case 2: return backward<2, 64>(a, accumulate, ws, st, sms, launches);
    case 4: return backward<4, 64>(a, accumulate, ws, st, sms, launches);
    default: return backward<8, 32>(a, accumulate, ws, st, sms, launches);
  }
}

}  // namespace e4b
