// Low-rank adapters of many groups of rows beside a shared projection, and
// their gradients. Positions p of group g (offsets[g] <= p < offsets[g+1]) with
// rows i = row ? row[p] : p, adapters A_g [r, K], B_g [N, r], weight w_g:
//   forward    s[p] = A_g x_i,  y_i = base_i + w_g B_g s[p]   (h_i = act(y_i))
//   backward   t[p] = w_g B_g^T dy_i,  dx_i = dx_base_i + A_g^T t[p]
//              dA_g = sum_p t[p] x_i^T,  dB_g = w_g sum_p dy_i s[p]^T
// With r <= 64 every product has far fewer operations than its rows have bytes
// to move, so each of x, y, dy and dx is read or written once, and what counts
// is that these accesses keep coming. The contractions (s, t, dA, dB) run over
// tiles that TMA brings to the tcgen05 tensor cores (csrc/lora_tc.cu). Here are
// the expansions (y, dx), straight between HBM and the registers of
// mma.sync.m16n8k16 fragments: a fragment's place in the output dimension is
// free, so each lane's eight consecutive bf16 values (one 16-byte access) are
// dealt to the fragment slots that the lane owns and no tile of y passes
// through shared memory; and s of few rows, where the launch and the split of K
// over the GPU count and 128-row tiles would be empty.
//
// Numbers: x, y, dy, A and B enter the MMAs as they are (bf16); sums are fp32.
// The fp32 values s and t enter an expansion as three bf16 terms (24 bits of
// mantissa), so that y and dx are what fp32 products give up to their one
// rounding, also where base takes the products away again. All reductions run
// in an order that depends on the sizes alone.
#include "adapters.h"
#include "common.cuh"
#include "lora_tc.h"
#include "lora_terms.cuh"
#include "lora_walk.cuh"
#include "sm100.cuh"

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

E4B_DEV uint4 ldg16(const uint16_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }
E4B_DEV uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Piece `index` of the groups' rows, cut into pieces of up to `piece`
// positions in group order.
struct Piece {
  int g;          // -1: no such piece
  int32_t row0;   // first position
  int32_t n;      // positions
};

// By one warp; the same answer in every lane. A lane takes a strip of the
// groups, so that all offsets are in flight together. offsets outside
// [0, R_max] are clamped: no position outside the row buffers is ever formed.
E4B_DEV Piece find_piece(const int64_t* __restrict__ offsets, int G, int64_t R_max, int piece, int index) {
  const int lane = threadIdx.x & 31;
  const int strip = (G + 31) / 32;
  const int lo = min(lane * strip, G), hi = min(lo + strip, G);
  auto clamped = [&](int g) { return int(min(max(__ldg(offsets + g), int64_t(0)), R_max)); };
  int64_t mine = 0;
#pragma unroll 4
  for (int g = lo; g < hi; ++g) mine += (max(clamped(g + 1) - clamped(g), 0) + piece - 1) / piece;
  int64_t incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  const uint32_t hit = __ballot_sync(0xffffffffu, incl > index);
  Piece t{-1, 0, 0};
  if (!hit) return t;
  const int src = __ffs(hit) - 1;
  if (lane == src) {
    int64_t left = index - (incl - mine);
    for (int g = lo; g < hi; ++g) {
      const int beg = clamped(g), n = max(clamped(g + 1) - beg, 0), np = (n + piece - 1) / piece;
      if (left < np) {
        t = Piece{g, beg + int(left) * piece, min(piece, n - int(left) * piece)};
        break;
      }
      left -= np;
    }
  }
  t.g = __shfl_sync(0xffffffffu, t.g, src);
  t.row0 = __shfl_sync(0xffffffffu, t.row0, src);
  t.n = __shfl_sync(0xffffffffu, t.n, src);
  return t;
}

// The row of position p, or -1 where the map points outside the rows.
E4B_DEV int32_t row_of(const int32_t* __restrict__ row, int64_t rows, int32_t p) {
  if (!row) return p;
  const int32_t i = __ldg(row + p);
  return i >= 0 && i < rows ? i : -1;
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

// ------------------------------------------------ expansions: y and dx
// out_i = base_i + (w v[p]) W over C columns: W is B_g [C, r] with v = s, w =
// w_g, or A_g [r, C] transposed (WT) with v = t, w = 1. Persistent CTAs walk
// equal runs of the list of (columns of eight warps, tile of 16 to 128
// positions). A warp owns two strips of 32 columns (adjacent, or a gate and an up
// strip), keeps its columns of W in registers while the group lasts, and takes a
// tile's positions 16 at a time, the rows of base of the next kAhead sixteens
// under way, past the end of the tile too (cp.async into the lane's own slots of
// shared memory: no barrier). v's fragments (three terms, in the order of the MMA's
// A operand) are staged in shared memory a tile ahead. Column c of n8-tile i of a
// strip is the strip's column 8 (c / 2) + 2 i + c % 2, so that a lane's results
// are eight consecutive columns: one 16-byte access to base, y and h. 8192 rows
// of 28672 columns, rank 16: about 165 us (5.7 TB/s); dx of 4096 columns 21 us;
// 65536 rows of 2 x 768 columns, rank 32, with the activation: about 94 us (3.2
// TB/s), where the 16 warps an SM load, multiply, activate, pack and store in turn.
// The third term costs 3 and 9 us of these; without it y is off by up to 2^-17 of
// what base takes away.
struct Expand {
  const uint16_t* w;
  bool scaled;
  int64_t C;
  const uint16_t* base;
  int64_t ld_base;
  uint16_t* y;
  int64_t ld_y;
  uint16_t* h;
  int64_t ld_h;
  const float* v;  // [slices][R_max][r]
  int slices;
  bool beside;     // nothing comes from the launch before this one but its own earlier work
  float* v_out;    // the slices' sum, written by the first columns' CTAs; or null
  int col_blocks;
  AnyTile tile;
  float alpha, limit;
};

constexpr int kAhead = 2;  // sixteens of base under way (one or three: 2 to 4 us more for 8192 rows of 28672)
static_assert(kAhead == 2, "expand_kernel waits for at most two later ones");
constexpr int kTerms = 3;

enum { kGluNone = 0, kGluHalves = 1, kGluInterleaved = 2 };

E4B_DEV uint4 pack8(const float (&a)[8]) {
  return make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]),
                    pack_bf16x2(a[6], a[7]));
}

// Four values of position p, j .. j + 3: the slices' sum.
E4B_DEV float4 sum_slices(const Adapters& d, const Expand& e, int32_t p, int j) {
  const float* at = e.v + int64_t(p) * d.r + j;
  float4 v = *reinterpret_cast<const float4*>(at);
#pragma unroll 4
  for (int k = 1; k < e.slices; ++k) {
    const float4 z = *reinterpret_cast<const float4*>(at + int64_t(k) * d.R_max * d.r);
    v = make_float4(v.x + z.x, v.y + z.y, v.z + z.z, v.w + z.w);
  }
  return v;
}

// KS: MMA k-steps over the rank (r <= 16 KS); ACT: the activation behind GLU.
// W's fragments take 8 KS registers a strip: above rank 32 a warp has one strip
// where the activation does not need two, so that two CTAs fit an SM.
template <int KS, int GLU>
constexpr int kStrips = KS > 2 && GLU == kGluNone ? 1 : 2;
template <int KS, int GLU>
constexpr int kExpandCtas = KS > 2 && kStrips<KS, GLU> == 2 ? 1 : 2;
// Sixteens of a tile, at most: above rank 32 with two CTAs an SM the terms of four fit
// (8192 rows, rank 64, 4096 columns: y 78 us, dx 82; one CTA with eight 106 and 92).
template <int KS, int GLU>
constexpr int kSixteens = KS > 2 && kExpandCtas<KS, GLU> == 2 ? 4 : kTile / 16;

template <int KS, int GLU, int ACT, bool WT>
__global__ void __launch_bounds__(kThreads, kExpandCtas<KS, GLU>)
expand_kernel(const __grid_constant__ Adapters d, const __grid_constant__ Expand e) {
  constexpr int ST = kStrips<KS, GLU>;
  struct Item {
    int32_t g, cb, row0, n;
  };
  extern __shared__ uint4 smem[];
  constexpr int SIX = kSixteens<KS, GLU>, UNITS = SIX * KS * 32 / kThreads;  // places of the fragments a thread
  using Frags = uint4[SIX][KS][kTerms][32];
  Frags* frags = reinterpret_cast<Frags*>(smem);                 // [2]
  uint4* ring = smem + 2 * sizeof(Frags) / sizeof(uint4);        // [kAhead + 1][2][ST][kThreads], with base
  __shared__ int32_t at[2][kTile];
  __shared__ Item items[3];
  __shared__ int64_t s_sum[kWarps], s_start[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int q = lane & 3, rr = lane >> 2;
  const int C = int(e.C), half = C / 2;
  const int limit[2] = {GLU == kGluHalves ? half : C, C};
  // first columns of the warp's strips
  auto strip = [&](int cb, int st) {
    const int c = (cb * kWarps + warp) * (GLU == kGluHalves ? 32 : 32 * ST);
    return GLU == kGluHalves ? st * half + c : c + 32 * st;
  };
  // a row's place: rows count from 0
  auto place = [](int32_t row, int64_t ld) { return uint64_t(uint32_t(row)) * uint64_t(ld); };

  const Run run = find_run<kThreads>(d.offsets, d.G, d.R_max, e.col_blocks, e.tile, s_sum, s_start);
  if (run.count == 0) {
    grid_dependency_wait();  // the grid must not complete before the launch it depends on
    return;
  }
  Walk<AnyTile> wk(d.offsets, d.G, d.R_max, run, e.tile, s_start);  // thread 0's: the item after the next
  auto note = [&](int64_t k) {
    items[k % 3] = Item{wk.g, wk.cb, int32_t(wk.row0()), wk.n()};
    if (k + 1 < run.count) wk.next();
  };
  if (tid == 0) {
    note(0);
    if (run.count > 1) note(1);
  }
  __syncthreads();

  uint32_t bf[ST][4][KS][2];
  auto load_w = [&](const Item& t) {
    const uint16_t* wg = e.w + int64_t(t.g) * e.C * d.r;
#pragma unroll
    for (int st = 0; st < ST; ++st) {
      if constexpr (WT) {
        const int n = strip(t.cb, st) + 8 * (rr >> 1);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const int j = 16 * ks + 4 * q;
          uint4 v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            v[k] = n < limit[st] && j + k < d.r ? ldg16(wg + int64_t(j + k) * e.C + n) : make_uint4(0, 0, 0, 0);
          const uint32_t sel = rr & 1 ? 0x7632 : 0x5410;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            bf[st][i][ks][0] = prmt(word(v[0], i), word(v[1], i), sel);
            bf[st][i][ks][1] = prmt(word(v[2], i), word(v[3], i), sel);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = strip(t.cb, st) + 8 * (rr >> 1) + 2 * i + (rr & 1);
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            const int j = 16 * ks + 4 * q;
            uint2 v = make_uint2(0, 0);
            if (n < limit[st] && j < d.r) v = __ldg(reinterpret_cast<const uint2*>(wg + int64_t(n) * d.r + j));
            bf[st][i][ks][0] = v.x;
            bf[st][i][ks][1] = v.y;
          }
        }
      }
    }
  };
  // v's share of this thread: its places of the tile's fragments, four values of
  // two rows each; and the row of position tid
  float4 vr[UNITS][2];
  float vw = 1.f;
  int32_t vrow = -1;
  auto load_v = [&](const Item& t) {
    vw = e.scaled && d.scale ? __ldg(d.scale + t.g) : 1.f;
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const int i = u * kThreads + tid, ks = (i >> 5) % KS, six = (i >> 5) / KS;
      const int m = 16 * six + (lane >> 2), j = 16 * ks + 4 * q;
#pragma unroll
      for (int k = 0; k < 2; ++k) {  // rows m and m + 8
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (m + 8 * k < t.n && j < d.r) {
          v = sum_slices(d, e, t.row0 + m + 8 * k, j);
          if (e.v_out && t.cb == 0) *reinterpret_cast<float4*>(e.v_out + int64_t(t.row0 + m + 8 * k) * d.r + j) = v;
        }
        vr[u][k] = v;
      }
    }
    if (tid < kTile) vrow = tid < t.n ? row_of(d.row, d.rows, t.row0 + tid) : -1;
  };
  auto store_v = [&](int buf) {
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const int i = u * kThreads + tid, ks = (i >> 5) % KS, six = (i >> 5) / KS;
      uint32_t w[4][kTerms];  // registers k and k + 2: row m + 8 k
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        split_pair(vw * vr[u][k].x, vw * vr[u][k].y, w[k]);
        split_pair(vw * vr[u][k].z, vw * vr[u][k].w, w[k + 2]);
      }
#pragma unroll
      for (int part = 0; part < kTerms; ++part)
        frags[buf][six][ks][part][lane] = make_uint4(w[0][part], w[1][part], w[2][part], w[3][part]);
    }
    if (tid < kTile) at[buf][tid] = vrow;
  };

  // W does not come from the launch before this one, which has itself waited
  // for all earlier work; nor does anything where it is `beside`, and the wait
  // comes at the end, for the launch after this one
  Item t = items[0];
  load_w(t);
  if (!e.beside) grid_dependency_wait();
  grid_launch_dependents();
  load_v(t);
  store_v(0);
  __syncthreads();

  int asked = 0, taken = 0;  // sixteens of base: asked for, and used
  auto slot = [&](int k, int i, int st) { return ring + ((k % (kAhead + 1) * 2 + i) * ST + st) * kThreads + tid; };
  // the lane's columns of an item
  struct Columns {
    int c[ST];
    bool in[ST];
  };
  auto columns = [&](int cb) {
    Columns k;
#pragma unroll
    for (int st = 0; st < ST; ++st) {
      k.c[st] = strip(cb, st) + 8 * q;
      k.in[st] = k.c[st] < limit[st];
    }
    return k;
  };
  auto fetch = [&](int buf, int six, const Columns& k) {
    if (e.base) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int32_t row = at[buf][16 * six + rr + 8 * i];
        const uint16_t* from = e.base + place(row, e.ld_base);
#pragma unroll
        for (int st = 0; st < ST; ++st)
          if (row >= 0 && k.in[st]) sm100::cp_async_16(slot(asked, i, st), from + k.c[st], 16);
      }
    }
    sm100::cp_async_commit();
    ++asked;
  };
  auto arrived = [&]() {  // the oldest sixteen
    const int later = asked - taken - 1;
    if (later >= 2) sm100::cp_async_wait<2>();
    else if (later == 1) sm100::cp_async_wait<1>();
    else sm100::cp_async_wait<0>();
  };

  int had = 0;  // sixteens of this item already asked for
  for (int64_t k = 0; k < run.count; ++k) {
    const int buf = int(k & 1);
    const bool more = k + 1 < run.count;
    Item next = t;
    if (more) {
      next = items[(k + 1) % 3];
      load_v(next);
    }
    const int sixteens = (t.n + 15) / 16, next_sixteens = (next.n + 15) / 16;
    const int stage_at = sixteens > kAhead ? sixteens - kAhead : 0;  // from here on the next item's rows are asked for
    int next_had = 0;
    const Columns cols = columns(t.cb);
    while (had < sixteens && had < kAhead) fetch(buf, had++, cols);
    for (int six = 0; six < sixteens; ++six) {
      if (more && six == stage_at) {
        __syncthreads();  // all warps are past the item that used these fragments
        store_v(buf ^ 1);
        if (tid == 0 && k + 2 < run.count) note(k + 2);
        __syncthreads();
      }
      if (had < sixteens)
        fetch(buf, had++, cols);
      else if (more && next_had < next_sixteens && next_had < kAhead)
        fetch(buf ^ 1, next_had++, next.cb == t.cb ? cols : columns(next.cb));
      arrived();
      int32_t row[2];
      float acc[ST][4][4];  // starts as base
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        row[i] = at[buf][16 * six + rr + 8 * i];
#pragma unroll
        for (int st = 0; st < ST; ++st) {
          const uint4 b = e.base && cols.in[st] && row[i] >= 0 ? *slot(taken, i, st) : make_uint4(0, 0, 0, 0);
          const uint32_t words[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const float2 f = unpack2(words[p]);
            acc[st][p][2 * i] = f.x;
            acc[st][p][2 * i + 1] = f.y;
          }
        }
      }
      ++taken;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int part = 0; part < kTerms; ++part) {
          const uint4 f = frags[buf][six][ks][part][lane];
#pragma unroll
          for (int st = 0; st < ST; ++st)
#pragma unroll
            for (int i = 0; i < 4; ++i) mma_bf16(acc[st][i], f.x, f.y, f.z, f.w, bf[st][i][ks][0], bf[st][i][ks][1]);
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (row[i] < 0) continue;
        float v[ST][8];
#pragma unroll
        for (int st = 0; st < ST; ++st) {
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            v[st][2 * p] = acc[st][p][2 * i];
            v[st][2 * p + 1] = acc[st][p][2 * i + 1];
          }
          if (e.y && cols.in[st]) *reinterpret_cast<uint4*>(e.y + place(row[i], e.ld_y) + cols.c[st]) = pack8(v[st]);
        }
        if constexpr (GLU == kGluHalves) {
          float h[8];
#pragma unroll
          for (int p = 0; p < 8; ++p) h[p] = gated<ACT == E4B_ACT_CLAMPED_GLU>(v[0][p], v[1][p], e.alpha, e.limit);
          if (cols.in[0]) *reinterpret_cast<uint4*>(e.h + place(row[i], e.ld_h) + cols.c[0]) = pack8(h);
        } else if constexpr (GLU == kGluInterleaved) {
#pragma unroll
          for (int st = 0; st < ST; ++st) {
            float h[4];
#pragma unroll
            for (int p = 0; p < 4; ++p) h[p] = gated<ACT == E4B_ACT_CLAMPED_GLU>(v[st][2 * p], v[st][2 * p + 1], e.alpha, e.limit);
            if (cols.in[st])
              *reinterpret_cast<uint2*>(e.h + place(row[i], e.ld_h) + cols.c[st] / 2) =
                  make_uint2(pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3]));
          }
        }
      }
    }
    if (next.g != t.g || next.cb != t.cb) load_w(next);
    t = next;
    had = next_had;
  }
  if (e.beside) grid_dependency_wait();
}

// The parts' sum: eight threads a float4 take every eighth part, and their
// sums meet in order.
__global__ void __launch_bounds__(kThreads)
sum_parts_kernel(const float* __restrict__ part, int parts, int64_t n4, float* __restrict__ out) {
  __shared__ float4 sums[kThreads / 32][32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, k0 = threadIdx.x >> 5;
  const int64_t i = int64_t(blockIdx.x) * 32 + lane;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float4 v) { s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w); };
  if (i < n4) {
#pragma unroll 4
    for (int k = k0; k < parts; k += kThreads / 32) add(reinterpret_cast<const float4*>(part)[int64_t(k) * n4 + i]);
  }
  sums[k0][lane] = s;
  __syncthreads();
  if (k0 || i >= n4) return;
#pragma unroll
  for (int k = 1; k < kThreads / 32; ++k) add(sums[k][lane]);
  reinterpret_cast<float4*>(out)[i] = s;
}

// --------------------------------------------------------------- launches
int tiles_of_rank(int r) { return r <= 8 ? 1 : r <= 16 ? 2 : r <= 32 ? 4 : 8; }

int64_t pieces_bound(int64_t G, int64_t R_max, int64_t piece) {
  const int64_t full = R_max / piece;
  return full + (G < R_max ? G : R_max);
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

Adapters adapters_of(const e4b_lora_args& a) {
  return Adapters{a.a, a.b, a.scale, a.offsets, a.row, a.rows, a.N, a.K, a.R_max, a.G, a.r};
}

ContractArgs contract_of(const e4b_lora_args& a, const uint16_t* z, int64_t ld_z, int64_t C, uint32_t flags) {
  ContractArgs c{};
  c.G = a.G;
  c.r = a.r;
  c.C = C;
  c.R_max = a.R_max;
  c.offsets = a.offsets;
  c.row = a.row;
  c.rows = a.rows;
  c.z = z;
  c.ld_z = ld_z;
  c.scale = a.scale;
  c.status = a.status;
  c.no_wait = (flags & E4B_FLAG_TEST_TIMEOUT) != 0;
  return c;
}

// s of a forward pass on the 128-row tiles of the tensor-core pass, or by warps
// that split K where there is little to do (a decode batch). Whole calls, y
// included, with one group and with 16, tiles against warps: rank 16, K = N =
// 4096, 512 rows 13.2 and 13.5 against 9.6 and 9.8 us, 2048 rows 19.2 and 16.7
// against 16.2 and 18.1; rank 64, 512 rows 22.1 and 16.7 against 20.8 and 19.5,
// 2048 rows 32.0 and 27.5 against 36.7 and 44.9; K = N = 1024, 2048 rows, rank 16
// 12.2 and 11.8 against 8.7 and 9.1, rank 64 21.3 and 19.7 against 18.9 and 21.5.
bool forward_uses_tiles(int64_t R_max, int64_t K, int r) { return double(R_max) * double(K) * r > 2e8; }

// Parts of s that warps make, at most: one 32-wide chunk a warp, 16.
int64_t most_slices(int64_t K) {
  const int64_t most = (K + 32 * kWarps - 1) / (32 * kWarps);
  return most < 16 ? most : 16;
}

// Parts of s. Few rows: enough CTAs to fill the GPU.
int forward_slices(int G, int r, int64_t K, int64_t R_max, int sms) {
  if (forward_uses_tiles(R_max, K, r)) return contract_blocks(G, r, K, R_max, true, false, sms);
  const int64_t tiles = pieces_bound(G, R_max, kShrinkRows);
  int64_t want = sms / (tiles > 0 ? tiles : 1);
  if (want > most_slices(K)) want = most_slices(K);
  return int(want < 1 ? 1 : want);
}

// At least forward_slices() times the rows, for every number of rows up to R_max.
// By warps, beyond one slice: 32 rows a CTA or fewer (there are R / 32 + min(G, R)
// pieces or none) and no more CTAs than SMs.
int64_t forward_part_rows(int G, int r, int64_t K, int64_t R_max, int sms) {
  int64_t found = R_max;
  const int64_t sliced = most_slices(K) * R_max, cap = int64_t(kShrinkRows) * sms;
  if (found < sliced && found < cap) found = sliced < cap ? sliced : cap;
  if (forward_uses_tiles(R_max, K, r)) {
    const int64_t rows = contract_out_rows(G, r, K, R_max, false, sms);
    if (found < rows) found = rows;
  }
  return found;
}

template <int KS, int GLU, int ACT, bool WT>
cudaError_t launch_expand_of(const Adapters& d, Expand e, cudaStream_t st, int sms) {
  constexpr int strips = kStrips<KS, GLU>;
  const int64_t cols = GLU == kGluHalves ? e.C / 2 : e.C, per = kWarps * (GLU == kGluHalves ? 32 : 32 * strips);
  e.col_blocks = int((cols + per - 1) / per);
  // the largest tile (a sixteen's MMAs need its factors staged) of which there are
  // enough to go round: 128 rows of one group, r 64, 4096 columns took 19 us less so
  const int64_t ctas = int64_t(sms) * kExpandCtas<KS, GLU>, groups = d.G < d.R_max ? d.G : d.R_max;
  e.tile.bits = kSixteens<KS, GLU> == 4 ? 6 : 7;
  while (e.tile.bits > 4 && e.col_blocks * ((d.R_max >> e.tile.bits) + (groups + 1) / 2) < ctas) --e.tile.bits;
  int64_t grid = e.col_blocks * pieces_bound(d.G, d.R_max, int64_t(1) << e.tile.bits);
  if (grid > ctas) grid = ctas;
  auto kernel = expand_kernel<KS, GLU, ACT, WT>;
  constexpr int staged = 2 * kSixteens<KS, GLU> * KS * kTerms * 32 * 16, ring = (kAhead + 1) * 2 * strips * kThreads * 16;
  const int smem = staged + (e.base ? ring : 0);
  static SmemAllowed allowed;
  const cudaError_t err = allow_smem(kernel, staged + ring, allowed);
  if (err != cudaSuccess) return err;
  return launch_dependent(kernel, dim3(unsigned(grid)), dim3(kThreads), smem, st, d, e);
}

template <int GLU, int ACT, bool WT>
cudaError_t launch_expand_as(const Adapters& d, const Expand& e, cudaStream_t st, int sms) {
  if (d.r <= 16) return launch_expand_of<1, GLU, ACT, WT>(d, e, st, sms);
  if (d.r <= 32) return launch_expand_of<2, GLU, ACT, WT>(d, e, st, sms);
  return launch_expand_of<4, GLU, ACT, WT>(d, e, st, sms);
}

cudaError_t launch_expand(const Adapters& d, const Expand& e, int layout, int act, cudaStream_t st, int sms) {
  if (!e.h) return launch_expand_as<kGluNone, 0, false>(d, e, st, sms);
  const bool clamped = act == E4B_ACT_CLAMPED_GLU;
  if (layout == E4B_GATE_UP_INTERLEAVED)
    return clamped ? launch_expand_as<kGluInterleaved, E4B_ACT_CLAMPED_GLU, false>(d, e, st, sms)
                   : launch_expand_as<kGluInterleaved, E4B_ACT_SWIGLU, false>(d, e, st, sms);
  return clamped ? launch_expand_as<kGluHalves, E4B_ACT_CLAMPED_GLU, false>(d, e, st, sms)
                 : launch_expand_as<kGluHalves, E4B_ACT_SWIGLU, false>(d, e, st, sms);
}

template <int JT>
cudaError_t launch_shrink(const Adapters& d, const e4b_lora_args& a, int slices, float* s, cudaStream_t st) {
  const int tiles = int(pieces_bound(a.G, a.R_max, kShrinkRows));
  return launch_dependent(shrink_kernel<JT>, dim3(tiles, slices), dim3(kThreads), 0, st, d, a.x, a.ld_x, slices, s);
}

// Sections that are large enough for every number of rows up to R_max.
struct BackPlan {
  size_t t_part, t, db_part, da_part, total;
};

BackPlan plan_backward(int G, int r, int64_t N, int64_t K, int64_t R_max, int sms) {
  BackPlan p;
  // t alone is cut otherwise than t and db together: room for either
  const int64_t a = contract_out_rows(G, r, N, R_max, true, sms), b = contract_out_rows(G, r, N, R_max, false, sms);
  size_t o = 0;
  p.t_part = o;  o = align256(o + size_t(a > b ? a : b) * r * 4);
  p.t = o;       o = align256(o + size_t(R_max) * r * 4);
  p.db_part = o; o = align256(o + contract_part_bytes(r, N, false, sms));  // with t there are no more
  p.da_part = o; o = align256(o + contract_part_bytes(r, K, false, sms));
  p.total = o;
  return p;
}

}  // namespace

size_t lora_workspace_bytes(int64_t G, int r, int64_t N, int64_t K, int64_t R_max, bool back, int sms) {
  if (back) return plan_backward(int(G), r, N, K, R_max, sms).total + 256;
  return align256(size_t(forward_part_rows(int(G), r, K, R_max, sms)) * r * 4) + 256;
}

cudaError_t launch_lora(const e4b_lora_args& a, void* ws, uint32_t flags, cudaStream_t st, int sms, int* launches) {
  const Adapters d = adapters_of(a);
  const int slices = forward_slices(a.G, a.r, a.K, a.R_max, sms);
  float* s = a.s && slices == 1 ? a.s : static_cast<float*>(ws);
  cudaError_t err;
  if (forward_uses_tiles(a.R_max, a.K, a.r)) {
    ContractArgs c = contract_of(a, a.x, a.ld_x, a.K, flags);
    c.w = a.a;
    c.out = s;
    err = launch_contract(c, st, sms);
  } else {
    switch (tiles_of_rank(a.r)) {
      case 1: err = launch_shrink<1>(d, a, slices, s, st); break;
      case 2: err = launch_shrink<2>(d, a, slices, s, st); break;
      case 4: err = launch_shrink<4>(d, a, slices, s, st); break;
      default: err = launch_shrink<8>(d, a, slices, s, st);
    }
  }
  if (err != cudaSuccess) return err;
  *launches = 1;
  if (!a.y && !a.h && slices == 1) return cudaSuccess;  // s alone was asked for
  const bool rows = a.y || a.h;  // else only s' parts are to be added
  const Expand e{a.b, true, a.N, rows ? a.base : nullptr, a.ld_base, a.y, a.ld_y, a.h, a.ld_h, s, slices, false,
                 slices > 1 ? a.s : nullptr, 0, AnyTile{}, a.glu_alpha, a.glu_limit};
  *launches = 2;
  return launch_expand(d, e, a.gate_up_layout, a.activation, st, sms);
}

cudaError_t launch_lora_backward(const e4b_lora_args& a, void* ws, uint32_t flags, cudaStream_t st, int sms,
                                 int* launches) {
  const Adapters d = adapters_of(a);
  const BackPlan p = plan_backward(a.G, a.r, a.N, a.K, a.R_max, sms);
  uint8_t* base = static_cast<uint8_t*>(ws);
  float* t = reinterpret_cast<float*>(base + p.t);
  const bool wants_t = a.da || a.dx, accumulate = (flags & E4B_FLAG_ACCUMULATE) != 0;
  *launches = 0;
  cudaError_t err;

  ContractArgs y = contract_of(a, a.dy, a.ld_dy, a.N, flags);
  if (wants_t) {
    y.w = a.b;
    y.w_t = true;
    y.scale_out = true;
    y.out = reinterpret_cast<float*>(base + p.t_part);
  }
  if (a.db) {
    y.v = a.s;
    y.scale_v = true;
    y.grad = a.db;
    y.grad_t = true;
    y.accumulate = accumulate;
    y.grad_part = reinterpret_cast<float*>(base + p.db_part);
  }
  const int parts = contract_blocks(a.G, a.r, a.N, a.R_max, wants_t, a.db != nullptr, sms);
  if (parts == 1) t = y.out;
  ContractArgs x = contract_of(a, a.x, a.ld_x, a.K, flags);
  if (a.da) {
    x.follows = true;
    x.v = t;
    x.grad = a.da;
    x.accumulate = accumulate;
    x.grad_part = reinterpret_cast<float*>(base + p.da_part);
  }
  if (a.R_max > 0) {
    if ((err = launch_contract(y, st, sms)) != cudaSuccess) return err;
    ++*launches;
    if (wants_t && parts > 1) {
      const int64_t n4 = a.R_max * a.r / 4;
      err = launch_dependent(sum_parts_kernel, dim3(unsigned((n4 + 31) / 32)), dim3(kThreads), 0, st,
                             const_cast<const float*>(y.out), parts, n4, t);
      if (err != cudaSuccess) return err;
      ++*launches;
    }
    if (a.da) {
      if ((err = launch_contract(x, st, sms)) != cudaSuccess) return err;
      ++*launches;
    }
    if (a.dx) {
      const Expand e{a.a, false, a.K, a.dx_base, a.ld_dx_base, a.dx, a.ld_dx, nullptr, 0, t, 1,
                     a.da != nullptr, nullptr, 0, AnyTile{}, 0.f, 0.f};  // da's pass has waited for t and does not write it
      if ((err = launch_expand_as<kGluNone, 0, true>(d, e, st, sms)) != cudaSuccess) return err;
      ++*launches;
    }
  }
  if (a.da || a.db) {
    err = launch_contract_finish(a.db ? &y : &x, a.db && a.da ? &x : nullptr, st, sms);
    if (err != cudaSuccess) return err;
    ++*launches;
  }
  return cudaSuccess;
}

}  // namespace e4b
