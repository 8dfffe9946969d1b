// The gated activation on stored gate_up rows, and its gradient. For gate g
// and up u of a pair, sg(v) = 1 / (1 + exp(-v)):
//   SwiGLU       h = g sg(g) u
//                dg = dh u sg(g) (1 + g (1 - sg(g))),  du = dh g sg(g)
//   clamped GLU  g' = min(g, L), u' = clamp(u, -L, L), h = (u' + 1) g' sg(a g')
//                dg = dh (u' + 1) sg(a g') (1 + a g' (1 - sg(a g'))) where g <= L, else 0
//                du = dh g' sg(a g') where |u| <= L, else 0
// Everything in fp32, rounded to bf16 once. The grouped GEMM applies the
// forward form to its accumulators; these kernels serve rows that have to be
// kept as they were before the activation: a training step's, or those an
// adapter adds to. Bound by HBM: 6 bytes a pair forward, 10 to 12 backward.
#include "adapters.h"
#include "common.cuh"

namespace e4b {
namespace {

constexpr int kGluThreads = 256;

E4B_DEV void unpack8(uint4 v, float (&f)[8]) {
  const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(q[i] << 16);
    f[2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
  }
}

E4B_DEV uint4 pack8(const float (&a)[8]) {
  return make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]),
                    pack_bf16x2(a[6], a[7]));
}

struct GluRows {
  const uint16_t* gu;
  int64_t ld_gu;
  const uint16_t* dh;
  int64_t ld_dh;
  uint16_t* h;
  int64_t ld_h;
  uint16_t* dgu;
  int64_t ld_dgu;
  int64_t I;
  float alpha, limit;
};

template <typename T>
E4B_DEV void put(void* p, T v) {
  *reinterpret_cast<T*>(p) = v;
}

// A lane's pairs of a row: eight (16 bytes of gates, 16 of ups) with the gate
// and up halves apart, four (16 bytes of pairs) where they alternate, so that
// every access of a warp covers whole lines.
template <bool INTERLEAVED>
constexpr int kPairs = INTERLEAVED ? 4 : 8;

template <bool INTERLEAVED, bool BACKWARD, bool CLAMPED>
struct GluVec {
  uint4 a, b;   // gates and ups, or (a alone) pairs
  uint4 d;      // dh (interleaved: x, y)
  __device__ __forceinline__ void load(const GluRows& r, int64_t row, int64_t v) {
    const uint16_t* src = r.gu + row * r.ld_gu;
    a = reinterpret_cast<const uint4*>(src)[v];
    if constexpr (!INTERLEAVED) b = reinterpret_cast<const uint4*>(src + r.I)[v];
    if constexpr (BACKWARD) {
      const uint16_t* dh = r.dh + row * r.ld_dh;
      if constexpr (INTERLEAVED) {
        const uint2 w = reinterpret_cast<const uint2*>(dh)[v];
        d = make_uint4(w.x, w.y, 0, 0);
      } else {
        d = reinterpret_cast<const uint4*>(dh)[v];
      }
    }
  }
  __device__ __forceinline__ void finish(const GluRows& r, int64_t row, int64_t v) const {
    constexpr int P = kPairs<INTERLEAVED>;
    float g[P], u[P], h[P];
    if constexpr (INTERLEAVED) {
      const uint32_t q[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < P; ++i) {
        g[i] = __uint_as_float(q[i] << 16);
        u[i] = __uint_as_float(q[i] & 0xFFFF0000u);
      }
    } else {
      unpack8(a, g);
      unpack8(b, u);
    }
    if constexpr (!BACKWARD) {
#pragma unroll
      for (int i = 0; i < P; ++i) h[i] = gated<CLAMPED>(g[i], u[i], r.alpha, r.limit);
    } else {
      float dw[8], dg[P], du[P];
      unpack8(d, dw);
      const float slope = CLAMPED ? r.alpha : 1.f;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        // comparisons that let NaN inputs through as NaN
        const bool gout = CLAMPED && g[i] > r.limit;
        const bool uout = CLAMPED && (u[i] > r.limit || u[i] < -r.limit);
        const float gc = gout ? r.limit : g[i];
        const float uc = CLAMPED ? (uout ? copysignf(r.limit, u[i]) : u[i]) + 1.f : u[i];
        const float sg = gate_sigmoid(gc, slope);
        const float f = gc * sg;
        h[i] = f * uc;  // as gated() has it
        // sg (1 + a g' (1 - sg)) as sg + a (g' sg) (1 - sg): no factor overflows where the gate is closed
        dg[i] = gout ? 0.f : dw[i] * (uc * fmaf(slope * f, 1.f - sg, sg));
        du[i] = uout ? 0.f : dw[i] * f;
      }
      uint16_t* dst = r.dgu + row * r.ld_dgu;
      if constexpr (INTERLEAVED) {
        put(reinterpret_cast<uint4*>(dst) + v, make_uint4(pack_bf16x2(dg[0], du[0]), pack_bf16x2(dg[1], du[1]),
                                                          pack_bf16x2(dg[2], du[2]), pack_bf16x2(dg[3], du[3])));
      } else {
        put(reinterpret_cast<uint4*>(dst) + v, pack8(dg));
        put(reinterpret_cast<uint4*>(dst + r.I) + v, pack8(du));
      }
    }
    if (!BACKWARD || r.h) {
      uint16_t* dst = r.h + row * r.ld_h;
      if constexpr (INTERLEAVED)
        put(reinterpret_cast<uint2*>(dst) + v, make_uint2(pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3])));
      else
        put(reinterpret_cast<uint4*>(dst) + v, pack8(h));
    }
  }
};

// Threads walk the rows' vectors in one flat order, kUnroll of them in flight;
// (row, vector) advance by the grid's stride without a division (stride =
// step_row * V + step_vec). A vector of gu is read before the same vector of
// dgu is written, by the same thread, so dgu may be gu. Two vectors a thread:
// 8192 rows of 14336 pairs take 107 us (the copy rate; one vector 125 us, four
// 121 us), and the gradient with h of 32764 clamped, alternating rows of 2880
// pairs 189 us (6.0 TB/s, 91% of the copy rate).
constexpr int kUnroll = 2;

template <bool INTERLEAVED, bool BACKWARD, bool CLAMPED>
__global__ void __launch_bounds__(kGluThreads, 2)
glu_kernel(GluRows a, int64_t V, int64_t step_row, int64_t step_vec, const int64_t* __restrict__ offsets,
           int32_t E, int64_t R_max) {
  const int64_t R = offsets ? min(offsets[E], R_max) : R_max;
  const int64_t i = int64_t(blockIdx.x) * kGluThreads + threadIdx.x;
  int64_t row = i / V, v = i - row * V;
  while (row < R) {
    GluVec<INTERLEAVED, BACKWARD, CLAMPED> w[kUnroll];
    int64_t rows[kUnroll], vs[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      rows[k] = row;
      vs[k] = v;
      if (row < R) w[k].load(a, row, v);
      row += step_row;
      v += step_vec;
      if (v >= V) {
        v -= V;
        ++row;
      }
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k)
      if (rows[k] < R) w[k].finish(a, rows[k], vs[k]);
  }
}

}  // namespace

cudaError_t launch_glu(const e4b_glu_args& a, bool backward, cudaStream_t st, int sms) {
  GluRows k{a.gu, a.ld_gu, a.dh, a.ld_dh, a.h, a.ld_h, a.dgu, a.ld_dgu, a.I, a.glu_alpha, a.glu_limit};
  const bool il = a.gate_up_layout == E4B_GATE_UP_INTERLEAVED;
  const int64_t V = a.I / (il ? kPairs<true> : kPairs<false>);
  int64_t grid = (a.R_max * V + kGluThreads - 1) / kGluThreads;
  const int64_t cap = int64_t(sms) * 32;
  if (grid > cap) grid = cap;
  const int64_t stride = grid * kGluThreads;
  const int64_t sr = stride / V, sv = stride % V;
  const bool clamped = a.activation == E4B_ACT_CLAMPED_GLU;
  using Kernel = void (*)(GluRows, int64_t, int64_t, int64_t, const int64_t*, int32_t, int64_t);
  static constexpr Kernel kernels[2][2][2] = {
      {{glu_kernel<false, false, false>, glu_kernel<false, false, true>},
       {glu_kernel<false, true, false>, glu_kernel<false, true, true>}},
      {{glu_kernel<true, false, false>, glu_kernel<true, false, true>},
       {glu_kernel<true, true, false>, glu_kernel<true, true, true>}}};
  const Kernel kernel = kernels[il][backward][clamped];
  kernel<<<int(grid), kGluThreads, 0, st>>>(k, V, sr, sv, a.offsets, a.E, a.R_max);
  return cudaGetLastError();
}

}  // namespace e4b
