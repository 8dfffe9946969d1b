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

// The hardware exp2 and reciprocal (relative error ~2^-20, far below bf16's
// half step). Below -87 the reciprocal flushes to zero, where the exact value
// is under 2^-125.
E4B_DEV float fast_sigmoid(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

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
  int act;
  float alpha, limit;
};

// Eight pairs of a row. gu is read before dgu is written, element for element
// by the same thread, so dgu may be gu.
template <bool INTERLEAVED, bool BACKWARD>
E4B_DEV void glu_vec(const GluRows& a, int64_t row, int64_t v) {
  float g[8], u[8];
  const uint16_t* src = a.gu + row * a.ld_gu;
  if constexpr (INTERLEAVED) {
    float w[16];
    const uint4 lo = reinterpret_cast<const uint4*>(src)[2 * v], hi = reinterpret_cast<const uint4*>(src)[2 * v + 1];
    unpack8(lo, reinterpret_cast<float(&)[8]>(w[0]));
    unpack8(hi, reinterpret_cast<float(&)[8]>(w[8]));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      g[i] = w[2 * i];
      u[i] = w[2 * i + 1];
    }
  } else {
    unpack8(reinterpret_cast<const uint4*>(src)[v], g);
    unpack8(reinterpret_cast<const uint4*>(src + a.I)[v], u);
  }
  float h[8];
  if constexpr (!BACKWARD) {
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = glu_act(a.act, g[i], u[i], a.alpha, a.limit);
    reinterpret_cast<uint4*>(a.h + row * a.ld_h)[v] = pack8(h);
  } else {
    float d[8], dg[8], du[8];
    unpack8(reinterpret_cast<const uint4*>(a.dh + row * a.ld_dh)[v], d);
    const bool clamped = a.act == E4B_ACT_CLAMPED_GLU;
    const float b = clamped ? a.alpha : 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // comparisons that let NaN inputs through as NaN
      const bool gout = clamped && g[i] > a.limit;
      const bool uout = clamped && (u[i] > a.limit || u[i] < -a.limit);
      const float gc = gout ? a.limit : g[i];
      const float uc = clamped ? (uout ? copysignf(a.limit, u[i]) : u[i]) + 1.f : u[i];
      const float sg = fast_sigmoid(b * gc);
      const float f = gc * sg;
      h[i] = f * uc;
      dg[i] = gout ? 0.f : d[i] * uc * (sg * fmaf(b * gc, 1.f - sg, 1.f));
      du[i] = uout ? 0.f : d[i] * f;
    }
    uint16_t* dst = a.dgu + row * a.ld_dgu;
    if constexpr (INTERLEAVED) {
      float w[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w[2 * i] = dg[i];
        w[2 * i + 1] = du[i];
      }
      reinterpret_cast<uint4*>(dst)[2 * v] = pack8(reinterpret_cast<float(&)[8]>(w[0]));
      reinterpret_cast<uint4*>(dst)[2 * v + 1] = pack8(reinterpret_cast<float(&)[8]>(w[8]));
    } else {
      reinterpret_cast<uint4*>(dst)[v] = pack8(dg);
      reinterpret_cast<uint4*>(dst + a.I)[v] = pack8(du);
    }
    if (a.h) reinterpret_cast<uint4*>(a.h + row * a.ld_h)[v] = pack8(h);
  }
}

// Threads walk the rows' vectors in one flat order; (row, vector) advance by
// the grid's stride without a division (stride = step_row * V + step_vec).
template <bool INTERLEAVED, bool BACKWARD>
__global__ void __launch_bounds__(kGluThreads)
glu_kernel(GluRows a, int64_t V, int64_t step_row, int64_t step_vec, const int64_t* __restrict__ offsets,
           int32_t E, int64_t R_max) {
  const int64_t R = offsets ? min(offsets[E], R_max) : R_max;
  const int64_t i = int64_t(blockIdx.x) * kGluThreads + threadIdx.x;
  int64_t row = i / V, v = i - row * V;
  while (row < R) {
    glu_vec<INTERLEAVED, BACKWARD>(a, row, v);
    row += step_row;
    v += step_vec;
    if (v >= V) {
      v -= V;
      ++row;
    }
  }
}

}  // namespace

cudaError_t launch_glu(const e4b_glu_args& a, bool backward, cudaStream_t st, int sms) {
  GluRows k{a.gu, a.ld_gu, a.dh, a.ld_dh, a.h, a.ld_h, a.dgu, a.ld_dgu, a.I, a.activation, a.glu_alpha, a.glu_limit};
  const int64_t V = a.I / 8;
  int64_t grid = (a.R_max * V + kGluThreads - 1) / kGluThreads;
  const int64_t cap = int64_t(sms) * 8;
  if (grid > cap) grid = cap;
  const int64_t stride = grid * kGluThreads;
  const int64_t sr = stride / V, sv = stride % V;
  const bool il = a.gate_up_layout == E4B_GATE_UP_INTERLEAVED;
  auto kernel = il ? (backward ? glu_kernel<true, true> : glu_kernel<true, false>)
                   : (backward ? glu_kernel<false, true> : glu_kernel<false, false>);
  kernel<<<int(grid), kGluThreads, 0, st>>>(k, V, sr, sv, a.offsets, a.E, a.R_max);
  return cudaGetLastError();
}

}  // namespace e4b
