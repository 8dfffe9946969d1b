// Token rows sorted by expert and back, and the gradients of both. With the
// routing pass' arrays (slot s = t * k + j, position p: perm[p] = s, inv[s] = p,
// -1 for a dropped slot), for bf16 rows of H values:
//   permute             xs[p] = x[perm[p] / k]
//   permute_backward    dx[t] = sum_j dxs[inv[t, j]]
//   unpermute           y[t]  = sum_j g[t, j] ys[inv[t, j]]
//   unpermute_backward  dys[p] = g[s] dy[t],  dg[s] = <dy[t], ys[p]>
// The sums over a token's slots run in slot order in fp32 and are rounded to
// bf16 once, so results do not change from run to run. All four are bound by
// HBM: a few operations per 16 bytes.
#include "adapters.h"
#include "common.cuh"

namespace e4b {
namespace {

constexpr int kRowThreads = 256;

E4B_DEV float2 unpack_bf16x2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

E4B_DEV void fma8(float (&acc)[8], uint4 v, float w) {
  const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack_bf16x2(q[i]);
    acc[2 * i] = fmaf(w, f.x, acc[2 * i]);
    acc[2 * i + 1] = fmaf(w, f.y, acc[2 * i + 1]);
  }
}

E4B_DEV uint4 pack8(const float (&a)[8]) {
  return make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]),
                    pack_bf16x2(a[6], a[7]));
}

E4B_DEV const uint4* vec_row(RowsIn r, int64_t i) { return reinterpret_cast<const uint4*>(r.p + i * r.ld); }
E4B_DEV uint4* vec_row(RowsOut r, int64_t i) { return reinterpret_cast<uint4*>(r.p + i * r.ld); }

// Results are not read again by these kernels: stored evict-first, so that the
// rows that are (a token's row by all its slots) stay in L2. Sorting 8192 rows
// of 2048 values to 65536 took 59 us so, 66 us with plain stores.
E4B_DEV void put(uint4* p, uint4 v) { __stcs(p, v); }

// How a warp's lanes cover a row of `vecs` 16-byte vectors: 1 << lane_bits
// lanes a row (fewer than 32 for short rows, so that no lanes idle), `chunks`
// pieces of (1 << lane_bits) * (vectors a lane holds). A unit is (row group,
// chunk).
struct RowSplit {
  int lane_bits;
  int chunks;
  int64_t vecs;
};

RowSplit split_rows(int64_t H, int kVec) {
  RowSplit s;
  s.vecs = H / 8;
  s.lane_bits = 0;
  while (s.lane_bits < 5 && (int64_t(1) << s.lane_bits) < s.vecs) ++s.lane_bits;
  const int64_t per = int64_t(kVec) << s.lane_bits;
  s.chunks = int((s.vecs + per - 1) / per);
  return s;
}

int grid_of(int64_t rows, RowSplit s, int sms, int per_sm) {
  const int64_t per_warp = 32 >> s.lane_bits;
  const int64_t units = (rows + per_warp - 1) / per_warp * s.chunks;
  const int64_t want = (units + kRowThreads / 32 - 1) / (kRowThreads / 32);
  const int64_t cap = int64_t(sms) * per_sm;
  return int(want < 1 ? 1 : (want < cap ? want : cap));
}

template <int kVec>
__global__ void __launch_bounds__(kRowThreads)
permute_kernel(RowsIn x, int64_t slots, RowSplit sp, const int32_t* __restrict__ perm, int32_t top_k,
               const int64_t* __restrict__ offsets, int32_t E, int64_t R_max, RowsOut xs) {
  const int lane = threadIdx.x & 31;
  const int sub = lane >> sp.lane_bits;           // row within the warp's rows
  const int col = lane & ((1 << sp.lane_bits) - 1);
  const int per_warp = 32 >> sp.lane_bits;
  const int64_t R = min(offsets[E], R_max);
  const int64_t units = (R + per_warp - 1) / per_warp * sp.chunks;
  const int64_t stride = int64_t(gridDim.x) * (kRowThreads / 32);
  for (int64_t u = int64_t(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5); u < units; u += stride) {
    const int64_t rg = u / sp.chunks;
    const int64_t p = rg * per_warp + sub;
    if (p >= R) continue;
    const int32_t slot = __ldg(perm + p);
    if (uint32_t(slot) >= uint64_t(slots)) continue;
    const uint4* src = vec_row(x, slot / top_k);
    uint4* dst = vec_row(xs, p);
    const int64_t c0 = ((u - rg * sp.chunks) * kVec << sp.lane_bits) + col;
    uint4 v[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int64_t c = c0 + (int64_t(i) << sp.lane_bits);
      if (c < sp.vecs) v[i] = __ldg(src + c);
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int64_t c = c0 + (int64_t(i) << sp.lane_bits);
      if (c < sp.vecs) put(dst + c, v[i]);
    }
  }
}

// One unit: a token's chunk. The rows of JB slots are in flight together, and
// the next unit's positions are on their way while this unit's rows are. Two
// slots by two vectors leave room for four CTAs on an SM, and the grid is those
// CTAs: 32760 rows of 2880 values to 8190 tokens took 40 us (90% of the copy
// rate); more bytes a lane and fewer warps, or more CTAs than fit, 44 to 76 us.
constexpr int kSumCtas = 4;
template <int JB, int kVec>
__global__ void __launch_bounds__(kRowThreads, kSumCtas)
sum_slots_kernel(RowsIn rows, int64_t R_max, RowSplit sp, const int32_t* __restrict__ inv,
                 const float* __restrict__ gates, int64_t T, int32_t top_k, RowsOut y) {
  const int lane = threadIdx.x & 31;
  const int sub = lane >> sp.lane_bits;
  const int col = lane & ((1 << sp.lane_bits) - 1);
  const int per_warp = 32 >> sp.lane_bits;
  const uint32_t units = uint32_t((T + per_warp - 1) / per_warp) * sp.chunks;
  const uint32_t stride = gridDim.x * (kRowThreads / 32);
  uint32_t u = blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  int32_t pos[JB];
  float wt[JB];
  auto fetch = [&](int64_t t, int j0) {
#pragma unroll
    for (int j = 0; j < JB; ++j) {
      const bool in = t < T && j0 + j < top_k;
      pos[j] = in ? __ldg(inv + t * top_k + j0 + j) : -1;
      wt[j] = in && gates ? __ldg(gates + t * top_k + j0 + j) : 1.f;
    }
  };
  if (u < units) fetch(int64_t(u / sp.chunks) * per_warp + sub, 0);
  for (; u < units; u += stride) {
    const uint32_t rg = u / sp.chunks;
    const int64_t t = int64_t(rg) * per_warp + sub;
    const int64_t c0 = (int64_t(u - rg * sp.chunks) * kVec << sp.lane_bits) + col;
    float acc[kVec][8] = {};
    for (int j0 = 0; j0 < top_k; j0 += JB) {
      uint4 v[JB][kVec];
      float w[JB];
#pragma unroll
      for (int j = 0; j < JB; ++j) {
        const bool on = pos[j] >= 0 && pos[j] < R_max;
        w[j] = on ? wt[j] : 0.f;  // a dropped slot's gate may be NaN
        const uint4* src = vec_row(rows, on ? pos[j] : 0);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const int64_t c = c0 + (int64_t(i) << sp.lane_bits);
          v[j][i] = on && c < sp.vecs ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
        }
      }
      if (j0 + JB < top_k)
        fetch(t, j0 + JB);
      else
        fetch(u + stride < units ? int64_t((u + stride) / sp.chunks) * per_warp + sub : T, 0);
#pragma unroll
      for (int j = 0; j < JB; ++j)
#pragma unroll
        for (int i = 0; i < kVec; ++i) fma8(acc[i], v[j][i], w[j]);
    }
    if (t >= T) continue;
    uint4* dst = vec_row(y, t);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int64_t c = c0 + (int64_t(i) << sp.lane_bits);
      if (c < sp.vecs) put(dst + c, pack8(acc[i]));
    }
  }
}

// One warp a slot: dys[p] = g dy[t] and the dot product of dy[t] with ys[p].
// Consecutive warps take a token's consecutive slots, so dy[t] comes from L1
// after its first reading.
__global__ void __launch_bounds__(kRowThreads)
unpermute_backward_kernel(RowsIn dy, RowsIn ys, int64_t R_max, int64_t vecs, const int32_t* __restrict__ inv,
                          const float* __restrict__ gates, int64_t slots, int32_t top_k, RowsOut dys,
                          float* __restrict__ dgates) {
  constexpr int kVec = 4;
  const int lane = threadIdx.x & 31;
  const int64_t stride = int64_t(gridDim.x) * (kRowThreads / 32);
  for (int64_t s = int64_t(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5); s < slots; s += stride) {
    const int32_t p = __ldg(inv + s);
    if (p < 0 || p >= R_max) {
      if (lane == 0 && dgates) dgates[s] = 0.f;
      continue;
    }
    const float g = gates ? __ldg(gates + s) : 1.f;
    const uint4* d = vec_row(dy, s / top_k);
    const uint4* r = dgates ? vec_row(ys, p) : nullptr;
    uint4* out = dys.p ? vec_row(dys, p) : nullptr;
    float dot = 0.f;
    for (int64_t c0 = lane; c0 < vecs; c0 += 32 * kVec) {
      uint4 a[kVec], b[kVec];
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int64_t c = c0 + 32 * i;
        if (c < vecs) {
          a[i] = __ldg(d + c);
          if (r) b[i] = __ldg(r + c);
        }
      }
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int64_t c = c0 + 32 * i;
        if (c >= vecs) continue;
        const uint32_t qa[4] = {a[i].x, a[i].y, a[i].z, a[i].w};
        if (out) {
          float f[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 v = unpack_bf16x2(qa[e]);
            f[2 * e] = g * v.x;
            f[2 * e + 1] = g * v.y;
          }
          put(out + c, pack8(f));
        }
        if (r) {
          const uint32_t qb[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 v = unpack_bf16x2(qa[e]), w = unpack_bf16x2(qb[e]);
            dot = fmaf(v.x, w.x, dot);
            dot = fmaf(v.y, w.y, dot);
          }
        }
      }
    }
    if (dgates) {
#pragma unroll
      for (int m = 16; m; m >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m);
      if (lane == 0) dgates[s] = dot;
    }
  }
}

}  // namespace

cudaError_t launch_permute(RowsIn x, int64_t T, int64_t H, const int32_t* perm, int32_t top_k,
                           const int64_t* offsets, int32_t E, int64_t R_max, RowsOut xs, cudaStream_t st, int sms) {
  const RowSplit sp = split_rows(H, 8);
  permute_kernel<8><<<grid_of(R_max, sp, sms, 16), kRowThreads, 0, st>>>(x, T * top_k, sp, perm, top_k, offsets, E,
                                                                     R_max, xs);
  return cudaGetLastError();
}

cudaError_t launch_sum_slots(RowsIn rows, int64_t R_max, int64_t H, const int32_t* inv, const float* gates,
                             int64_t T, int32_t top_k, RowsOut y, cudaStream_t st, int sms) {
  const RowSplit sp = split_rows(H, 2);
  const int grid = grid_of(T, sp, sms, kSumCtas);
  sum_slots_kernel<2, 2><<<grid, kRowThreads, 0, st>>>(rows, R_max, sp, inv, gates, T, top_k, y);
  return cudaGetLastError();
}

cudaError_t launch_unpermute_backward(RowsIn dy, RowsIn ys, int64_t R_max, int64_t H, const int32_t* inv,
                                      const float* gates, int64_t T, int32_t top_k, RowsOut dys, float* dgates,
                                      cudaStream_t st, int sms) {
  const int64_t slots = T * top_k;
  const int64_t want = (slots + kRowThreads / 32 - 1) / (kRowThreads / 32);
  const int64_t cap = int64_t(sms) * 16;
  unpermute_backward_kernel<<<int(want < cap ? want : cap), kRowThreads, 0, st>>>(
      dy, ys, R_max, H / 8, inv, gates, slots, top_k, dys, dgates);
  return cudaGetLastError();
}

}  // namespace e4b
