// The adapters' contractions on the 5th-generation tensor cores: one pass over
// a buffer of bf16 rows z_i, in groups of positions p (i = row ? row[p] : p),
// for either or both of
//   out[p] = w_g W_g z_i            over a row's C columns (s = A x, t = w B^T dy)
//   grad_g = sum_p w_g v[p] z_i^T   over a group's positions (dB from dy, dA from x)
// Both contract the same tile of 128 positions x 128 columns, the first along
// its columns and the second along its rows, so a backward pass reads dy once
// for two results. With r <= 64 the pass moves 2 bytes for every 2 r (out) or
// 6 r (grad) FLOP and is bound by HBM; the tensor cores read the tile from
// shared memory in both directions (K-major and MN-major descriptors of the
// same 128B-swizzled boxes), so no thread touches it.
//
// Numbers: z and W enter as they are (bf16), sums are fp32 in TMEM. The fp32
// values v enter as three bf16 terms hi + mid + lo (24 bits of mantissa, one sign:
// lora_terms.cuh), which makes the fp32 gradients as exact as fp32 products, and
// infinite where these are: two terms left a relative error of 2^-17 a product. The
// terms lie side by side as columns of one B
// operand (N = 3 * rank) up to rank 32, and are added when TMEM is read: three
// MMAs into one accumulator would read the tile from shared memory, and issue,
// three times.
// An MMA truncates its sum, so that n of them in one accumulator leave it 1.2e-8
// n too small (2.1e-6 after 128, measured), and dA inherits t's share. Sums
// therefore leave TMEM after kOutChain column tiles and kGradChain row tiles and
// go on in fp32 additions: within 1e-6, as products and sums of fp32 are.
//
// One persistent CTA per SM. The work is the list of (column block, row tile)
// in that order, cut into equal runs for the CTAs, so that the groups' sizes do
// not unbalance it; a CTA accumulates a group's gradient in TMEM over the
// consecutive row tiles of its run, and writes it to its place when it took all
// the group's tiles, else (the first and last of its run) to a part, with a note
// of whose it is; finish_kernel sums the parts in CTA order: results depend on
// the sizes alone.
//   warp 0       TMA: W's box, and the tile's where its rows lie together (in
//                boxes of 32 rows at a group's end)
//   warp 1       TMEM, the MMAs of out; warp 14 those of grad (an MMA this narrow
//                takes less time than its issue, about 60 cycles: one thread for
//                both took 1.0 us a tile, above the 0.74 us that HBM needs)
//   warps 2-5    v's terms of each row tile, in the operand's layout
//   warps 6-9    TMEM to out and grad
//   warps 10-13  mapped rows, by cp.async into the same swizzled boxes (four-row
//                TMA gathers took 45 ns each: three times as long as whole boxes);
//                without a map they share the terms
//   warp 15      zeros in place of the rows behind a group's end that a gradient's
//                MMAs read, so that no other group's values meet these
// s of 65536 rows of 2048, rank 16 or 32: 54 us (5.0 TB/s); t and dB of 8192 rows of
// 28672, rank 16: 94 to 100 us (4.7 to 5.0 TB/s), t or dB alone 85 to 94; rank 64:
// 280 us, where 24 MMAs and 48 KB of terms a tile leave no slack.
// Every wait is bounded; one that gives up records E4B_ERR_DEVICE_TIMEOUT,
// stops all roles, drains the copies and MMAs in flight, frees TMEM and returns.
#include <cuda.h>

#include <type_traits>

#include "common.cuh"
#include "lora_tc.h"
#include "lora_terms.cuh"
#include "lora_walk.cuh"
#include "sm100.cuh"
#include "tmap.h"

namespace e4b {
namespace {

using namespace sm100;

constexpr int kThreads = 512;
constexpr int kLoadWarp = 10, kLoadWarps = 4, kGradWarp = 14, kZeroWarp = 15;
constexpr int kNoteThread = 8 * 32;              // of the results' warps, writes the CTA's notes
static_assert(kTile == 128, "positions, and columns, of an operand tile");
constexpr uint32_t kBox = kTile * 128;           // bytes of 128 rows of 64 columns
constexpr int kEdge = 32;                        // rows of the boxes at a group's end
constexpr uint32_t kZBytes = 2 * kBox;           // a tile
constexpr int kOutChain = 2, kGradChain = 8;     // tiles of eight MMAs
// TMEM columns of a tile's gradient: the three terms' sums, or above rank 32,
// where these would leave room for two tiles, hi's and the others'.
__host__ __device__ constexpr int grad_width(int rp) { return rp <= 32 ? 3 * rp : 2 * rp; }
constexpr int kMaxStages = 6;
constexpr int kMaxChunks = 512 / grad_width(16); // column tiles of a block whose gradients TMEM holds, at most
constexpr uint32_t kSmemLimit = 232448;

// A part of a gradient: its group and column block, and whether it is the first
// of the group's. group < 0: none.
struct Note {
  int32_t group, block, first;
};

struct Pass {
  int64_t C, R_max, rows, ld_z;
  const uint16_t* z;
  const int64_t* offsets;
  const int32_t* row;
  const float* scale;
  float* out;
  const float* v;
  float* grad;
  float* grad_part;
  Note* notes;  // of the parts, two a CTA
  int32_t* status;
  int G, r;
  int blocks, chunks;  // column blocks; column tiles of a block
  int stages, vbufs;
  uint32_t limit;
  uint8_t w_t, scale_out, scale_v, grad_t, accumulate, follows;
};

// Shared memory, from a 1024-byte boundary: stages of (tile, W's box), the
// buffers of v's terms, then barriers and scalars.
struct Layout {
  uint32_t stage, terms, misc, total;
};
__host__ __device__ inline Layout layout_of(const Pass& p, bool out, bool grad, int rp) {
  Layout l;
  l.stage = kZBytes + (out ? 2 * kTile * rp : 0);
  l.terms = l.stage * p.stages;
  l.misc = l.terms + (grad ? p.vbufs * 6 * kTile * rp : 0);
  l.total = l.misc + 1024 + 1024;  // barriers and scalars, alignment
  return l;
}

// Shared-memory descriptors, built once: a step adds its bytes / 16 to the low
// word (the address field cannot overflow into its neighbour below 256 KB).
// Without swizzle: core matrices of 8 x 16 bytes, lbo bytes apart along K and
// sbo along M or N.
E4B_DEV uint64_t plain_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t((lbo >> 4) & 0x3FFFu) << 16) |
         (uint64_t((sbo >> 4) & 0x3FFFu) << 32) | (uint64_t(1) << 46);
}
// MN-major, one swizzle span (32, 64 or 128 bytes) wide: 8 K-rows of a span
// after one another.
E4B_DEV uint64_t span_desc(uint32_t saddr, uint32_t span) {
  const uint64_t layout = span == 128 ? 2 : span == 64 ? 4 : 6;
  return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t(1) << 16) | (uint64_t((8 * span) >> 4) << 32) |
         (uint64_t(1) << 46) | (layout << 61);
}
E4B_DEV uint64_t step_desc(uint64_t d, uint32_t bytes) {
  return (d & 0xFFFFFFFF00000000ull) | uint32_t(uint32_t(d) + (bytes >> 4));
}

// A slot of a ring and the parity of its use, without a division.
struct Ring {
  int n, slot = 0;
  uint32_t parity = 0;
  E4B_DEV explicit Ring(int slots) : n(slots) {}
  E4B_DEV void next() {
    if (++slot == n) {
      slot = 0;
      parity ^= 1u;
    }
  }
};

// A warp's wait: one lane polls.
E4B_DEV bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t limit, const volatile int* abort) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = mbar_wait_bounded(bar, parity, limit, abort);
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// Eight values as three bf16 terms.
E4B_DEV void split3(float4 x, float4 y, float w, uint4 (&t)[3]) {
  const float v[8] = {w * x.x, w * x.y, w * x.z, w * x.w, w * y.x, w * y.y, w * y.z, w * y.w};
  uint32_t q[4][3];
#pragma unroll
  for (int i = 0; i < 4; ++i) split_pair(v[2 * i], v[2 * i + 1], q[i]);
#pragma unroll
  for (int k = 0; k < 3; ++k) t[k] = make_uint4(q[0][k], q[1][k], q[2][k], q[3][k]);
}

template <bool OUT, bool GRAD, int RP>  // RP: the rank's operand width, 16, 32 or 64
__global__ void __launch_bounds__(kThreads, 1)
contract_kernel(const __grid_constant__ CUtensorMap tm_tile, const __grid_constant__ CUtensorMap tm_edge,
                const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ Pass p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const Layout lay = layout_of(p, OUT, GRAD, RP);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + lay.misc);
  uint64_t* loaded = full + kMaxStages;
  uint64_t* empty = loaded + kMaxStages;
  uint64_t* t_full = empty + kMaxStages;
  uint64_t* t_empty = t_full + 2;
  uint64_t* v_full = t_empty + 2;
  uint64_t* v_empty = v_full + 2;
  uint64_t* g_full = v_empty + 2;
  uint64_t* drained = g_full + 1;      // [2]
  uint64_t* g_empty = drained + 2;     // [kMaxChunks]
  int64_t* s_sum = reinterpret_cast<int64_t*>(g_empty + kMaxChunks);  // [kThreads / 32]
  int64_t* s_start = s_sum + kThreads / 32;                           // group, tile
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(s_start + 2);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    if (!p.row) {
      prefetch_tensormap(&tm_tile);
      prefetch_tensormap(&tm_edge);
    }
    if (OUT) prefetch_tensormap(&tm_w);
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&loaded[s], p.row ? kLoadWarps : 1);
      mbar_init(&empty[s], OUT && GRAD ? 2 : 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&t_full[b], 1);
      mbar_init(&t_empty[b], 128);
      mbar_init(&drained[b], 1);
      mbar_init(&v_full[b], p.row ? 128 : 256);
      mbar_init(&v_empty[b], 1);
    }
    mbar_init(g_full, 1);
    if (GRAD)
      for (int c = 0; c < p.chunks; ++c) mbar_init(&g_empty[c], 128);
    *s_abort = 0;
    mbar_init_fence();
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  // offsets do not come from the launch before this one where that is a part of
  // the same call, which has itself waited for all earlier work
  if (!p.follows) grid_dependency_wait();
  const Run run = find_run<kThreads>(p.offsets, p.G, p.R_max, p.blocks, FullTile{}, s_sum, s_start);  // has barriers
  if (p.follows) grid_dependency_wait();
  grid_launch_dependents();
  if (GRAD && tid == kNoteThread) p.notes[2 * blockIdx.x] = p.notes[2 * blockIdx.x + 1] = Note{-1, 0, 0};
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const int64_t count = run.count;
  if (count == 0) {  // uniform
    if (warp == 1) tmem_dealloc(tmem, 512);
    return;
  }

  const int all_chunks = int((p.C + kTile - 1) / kTile);
  constexpr int rp = RP;
  constexpr bool side_by_side = RP <= 32;  // all three terms, or hi and mid + lo
  constexpr int gw = grad_width(RP);       // TMEM columns of a tile's gradient
  const uint32_t d_grad = tmem + (OUT ? 2 * rp : 0);
  Walk<FullTile> wk(p.offsets, p.G, p.R_max, run, FullTile{}, s_start);
  auto chunks_of = [&](int cb) { return min(p.chunks, all_chunks - cb * p.chunks); };
  auto give_up = [&]() {
    *s_abort = 1;
    record_status(p.status, E4B_ERR_DEVICE_TIMEOUT);
  };

  // Between a stage's copies and its MMAs along the positions there is always a
  // warp that completes it (`loaded`): a parity wait must never be two uses of
  // its barrier away, so no role may skip stages that another walks. The MMAs
  // along the columns take the stage as TMA completes it, with rows past a
  // group's end that only make results that are not written.
  // rows of the tile that the MMAs read, or whose results count
  auto rows_read = [&]() { return GRAD ? (wk.n() + 15) / 16 * 16 : wk.n(); };

  // v's terms, by four warps or (without a map) eight. A thread takes eights of a
  // position's values, GR of which the operand has. Neighbouring lanes take eight
  // positions, whose 16-byte stores fill a line of banks, by up to four eights, so
  // that a load touches whole sectors of few lines. The terms are made before the
  // wait for their buffer.
  auto terms_by = [&](auto warps, int first) {
    constexpr int GR = RP / 8, LG = GR < 4 ? GR : 4;  // eights of a position; of them side by side in a warp
    constexpr int LP = 32 / LG, PS = kTile / warps.value / LP, UNITS = PS * (GR / LG);  // positions side by side, after one another
    const int eight0 = (lane >> 3) % LG, m0 = first * (kTile / warps.value) + (lane >> 3) / LG * 8 + (lane & 7);
    Ring vr(p.vbufs);
    for (int64_t k = 0; k < count; ++k) {
      const int64_t row0 = wk.row0();
      const int n = wk.n();
      const float w = p.scale_v && p.scale ? __ldg(p.scale + wk.g) : 1.f;
      float4 x[UNITS][2];
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        const int m = m0 + u % PS * LP, j = 8 * (eight0 + u / PS * LG);
        bool in = m < n && j < p.r;
        if (in && p.row) {
          const int32_t at = __ldg(p.row + row0 + m);
          in = at >= 0 && at < p.rows;
        }
        const float4* from = reinterpret_cast<const float4*>(p.v + (row0 + m) * p.r + j);
        x[u][0] = in ? __ldg(from) : make_float4(0.f, 0.f, 0.f, 0.f);
        x[u][1] = in ? __ldg(from + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      uint4 t[UNITS][3];
#pragma unroll
      for (int u = 0; u < UNITS; ++u) split3(x[u][0], x[u][1], w, t[u]);
      if (!warp_wait(&v_empty[vr.slot], vr.parity ^ 1u, p.limit, s_abort)) {
        give_up();
        break;
      }
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        const int m = m0 + u % PS * LP, eight = eight0 + u / PS * LG;
        uint8_t* dst = smem + lay.terms + vr.slot * 6 * kTile * rp + ((m >> 3) * (3 * GR) + eight) * 128 + (m & 7) * 16;
#pragma unroll
        for (int q = 0; q < 3; ++q) *reinterpret_cast<uint4*>(dst + q * GR * 128) = t[u][q];
      }
      fence_proxy_async_smem();
      mbar_arrive(&v_full[vr.slot]);
      vr.next();
      if (k + 1 < count) wk.next();
    }
  };
  auto make_terms = [&](int first) {
    if constexpr (GRAD) {
      if (p.row) terms_by(std::integral_constant<int, 4>{}, first);
      else terms_by(std::integral_constant<int, 8>{}, first);
    }
  };

  // The MMAs that this thread issued, and their arrivals, have to finish before TMEM
  // is freed and the CTA ends. No other role's end says so: one that gives up after
  // this thread's last issue does not wait for it.
  auto drain = [&](uint64_t* bar) {
    mma_commit(bar);
    mbar_wait_bounded(bar, 0, kWaitPolls, nullptr);
  };

  if (warp == 0) {
    // ------------------------------------------------------------ TMA
    // Mapped rows of a gradient alone need no copy, and nobody waits for `full`:
    // walking their stages this thread could fall a whole ring behind.
    if (lane == 0 && (OUT || !p.row)) {
      Ring st(p.stages);
      int64_t i = 0;
      bool aborted = false;
      for (int64_t k = 0; k < count && !aborted; ++k) {
        const int32_t row0 = int32_t(wk.row0());
        const int edges = p.row ? 0 : (rows_read() + kEdge - 1) / kEdge;
        const uint32_t bytes = edges * (kEdge * 256) + (OUT ? 2 * kTile * rp : 0);
        const int nc = chunks_of(wk.cb);
        int32_t x = wk.cb * p.chunks * kTile;
        for (int c = 0; c < nc; ++c, ++i, x += kTile, st.next()) {
          if (!mbar_wait_bounded(&empty[st.slot], st.parity ^ 1u, p.limit, s_abort)) {
            give_up();
            aborted = true;
            break;
          }
          uint64_t* bar = &full[st.slot];
          uint8_t* dst = smem + st.slot * lay.stage;
          mbar_arrive_expect_tx(bar, bytes);
          if (edges == kTile / kEdge) {
            tma_load_2d(dst, &tm_tile, bar, x, row0);
            tma_load_2d(dst + kBox, &tm_tile, bar, x + 64, row0);
          } else {
            for (int e = 0; e < edges; ++e) {
              tma_load_2d(dst + e * kEdge * 128, &tm_edge, bar, x, row0 + e * kEdge);
              tma_load_2d(dst + e * kEdge * 128 + kBox, &tm_edge, bar, x + 64, row0 + e * kEdge);
            }
          }
          if (OUT) {
            if (p.w_t) {
              tma_load_3d(dst + kZBytes, &tm_w, bar, 0, x, wk.g);
            } else {
              tma_load_3d(dst + kZBytes, &tm_w, bar, x, 0, wk.g);
              tma_load_3d(dst + kZBytes + 128 * rp, &tm_w, bar, x + 64, 0, wk.g);
            }
          }
        }
        if (k + 1 < count) wk.next();
      }
      // every copy issued has to land before the CTA can exit
      for (int64_t q = i > p.stages ? i - p.stages : 0; q < i; ++q)
        mbar_wait_bounded(&full[q % p.stages], uint32_t(q / p.stages) & 1u, kWaitPolls, nullptr);
    }
  } else if (warp == 1) {
    // ------------------------------------------------- MMAs along the columns
    if (OUT && lane == 0) {
      const uint32_t id = idesc_bf16_f32(kTile, rp) | (p.w_t ? 1u << 16 : 0u);
      // W's steps along its 128 columns: 16 of them, 64 of them
      const uint32_t w_step = p.w_t ? 32 * rp : 32, w_half = 128 * rp;
      const uint32_t z0 = smem_u32(smem);
      const uint64_t zd0 = sw128_kmajor_desc(z0);
      const uint64_t wd0 = p.w_t ? span_desc(z0 + kZBytes, 2 * rp) : sw128_kmajor_desc(z0 + kZBytes);
      Ring st(p.stages), tr(2);
      bool aborted = false;
      for (int64_t k = 0; k < count && !aborted; ++k) {
        const int nc = chunks_of(wk.cb);
        for (int c = 0; c < nc; ++c, st.next()) {
          const int link = c % kOutChain;
          if (!mbar_wait_bounded(&full[st.slot], st.parity, p.limit, s_abort) ||
              (p.row && !mbar_wait_bounded(&loaded[st.slot], st.parity, p.limit, s_abort)) ||
              (link == 0 && !mbar_wait_bounded(&t_empty[tr.slot], tr.parity ^ 1u, p.limit, s_abort))) {
            give_up();
            aborted = true;
            break;
          }
          tc_fence_after();
          const uint32_t at = st.slot * lay.stage, d = tmem + tr.slot * rp;
          const uint64_t zd = step_desc(zd0, at), wd = step_desc(wd0, at);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_bf16_ss(d, step_desc(zd, (kk >> 2) * kBox + (kk & 3) * 32),
                        step_desc(wd, uint32_t(kk >> 2) * w_half + uint32_t(kk & 3) * w_step), id, (link | kk) ? 1u : 0u);
          mma_commit(&empty[st.slot]);
          if (link == kOutChain - 1 || c + 1 == nc) {
            mma_commit(&t_full[tr.slot]);
            tr.next();
          }
        }
        if (k + 1 < count) wk.next();
      }
      drain(&drained[0]);
    }
  } else if (warp == kGradWarp) {
    // ----------------------------------------------- MMAs along the positions
    if (GRAD && lane == 0) {
      constexpr uint32_t mn_major = (1u << 15) | (1u << 16);  // both operands
      const uint32_t id = idesc_bf16_f32(kTile, gw) | mn_major, id_lo = idesc_bf16_f32(kTile, rp) | mn_major;
      constexpr uint32_t vk = uint32_t(3 * rp / 8) * 128;  // bytes of 8 positions of v's terms
      const uint32_t z0 = smem_u32(smem);
      const uint64_t zd0 = sw128_mnmajor_desc(z0, kBox, 1024), vd0 = plain_desc(z0 + lay.terms, vk, 128);
      Ring st(p.stages), vr(p.vbufs);
      uint32_t g_phase = 0;
      bool aborted = false;
      bool fresh = true;  // first row tile of a chain
      int chain = 0;
      for (int64_t k = 0; k < count && !aborted; ++k) {
        if (!mbar_wait_bounded(&v_full[vr.slot], vr.parity, p.limit, s_abort)) {
          give_up();
          break;
        }
        const int steps = (wk.n() + 15) / 16;
        const int nc = chunks_of(wk.cb);
        const uint64_t vd = step_desc(vd0, vr.slot * 6 * kTile * rp);
        uint32_t d = d_grad;
        for (int c = 0; c < nc; ++c, d += gw, st.next()) {
          if (!mbar_wait_bounded(&loaded[st.slot], st.parity, p.limit, s_abort) ||
              (fresh && !mbar_wait_bounded(&g_empty[c], ((g_phase >> c) & 1u) ^ 1u, p.limit, s_abort))) {
            give_up();
            aborted = true;
            break;
          }
          tc_fence_after();
          if (fresh) g_phase ^= 1u << c;
          const uint64_t zd = step_desc(zd0, st.slot * lay.stage);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            if (kk >= steps) break;
            const uint64_t zs = step_desc(zd, kk * 2048), vs = step_desc(vd, kk * 2 * vk);
            mma_bf16_ss(d, zs, vs, id, !fresh || kk ? 1u : 0u);
            if constexpr (!side_by_side) mma_bf16_ss(d + rp, zs, step_desc(vs, 32 * rp), id_lo, 1u);
          }
          mma_commit(&empty[st.slot]);
        }
        if (aborted) break;
        mma_commit(&v_empty[vr.slot]);
        fresh = ++chain == kGradChain || wk.last();
        if (fresh || k + 1 == count) mma_commit(g_full);
        if (fresh) chain = 0;
        vr.next();
        if (k + 1 < count) wk.next();
      }
      drain(&drained[1]);
    }
  } else if (warp < 6) {
    make_terms(warp - 2);
  } else if (warp >= kLoadWarp && warp < kLoadWarp + kLoadWarps) {
    // -------------------------------------------- mapped rows, or v's terms
    const int w4 = warp - kLoadWarp;
    if (!p.row) {
      make_terms(4 + w4);
    } else {
      // A warp copies 32 rows of the tile, two at a time, and tells of a stage
      // when the copies of the stages after it are under way too.
      const int m0 = w4 * 32, hi = lane >> 4, piece = lane & 15;  // 16 bytes of a row's 256
      Ring st(p.stages), told(p.stages);
      int pending = 0;
      bool aborted = false;
      auto tell = [&]() {  // the copies of the oldest stage have landed
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&loaded[told.slot]);
        told.next();
        --pending;
      };
      for (int64_t k = 0; k < count && !aborted; ++k) {
        const int n = wk.n(), rows = rows_read();
        int32_t at = -1;  // row m0 + lane
        if (m0 + lane < n) {
          at = __ldg(p.row + wk.row0() + m0 + lane);
          if (at >= p.rows) at = -1;
        }
        const uint16_t* src[16];  // of rows m0 + 2 u + hi; those of no position read as zeros
        uint32_t on = 0;
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          const int32_t row = __shfl_sync(0xffffffffu, at, 2 * u + hi);
          if (row >= 0) on |= 1u << u;
          src[u] = p.z + (row >= 0 ? int64_t(row) * p.ld_z + 8 * piece : 0);
        }
        const int nc = chunks_of(wk.cb);
        int64_t x = int64_t(wk.cb) * p.chunks * kTile;
        for (int c = 0; c < nc; ++c, x += kTile, st.next()) {
          if (!warp_wait(&empty[st.slot], st.parity ^ 1u, p.limit, s_abort)) {
            give_up();
            aborted = true;
            break;
          }
          const bool in = x + 8 * piece < p.C;
          uint8_t* dst = smem + st.slot * lay.stage + (piece >> 3) * kBox + (m0 + hi) * 128;
#pragma unroll
          for (int u = 0; u < 16; ++u) {
            if (m0 + 2 * u + hi >= rows) continue;
            const bool yes = in && (on >> u & 1u);
            cp_async_16(dst + u * 256 + (((piece & 7) ^ ((2 * u + hi) & 7)) << 4), yes ? src[u] + x : p.z, yes ? 16 : 0);
          }
          cp_async_commit();
          ++pending;
          if (p.stages > 3) {
            if (pending > 3) {
              cp_async_wait<3>();
              tell();
            }
          } else if (pending > 2) {
            cp_async_wait<2>();
            tell();
          }
        }
        if (k + 1 < count) wk.next();
      }
      cp_async_wait_all();
      while (pending) tell();
    }
  } else if (warp == kZeroWarp) {
    // ------- zeros behind a group's last row, up to the MMA's next step of 16
    if (GRAD && !p.row) {
      Ring st(p.stages);
      bool aborted = false;
      for (int64_t k = 0; k < count && !aborted; ++k) {
        const int n = wk.n(), rows = rows_read(), nc = chunks_of(wk.cb);
        for (int c = 0; c < nc; ++c, st.next()) {
          if (!warp_wait(&full[st.slot], st.parity, p.limit, s_abort)) {
            give_up();
            aborted = true;
            break;
          }
          if (n < rows) {
            uint8_t* z = smem + st.slot * lay.stage + (lane >> 3 & 1) * kBox + (lane & 7) * 16;
            for (int m = n + (lane >> 4); m < rows; m += 2) *reinterpret_cast<uint4*>(z + m * 128) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(&loaded[st.slot]);
        }
        if (k + 1 < count) wk.next();
      }
    }
  } else {
    // ---------------------------------------------------- results from TMEM
    const int q = warp & 3;  // the TMEM lanes this warp may read
    const int m = q * 32 + lane;
    const uint32_t lanes = uint32_t(q * 32) << 16;
    Ring tr(2);
    uint32_t chains = 0;
    int chain = 0;
    bool direct = false, later = false;  // the gradient goes to its place; it is there in part
    int part = 0;
    for (int64_t k = 0; k < count; ++k) {
      if constexpr (OUT) {
        float sum[RP];
        const int nc = chunks_of(wk.cb);
        bool ok = true;
        for (int c = 0; c < nc; c += kOutChain, tr.next()) {
          ok = warp_wait(&t_full[tr.slot], tr.parity, p.limit, s_abort);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int j0 = 0; j0 < RP; j0 += 16) {
            uint32_t v[16];
            tmem_ld_32x32b_x16(tmem + lanes + tr.slot * rp + j0, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) sum[j0 + j] = c ? sum[j0 + j] + __uint_as_float(v[j]) : __uint_as_float(v[j]);
          }
          tc_fence_before();
          mbar_arrive(&t_empty[tr.slot]);
        }
        if (!ok) {
          give_up();
          break;
        }
        const float w = p.scale_out && p.scale ? __ldg(p.scale + wk.g) : 1.f;
        float* dst = p.out + (int64_t(wk.cb) * p.R_max + wk.row0() + m) * p.r;
#pragma unroll
        for (int j = 0; j < RP; j += 4)
          if (m < wk.n() && j < p.r)
            *reinterpret_cast<float4*>(dst + j) = make_float4(w * sum[j], w * sum[j + 1], w * sum[j + 2], w * sum[j + 3]);
      }
      if constexpr (GRAD) {
        if (k == 0 || wk.first()) {  // the next gradient of this run
          direct = wk.first() && wk.tiles <= count - k;
          later = false;
          part = 2 * int(blockIdx.x) + (k ? 1 : 0);
          if (!direct && tid == kNoteThread) p.notes[part] = Note{wk.g, wk.cb, wk.first()};
        }
        const bool fresh = ++chain == kGradChain || wk.last();
        if (fresh || k + 1 == count) {
          chain = 0;
          if (!warp_wait(g_full, chains++ & 1u, p.limit, s_abort)) {
            give_up();
            break;
          }
          tc_fence_after();
          const int64_t block = int64_t(p.chunks) * kTile;  // columns of a part
          const int64_t col0 = direct ? wk.cb * block : 0, width = direct ? p.C : block;
          float* dst = direct ? p.grad + int64_t(wk.g) * p.C * p.r : p.grad_part + part * block * p.r;
          const bool add = later || (direct && p.accumulate);
          later = true;
          // this thread's column of chunk c: its rank's values lie `step` apart
          const int nc = chunks_of(wk.cb);
          const int64_t left = p.C - wk.cb * block - m;  // chunk c is within the columns where 128 c < left
          float* at = dst + (p.grad_t ? (col0 + m) * p.r : col0 + m);
          const int64_t chunk_step = p.grad_t ? int64_t(kTile) * p.r : kTile;
          float old[16];  // what the next values are added to
          auto fetch_old = [&](int c, int j0) {
            const float* o = at + c * chunk_step;
            const bool in = add && c < nc && c * kTile < left;
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              if (p.grad_t) {
                const float4 v = in && j0 + j < p.r ? *reinterpret_cast<const float4*>(o + j0 + j) : make_float4(0.f, 0.f, 0.f, 0.f);
                old[j] = v.x;
                old[j + 1] = v.y;
                old[j + 2] = v.z;
                old[j + 3] = v.w;
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) old[j + i] = in && j0 + j < p.r ? o[(j0 + j + i) * width] : 0.f;
              }
            }
          };
          if (add) fetch_old(0, 0);
          for (int c = 0; c < nc; ++c) {
#pragma unroll
            for (int j0 = 0; j0 < RP; j0 += 16) {
              float f[16];
              uint32_t v[16];
              const uint32_t from = d_grad + lanes + uint32_t(c * gw + j0);
              tmem_ld_32x32b_x16(from, v);
              uint32_t v1[16];
              tmem_ld_32x32b_x16(from + rp, v1);
              if constexpr (side_by_side) {
                uint32_t v2[16];
                tmem_ld_32x32b_x16(from + 2 * rp, v2);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  f[j] = (__uint_as_float(v2[j]) + __uint_as_float(v1[j])) + __uint_as_float(v[j]);
              } else {
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) f[j] = __uint_as_float(v1[j]) + __uint_as_float(v[j]);
              }
              if (j0 + 16 >= RP) {
                tc_fence_before();
                mbar_arrive(&g_empty[c]);
              }
              if (add) {
#pragma unroll
                for (int j = 0; j < 16; ++j) f[j] += old[j];
                if (j0 + 16 < RP) fetch_old(c, j0 + 16);
                else fetch_old(c + 1, 0);
              }
              if (c * kTile >= left) continue;
              float* o = at + c * chunk_step;
#pragma unroll
              for (int j = 0; j < 16; j += 4) {
                if (j0 + j >= p.r) break;
                if (p.grad_t) {
                  *reinterpret_cast<float4*>(o + j0 + j) = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
                } else {
#pragma unroll
                  for (int i = 0; i < 4; ++i) o[(j0 + j + i) * width] = f[j + i];
                }
              }
            }
          }
        }
      }
      if (k + 1 < count) wk.next();
    }
  }

  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The gradients that several CTAs share (the parts' sum, in CTA order) and
// those of groups without rows (zero).
struct Finish {
  Pass p;
  int ctas;  // of the pass; 0 where there were no rows
};

// The parts that begin in CTA b of the pass: each goes on in the first parts of
// the CTAs after it. kFinishVecs vectors a thread, in flight together.
constexpr int kFinishThreads = 256, kFinishVecs = 4;
E4B_DEV void finish_parts(const Finish& f, int b) {
  const Pass& p = f.p;
  __shared__ int s_last;
  const int64_t block = int64_t(p.chunks) * kTile, part = block * p.r;
  const Note notes[2] = {p.notes[2 * b], p.notes[2 * b + 1]};
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    const Note note = k ? notes[1] : notes[0];
    if (note.group < 0 || !note.first) continue;  // uniform
    __syncthreads();
    if (threadIdx.x == 0) s_last = f.ctas - 1;
    __syncthreads();
    for (int c = b + 1 + threadIdx.x; c < f.ctas; c += kFinishThreads) {  // the first CTA that does not go on with it
      const Note more = p.notes[2 * c];
      if (more.group != note.group || more.block != note.block || more.first) atomicMin(&s_last, c - 1);
    }
    __syncthreads();
    const int last = s_last;
    const int64_t c0 = note.block * block;
    const int cols = int(min(block, p.C - c0));
    // values that lie together: the block's columns by r, or r rows of its columns
    const int len4 = (p.grad_t ? cols * p.r : cols) / 4, lines = p.grad_t ? 1 : p.r;
    float* dst = p.grad + int64_t(note.group) * p.C * p.r + (p.grad_t ? c0 * p.r : c0);
    const int total = lines * len4, step = kFinishThreads * int(gridDim.y);
    for (int i0 = int(blockIdx.y) * kFinishThreads + int(threadIdx.x); i0 < total; i0 += kFinishVecs * step) {
      float4 s[kFinishVecs];
      int64_t src[kFinishVecs], to[kFinishVecs];
#pragma unroll
      for (int v = 0; v < kFinishVecs; ++v) {
        const int i = i0 + v * step, line = i / len4, at = (i - line * len4) * 4;
        to[v] = i < total ? line * p.C + at : -1;
        src[v] = line * block + at;
        s[v] = p.accumulate && to[v] >= 0 ? *reinterpret_cast<const float4*>(dst + to[v]) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll 2
      for (int c = b; c <= last; ++c) {
        const float* from = p.grad_part + (2 * c + (c == b ? k : 0)) * part;
#pragma unroll
        for (int v = 0; v < kFinishVecs; ++v) {
          if (to[v] < 0) continue;
          const float4 z = __ldg(reinterpret_cast<const float4*>(from + src[v]));
          s[v] = make_float4(s[v].x + z.x, s[v].y + z.y, s[v].z + z.z, s[v].w + z.w);
        }
      }
#pragma unroll
      for (int v = 0; v < kFinishVecs; ++v)
        if (to[v] >= 0) *reinterpret_cast<float4*>(dst + to[v]) = s[v];
    }
  }
}

// This CTA's share of the gradients of group g, which has no rows.
E4B_DEV void finish_empty(const Pass& p, int g) {
  const int64_t n4 = p.C * p.r / 4;
  float4* dst = reinterpret_cast<float4*>(p.grad) + int64_t(g) * n4;
  for (int64_t i = int64_t(blockIdx.x) * kFinishThreads + threadIdx.x; i < n4; i += int64_t(gridDim.x) * kFinishThreads)
    dst[i] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// CTAs (x, y): piece y of the first pass' parts, then of the second's; those of the
// first pieces share the groups without rows.
__global__ void __launch_bounds__(kFinishThreads)
finish_kernel(const __grid_constant__ Finish a, const __grid_constant__ Finish b) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int x = blockIdx.x;
  if (x < a.ctas) finish_parts(a, x);
  else if (x < a.ctas + b.ctas) finish_parts(b, x - a.ctas);
  if (a.p.accumulate || blockIdx.y) return;
  const Pass& p = a.p;
  __shared__ uint32_t s_empty[kFinishThreads / 32];
  for (int g0 = 0; g0 < p.G; g0 += kFinishThreads) {
    const int g = g0 + int(threadIdx.x);
    int64_t beg, end;
    const uint32_t empty = __ballot_sync(0xffffffffu, g < p.G && group_tiles(p.offsets, g, p.R_max, beg, end, FullTile{}) == 0);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_empty[threadIdx.x >> 5] = empty;
    __syncthreads();
    for (int w = 0; w < kFinishThreads / 32; ++w)
      for (uint32_t left = s_empty[w]; left; left &= left - 1) {
        const int k = g0 + 32 * w + __ffs(left) - 1;
        finish_empty(a.p, k);
        if (b.p.grad) finish_empty(b.p, k);
      }
  }
}

// ---------------------------------------------------------------- the plan
struct Plan {
  int rp, chunks, blocks, vbufs, stages;
};

int operand_width(int r) { return r <= 16 ? 16 : r <= 32 ? 32 : 64; }

// The choices of a pass' column tiles a block: at most those whose gradients TMEM
// holds; without a gradient up to 64, in steps that grow (this runs on the host
// for every call).
struct Choices {
  int r, sms, most;
  int64_t all;  // column tiles
  bool out, grad;
  Choices(int rank, int64_t C, bool o, bool g, int n) : r(rank), sms(n), all((C + kTile - 1) / kTile), out(o), grad(g) {
    const int rp = operand_width(rank);
    most = g ? (512 - (o ? 2 * rp : 0)) / grad_width(rp) : 64;
    if (most > all) most = int(all);
  }
  int after(int c) const { return c + (grad || c < 4 ? 1 : c < 16 ? 4 : 16); }
  int64_t blocks(int c) const { return (all + c - 1) / c; }
  // The estimated time, in units of one tile's 32 KB from HBM: the longest run's
  // items (for each, besides its tiles, half a unit, or with a gradient of a wide
  // rank, whose terms have one buffer, more), the last gradients' way out of TMEM,
  // the parts of `out` written and read again.
  double item(int c) const { return double(c) + (grad && operand_width(r) == 64 ? 1.5 : 0.5); }
  double last(int c) const { return grad ? 0.5 * double(c) : 0.0; }
  double parts(int c) const { return out && blocks(c) > 1 ? double(blocks(c)) * r / (32.0 * sms) : 0.0; }
  double time(int c, int64_t tiles) const {
    return double((blocks(c) * tiles + sms - 1) / sms) * item(c) + last(c) + parts(c) * double(tiles);
  }
};

// Row tiles, an estimate: groups may end anywhere in one. Never fewer for more rows.
int64_t row_tiles(int G, int64_t R_max) {
  const int64_t groups = G < R_max ? G : R_max, tiles = R_max / kTile + (groups + 1) / 2;
  return tiles < groups ? groups : tiles;
}

Plan plan_of(int G, int r, int64_t C, int64_t R_max, bool out, bool grad, int sms) {
  Plan q;
  q.rp = operand_width(r);
  const Choices ch(r, C, out, grad, sms);
  const int64_t tiles = row_tiles(G, R_max);
  double best = 0;
  q.chunks = 0;
  for (int c = 1; c <= ch.most; c = ch.after(c)) {
    const double t = ch.time(c, tiles);
    if (!q.chunks || t <= best) {
      best = t;
      q.chunks = c;
    }
  }
  q.blocks = int(ch.blocks(q.chunks));
  q.vbufs = q.rp <= 32 ? 2 : 1;
  const int64_t terms = grad ? int64_t(q.vbufs) * 6 * kTile * q.rp : 0;
  const int64_t stage = kZBytes + (out ? 2 * kTile * q.rp : 0);
  q.stages = int((int64_t(kSmemLimit) - 2048 - terms) / stage);
  if (q.stages > kMaxStages) q.stages = kMaxStages;
  return q;
}

int64_t part_floats(int r, int chunks, int sms) { return int64_t(2) * sms * chunks * kTile * r; }

Pass pass_of(const ContractArgs& a, const Plan& q, int sms) {
  Pass p{};
  p.C = a.C;
  p.R_max = a.R_max;
  p.rows = a.row ? a.rows : a.R_max;
  p.ld_z = a.ld_z;
  p.z = a.z;
  p.offsets = a.offsets;
  p.row = a.row;
  p.scale = a.scale;
  p.out = a.out;
  p.v = a.v;
  p.grad = a.grad;
  p.grad_part = a.grad_part;
  p.notes = a.grad ? reinterpret_cast<Note*>(a.grad_part + part_floats(a.r, q.chunks, sms)) : nullptr;
  p.status = a.status;
  p.G = a.G;
  p.r = a.r;
  p.blocks = q.blocks;
  p.chunks = q.chunks;
  p.stages = q.stages;
  p.vbufs = q.vbufs;
  p.limit = a.no_wait ? 0u : kWaitPolls;
  p.w_t = a.w_t;
  p.scale_out = a.scale_out;
  p.scale_v = a.scale_v;
  p.grad_t = a.grad_t;
  p.accumulate = a.accumulate;
  p.follows = a.follows;
  return p;
}

template <bool OUT, bool GRAD, int RP>
cudaError_t launch(const CUtensorMap& tile, const CUtensorMap& edge, const CUtensorMap& w, const Pass& p, cudaStream_t st, int sms) {
  auto kernel = contract_kernel<OUT, GRAD, RP>;
  const uint32_t smem = layout_of(p, OUT, GRAD, RP).total;
  static SmemAllowed allowed;
  const cudaError_t err = allow_smem(kernel, int(kSmemLimit), allowed);
  if (err != cudaSuccess) return err;
  return launch_dependent(kernel, dim3(sms), dim3(kThreads), smem, st, tile, edge, w, p);
}

template <int RP>
cudaError_t launch_as(const ContractArgs& a, const CUtensorMap& tile, const CUtensorMap& edge, const CUtensorMap& w,
                      const Pass& p, cudaStream_t st, int sms) {
  if (!a.grad) return launch<true, false, RP>(tile, edge, w, p, st, sms);
  if (!a.out) return launch<false, true, RP>(tile, edge, w, p, st, sms);
  return launch<true, true, RP>(tile, edge, w, p, st, sms);
}

}  // namespace

int contract_blocks(int G, int r, int64_t C, int64_t R_max, bool out, bool grad, int sms) {
  return plan_of(G, r, C, R_max, out, grad, sms).blocks;
}

// A pass takes c column tiles a block only where no other choice d is estimated
// to be faster. With time(c) >= rate(c) tiles + last(c), rate the time a row tile,
// and time(d) < rate(d) tiles + item(d) + last(d) this ends at
//   tiles = (item(d) + last(d) - last(c)) / (rate(c) - rate(d)), rate(c) > rate(d),
// whatever the longest runs are rounded to. So c's parts are no more than those of
// the most rows with as few tiles.
int64_t contract_out_rows(int G, int r, int64_t C, int64_t R_max, bool grad, int sms) {
  const Choices ch(r, C, true, grad, sms);
  const int64_t tiles = row_tiles(G, R_max);
  auto rate = [&](int c) { return double(ch.blocks(c)) * ch.item(c) / sms + ch.parts(c); };
  int64_t found = R_max;
  for (int c = 1; c <= ch.most; c = ch.after(c)) {
    double end = double(tiles);
    for (int d = 1; d <= ch.most; d = ch.after(d)) {
      const double more = rate(c) - rate(d);
      if (more > 1e-9) {
        const double e = (ch.item(d) + ch.last(d) - ch.last(c)) / more + 1.0;  // 1: for the roundings here
        if (e < end) end = e;
      }
    }
    if (end < 1.0) continue;
    const int64_t t = int64_t(end);
    // the most rows of at most t tiles: below G rows each is one
    int64_t rows = R_max;
    if (t < tiles) rows = t < G ? t : kTile * (t - (G + 1) / 2) + kTile - 1;
    if (rows < G && t >= G) rows = G;
    if (rows > R_max) rows = R_max;
    if (ch.blocks(c) * rows > found) found = ch.blocks(c) * rows;
  }
  return found;
}

size_t contract_part_bytes(int r, int64_t C, bool out, int sms) {
  return size_t(part_floats(r, Choices(r, C, out, true, sms).most, sms)) * 4 + size_t(2) * sms * sizeof(Note);
}

cudaError_t launch_contract(const ContractArgs& a, cudaStream_t st, int sms) {
  const Plan q = plan_of(a.G, a.r, a.C, a.R_max, a.out != nullptr, a.grad != nullptr, sms);
  const Pass p = pass_of(a, q, sms);
  CUtensorMap tile{}, edge{}, w{};
  bool ok = true;
  if (!a.row) {  // mapped rows do not come by TMA
    ok = encode_2d(&tile, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.z, uint64_t(a.C), uint64_t(p.rows), uint64_t(a.ld_z) * 2, 64,
                   kTile, CU_TENSOR_MAP_SWIZZLE_128B) &&
         encode_2d(&edge, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.z, uint64_t(a.C), uint64_t(p.rows), uint64_t(a.ld_z) * 2, 64,
                   kEdge, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  if (a.out) {
    // a group's matrix is a plane of its own, so that a box past its edge reads zeros
    const CUtensorMapSwizzle span = q.rp == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
                                    : q.rp == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                 : CU_TENSOR_MAP_SWIZZLE_32B;
    ok = ok && (a.w_t ? encode_planes(&w, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.w, a.r, a.C, a.G, 2, q.rp, kTile, span)
                      : encode_planes(&w, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.w, a.C, a.r, a.G, 2, 64, q.rp,
                                      CU_TENSOR_MAP_SWIZZLE_128B));
  }
  if (!ok) return cudaErrorInvalidValue;
  if (q.rp == 16) return launch_as<16>(a, tile, edge, w, p, st, sms);
  if (q.rp == 32) return launch_as<32>(a, tile, edge, w, p, st, sms);
  return launch_as<64>(a, tile, edge, w, p, st, sms);
}

cudaError_t launch_contract_finish(const ContractArgs* a, const ContractArgs* b, cudaStream_t st, int sms) {
  Finish f[2] = {};
  int ctas = 0, i = 0, most = 0;
  for (const ContractArgs* c : {a, b}) {
    if (!c) continue;
    f[i].p = pass_of(*c, plan_of(c->G, c->r, c->C, c->R_max, c->out != nullptr, true, sms), sms);
    f[i].ctas = c->R_max > 0 ? sms : 0;
    ctas += f[i].ctas;
    if (most < f[i].p.chunks) most = f[i].p.chunks;
    ++i;
  }
  if (!ctas) ctas = 2 * sms;
  const int per = kFinishThreads * kFinishVecs * 4, pieces = (most * kTile * a->r + per - 1) / per;
  return launch_dependent(finish_kernel, dim3(unsigned(ctas), unsigned(pieces)), dim3(kFinishThreads), 0, st, f[0], f[1]);
}

}  // namespace e4b
