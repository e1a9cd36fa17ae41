// Attention of a tree of drafted tokens over the cache on the 5th-generation
// tensor cores: the kernel of nc_tree_attention for trees with many rows (the
// definition is in nc_tree.cu, which also holds the kernel for few rows).
//
// A unit of work is (cache row b, kv head, pair of row tiles).  A row tile is
// 128 / G nodes by the G query heads of the group (row = node * G + head), so
// every K/V tile is read once for all of them.  A unit's key tiles are its
// committed keys from the window's first on, 128 at a time, then one tile of
// the drafted keys.  The last committed tile is moved back to end at the row's
// length (keys that the tile before it has are masked): no position behind the
// length is ever loaded, so what is there cannot reach P V.  Positions before 0
// and nodes past N read as zeros; V of unused nodes is overwritten with zeros
// in shared memory.
//
// The tiles of all units in a row are dealt evenly to one CTA per SM, from the
// lengths on the device: rows of any lengths keep all SMs busy to the end.  A
// unit that one CTA handles whole goes straight to `out`; the pieces of a cut
// one leave (max, sum, O) in the workspace (at most two pieces a CTA) and
// tree_tc_merge_kernel joins them in tile order, so results do not depend on
// timing.
//
// Warp roles: 0 TMA (K and V tiles in two rings of two); 1 MMA issue; 2-5 and
// 6-9 two softmax streams of 128 threads, a row a thread.  With two row tiles,
// stream w takes row tile w and both use every K/V tile; with one, stream w
// takes every other key tile and the two (max, sum, O) are joined from tensor
// memory at the end.  While one stream's softmax runs, the tensor cores work
// for the other: PV_w(i - 1), S_w(i) are issued in turn for w = 0, 1.  Tensor
// memory: S_0, S_1 (128 columns each; P replaces the first half in 16 bits),
// O_0, O_1 (D columns each).  O is rescaled only when the running maximum grows
// by more than 2^8, as in the other attention kernels.
// Every wait is bounded; on timeout the CTA records NC_DEV_TIMEOUT, lets its
// copies and products land, frees its tensor memory and exits.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "nc_half.cuh"
#include "nc_internal.h"
#include "nc_ptx.cuh"

namespace nc {
namespace tree_tc {

constexpr int BM = 128, BKV = 128;
constexpr int NUM_THREADS = 64 + 256;
constexpr int ATOM = 128 * 128;  // bytes of one [128 rows][64 x 16-bit] swizzle tile
constexpr int kMaxB = 1024;      // rows whose tile counts a CTA keeps
constexpr float kRescaleLog2 = 8.0f;

template <int D>
struct Geo {
  static constexpr int KA = D / 64;
  static constexpr int TILE = KA * ATOM;        // one Q, K or V tile
  static constexpr int OFF_K = 2 * TILE;        // after the two Q tiles
  static constexpr int OFF_V = OFF_K + 2 * TILE;
  static constexpr int OFF_BAR = OFF_V + 2 * TILE;
  static constexpr int OFF_X = OFF_BAR + 256;   // (max, sum) of both streams, by piece parity [2][2][128][2]
  static constexpr int OFF_PRE = OFF_X + 2 * 2 * 128 * 2 * 4;
  static constexpr int SMEM_BYTES = OFF_PRE + (kMaxB + 1) * 8;
};

struct Bars {
  uint64_t q_full, q_empty;
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t o_free;
  uint64_t xbar;
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

struct Params {
  const int32_t* lens;
  const uint32_t* mask;
  uint16_t* out;
  float* part;  // [CTAs][2][256][D] then [CTAs][2][256][2]
  int B, N, H, Hkv, T_max, win;
  int G, npt, tiles_r, pairs;  // query heads a kv head, nodes a row tile, row tiles, pairs of them
  float scale_log2;
  uint32_t* dev_status;
  uint64_t limit_ns;
};

struct Row {  // one cache row's committed keys
  int len, lo, n_c;
};

__device__ __forceinline__ Row row_of(const Params& p, int b) {
  Row r;
  r.len = min(max(p.lens[b], 0), p.T_max);
  r.lo = max(0, r.len - p.win + 1);
  r.n_c = (r.len - r.lo + BKV - 1) / BKV;
  return r;
}

// pre[b] = tiles of one unit summed over the rows before b (times the units of
// a row: the linear tile index of row b's first tile); pre[B] = all tiles.
__device__ __forceinline__ void fill_prefix(const Params& p, int64_t* pre) {
  const int upr = p.Hkv * p.pairs;
  for (int b = threadIdx.x; b < p.B; b += blockDim.x) pre[b + 1] = (int64_t)(row_of(p, b).n_c + 1) * upr;
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int64_t run = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      int64_t v = b0 + lane < p.B ? pre[b0 + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
      }
      if (b0 + lane < p.B) pre[b0 + lane + 1] = run + v;
      run += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) pre[0] = 0;
  }
  __syncthreads();
}

struct Seg {
  int b, g, pair;  // the unit
  int t0, n;       // its tiles [t0, t0 + n) ...
  int units_t;     // ... of this many
  bool two;        // two row tiles (streams share the key tiles)
  int64_t u0;      // linear index of the unit's first tile
};

// The piece of work at linear tile x (< end).
__device__ __forceinline__ Seg seg_at(const Params& p, const int64_t* pre, int64_t x, int64_t end) {
  int lo = 0, hi = p.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (pre[mid] <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int upr = p.Hkv * p.pairs;
  Seg s;
  s.b = lo;
  s.units_t = (int)((pre[lo + 1] - pre[lo]) / upr);
  const int64_t rem = x - pre[lo];
  const int u = (int)(rem / s.units_t);
  s.t0 = (int)(rem - (int64_t)u * s.units_t);
  s.pair = u % p.pairs;
  s.g = u / p.pairs;
  s.n = (int)min((int64_t)(s.units_t - s.t0), end - x);
  s.two = 2 * s.pair + 1 < p.tiles_r;
  s.u0 = x - s.t0;
  return s;
}

__device__ __forceinline__ int64_t cta_begin(int64_t total, int c, int n) { return total * c / n; }

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int D, bool F16>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmC,
                   const __grid_constant__ CUtensorMap tmD, const Params p) {
  using G = Geo<D>;
  constexpr uint32_t IDESC_S = idesc_f32acc(BM, BKV, F16);
  constexpr uint32_t IDESC_PV = idesc_f32acc_bmn(BM, D, F16);
  constexpr uint32_t TMEM_COLS = 512;
  constexpr uint32_t O_COL = 2 * BKV;

  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if ((smem_u32(smem_raw) & 1023u) != 0) {  // the swizzled tiles need an aligned base
    if (threadIdx.x == 0 && p.dev_status) atomicOr(p.dev_status, NC_DEV_SMEM_ALIGN);
    return;
  }
  uint8_t* sm = smem_raw;
  Bars* bar = reinterpret_cast<Bars*>(sm + G::OFF_BAR);
  float* xval = reinterpret_cast<float*>(sm + G::OFF_X);
  int64_t* pre = reinterpret_cast<int64_t*>(sm + G::OFF_PRE);
  const uint32_t s_q = smem_u32(sm), s_k = s_q + G::OFF_K, s_v = s_q + G::OFF_V;
  const uint32_t warp = warp_id_sync();
  const uint32_t lane = lane_id();

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bar->q_full), 1);
    mbar_init(smem_u32(&bar->q_empty), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bar->k_full[i]), 1);
      mbar_init(smem_u32(&bar->k_empty[i]), 1);
      mbar_init(smem_u32(&bar->v_full[i]), 1);
      mbar_init(smem_u32(&bar->v_empty[i]), 1);
      mbar_init(smem_u32(&bar->s_full[i]), 1);
      mbar_init(smem_u32(&bar->p_full[i]), 4);
      mbar_init(smem_u32(&bar->o_full[i]), 1);
    }
    mbar_init(smem_u32(&bar->o_free), 8);
    mbar_init(smem_u32(&bar->xbar), 8);
    mbar_init(smem_u32(&bar->drain), 1);
    bar->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmC);
    prefetch_tmap(&tmD);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&bar->tmem_base), TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  fill_prefix(p, pre);  // ends with __syncthreads
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;
  const WaitCtl ctl{&bar->abort_flag, p.dev_status, p.limit_ns};
  const int64_t total = pre[p.B];
  const int64_t x_begin = cta_begin(total, blockIdx.x, gridDim.x), x_end = cta_begin(total, blockIdx.x + 1, gridDim.x);

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer
      uint32_t outstanding = 0, out_phase = 0;  // bits 0,1: K slots; 2: Q; 3,4: V slots
      int gt = 0, n = 0;                        // tiles and pieces done before
      bool ok = true;
      for (int64_t x = x_begin; x < x_end && ok; ++n) {
        const Seg sg = seg_at(p, pre, x, x_end);
        const Row rw = row_of(p, sg.b);
        if (!mbar_wait(smem_u32(&bar->q_empty), (n & 1) ^ 1, ctl)) break;
        const int nq = sg.two ? 2 : 1;
        const uint32_t qbytes = (uint32_t)(p.G * p.npt) * 128u * G::KA;
        mbar_arrive_expect_tx(smem_u32(&bar->q_full), qbytes * nq);
        for (int w = 0; w < nq; ++w)
          for (int a = 0; a < G::KA; ++a)
            tma_load_4d(s_q + w * G::TILE + a * ATOM, &tmQ, a * 64, sg.g * p.G, (2 * sg.pair + w) * p.npt, sg.b,
                        smem_u32(&bar->q_full));
        outstanding |= 4u;
        out_phase = (out_phase & ~4u) | ((uint32_t)(n & 1) << 2);
        // V runs one tile behind K
        for (int j = 0; j <= sg.n; ++j) {
          for (int kv = 0; kv < 2; ++kv) {
            const int jj = j - kv;
            if (jj < 0 || jj >= sg.n) continue;
            const int gi = gt + jj, st = gi & 1;
            const uint32_t use = (uint32_t)(gi >> 1);
            uint64_t* full = kv ? &bar->v_full[st] : &bar->k_full[st];
            if (!mbar_wait(smem_u32(kv ? &bar->v_empty[st] : &bar->k_empty[st]), (use & 1) ^ 1, ctl)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(smem_u32(full), G::TILE);
            const uint32_t dst = (kv ? s_v : s_k) + st * G::TILE;
            const int t = sg.t0 + jj, head = kv * p.Hkv + sg.g;
            const bool draft = t == rw.n_c;
            const int row = draft ? 0 : min(rw.lo + t * BKV, rw.len - BKV);
            for (int a = 0; a < G::KA; ++a)
              tma_load_4d(dst + a * ATOM, draft ? &tmD : &tmC, a * 64, head, row, sg.b, smem_u32(full));
            const int bit = kv * 3 + st;
            outstanding |= 1u << bit;
            out_phase = (out_phase & ~(1u << bit)) | ((use & 1) << bit);
          }
          if (!ok) break;
        }
        gt += sg.n;
        x += sg.n;
      }
      if (!ok || bar->abort_flag) {  // let the copies in flight land
        int zero = 0;
        const WaitCtl dctl{&zero, nullptr, p.limit_ns};
        for (int st = 0; st < 2; ++st) {
          if (outstanding & (1u << st)) mbar_wait(smem_u32(&bar->k_full[st]), (out_phase >> st) & 1u, dctl);
          if (outstanding & (8u << st)) mbar_wait(smem_u32(&bar->v_full[st]), (out_phase >> (3 + st)) & 1u, dctl);
        }
        if (outstanding & 4u) mbar_wait(smem_u32(&bar->q_full), (out_phase >> 2) & 1u, dctl);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---------------- MMA issuer
      int gt = 0, n = 0;
      int gp[2] = {0, 0};  // P V products issued for each stream
      bool ok = true;
      for (int64_t x = x_begin; x < x_end && ok; ++n) {
        const Seg sg = seg_at(p, pre, x, x_end);
        if (!mbar_wait(smem_u32(&bar->q_full), n & 1, ctl)) break;
        tc_fence_after();
        const int steps = sg.two ? sg.n : (sg.n + 1) / 2;
        bool freed = n == 0;
        for (int i = 0; i <= steps && ok; ++i) {
          for (int w = 0; w < 2 && ok; ++w) {
            const int tp = sg.two ? i - 1 : 2 * (i - 1) + w;  // tile of PV_w(i - 1)
            if (i > 0 && tp < sg.n) {
              const int gi = gt + tp, st = gi & 1;
              if (!mbar_wait(smem_u32(&bar->v_full[st]), (uint32_t)(gi >> 1) & 1, ctl) ||
                  !mbar_wait(smem_u32(&bar->p_full[w]), (uint32_t)gp[w] & 1, ctl) ||
                  (!freed && !mbar_wait(smem_u32(&bar->o_free), (uint32_t)(n - 1) & 1, ctl))) {
                ok = false;
                break;
              }
              freed = true;
              ++gp[w];
              tc_fence_after();
              const uint32_t vbase = s_v + st * G::TILE;
#pragma unroll
              for (int k = 0; k < BKV / 16; ++k)
                umma_f16_ts(tmem + O_COL + w * D, tmem + w * BKV + 8 * k, sw128_desc(vbase + k * 2048, ATOM, 1024),
                            IDESC_PV, (i > 1 || k > 0) ? 1u : 0u);
              if (!sg.two || w == 1) umma_commit(smem_u32(&bar->v_empty[st]));
              if (sg.two ? i == steps : tp + 2 >= sg.n) umma_commit(smem_u32(&bar->o_full[w]));
            }
            const int ts = sg.two ? i : 2 * i + w;  // tile of S_w(i)
            if (i < steps && ts < sg.n) {
              const int gi = gt + ts, st = gi & 1;
              if (!mbar_wait(smem_u32(&bar->k_full[st]), (uint32_t)(gi >> 1) & 1, ctl)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint32_t qbase = s_q + (sg.two ? w * G::TILE : 0), kbase = s_k + st * G::TILE;
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = (k >> 2) * ATOM + (k & 3) * 32;
                umma_f16(tmem + w * BKV, sw128_kmajor_desc(qbase + off), sw128_kmajor_desc(kbase + off), IDESC_S,
                         k > 0 ? 1u : 0u);
              }
              umma_commit(smem_u32(&bar->s_full[w]));
              if (!sg.two || w == 1) umma_commit(smem_u32(&bar->k_empty[st]));
              if (ts == sg.n - 1 && (!sg.two || w == 1)) umma_commit(smem_u32(&bar->q_empty));
            }
          }
        }
        gt += sg.n;
        x += sg.n;
      }
      umma_commit(smem_u32(&bar->drain));
      int zero = 0;
      const WaitCtl dctl{&zero, nullptr, p.limit_ns};
      mbar_wait(smem_u32(&bar->drain), 0, dctl);
    }
  } else {
    // ---------------- softmax streams
    const int w = (int)(warp - 2) / 4;  // this warp's stream
    const uint32_t quarter = warp & 3u;
    const int r = (int)(quarter * 32 + lane);  // this thread's row of the tile
    const uint32_t lane_off = (quarter * 32u) << 16;
    const uint32_t scol = tmem + lane_off + w * BKV, ocol = tmem + lane_off + O_COL;
    const float thresh = kRescaleLog2 / p.scale_log2;
    const int W = (p.N + 31) / 32;
    int gt = 0, n = 0, gs = 0, go[2] = {0, 0};
    bool ok = true;
    for (int64_t x = x_begin; x < x_end && ok; ++n) {
      const Seg sg = seg_at(p, pre, x, x_end);
      const Row rw = row_of(p, sg.b);
      const int my_tile = 2 * sg.pair + (sg.two ? w : 0);
      const int node = my_tile * p.npt + r / p.G;
      const bool live_row = r < p.G * p.npt && node < p.N;
      uint32_t see[4] = {0u, 0u, 0u, 0u};  // the node's ancestors; all 0: unused
      int depth = -1;
      if (live_row) {
        const uint32_t* mrow = p.mask + ((int64_t)sg.b * p.N + node) * W;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k < W) {
            see[k] = mrow[k];
            depth += __popc(see[k]);
          }
        bool own = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) own = own || (k == (node >> 5) && ((see[k] >> (node & 31)) & 1u));
        if (!own) {
          depth = -1;
#pragma unroll
          for (int k = 0; k < 4; ++k) see[k] = 0u;
        }
      }
      const bool live_warp = __any_sync(0xffffffffu, depth >= 0);
      const int tmin = depth >= 0 ? rw.len + depth - p.win + 1 : 0;  // first visible position (unused rows: any)
      float m_used = -INFINITY, l = 0.0f;
      bool first = true;
      for (int j = sg.two ? 0 : w; j < sg.n; j += sg.two ? 1 : 2) {
        if (__any_sync(0xffffffffu, !mbar_wait(smem_u32(&bar->s_full[w]), (uint32_t)gs & 1, ctl))) {
          ok = false;
          break;
        }
        ++gs;
        tc_fence_after();
        const int t = sg.t0 + j;
        const bool draft = t == rw.n_c;
        if (draft) {
          // V of unused nodes: zeros
          uint32_t used[4] = {0u, 0u, 0u, 0u};
          bool hole = false;
          for (int k = 0; k < W; ++k) {
            const int i = k * 32 + (int)lane;
            const bool u = i < p.N && ((p.mask[((int64_t)sg.b * p.N + i) * W + k] >> lane) & 1u);
            const uint32_t bal = __ballot_sync(0xffffffffu, u);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (q == k) used[q] = bal;
            hole = hole || __any_sync(0xffffffffu, i < p.N && !u);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) see[k] &= used[k];
          if (hole) {
            const int gi = gt + j, st = gi & 1;
            if (__any_sync(0xffffffffu, !mbar_wait(smem_u32(&bar->v_full[st]), (uint32_t)(gi >> 1) & 1, ctl))) {
              ok = false;
              break;
            }
            bool mine = false;
#pragma unroll
            for (int k = 0; k < 4; ++k) mine = mine || (k == (int)quarter && r < p.N && !((used[k] >> lane) & 1u));
            if (mine) {
              uint4* v = reinterpret_cast<uint4*>(sm + G::OFF_V + st * G::TILE + r * 128);
#pragma unroll
              for (int a = 0; a < G::KA; ++a)
#pragma unroll
                for (int q = 0; q < 8; ++q) v[a * (ATOM / 16) + q] = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
          }
        }
        if (live_warp) {
          // The scores are read twice (maximum, then weights) rather than held: 128
          // of them in registers spill.  P of 64 keys takes 32 columns, all read by then.
          int first_key = 0;  // committed tile: first visible column
          bool masked = draft;
          if (!draft) {
            const int start = min(rw.lo + t * BKV, rw.len - BKV);
            first_key = max(rw.lo + t * BKV, tmin) - start;
            masked = __any_sync(0xffffffffu, first_key > 0);
          }
          auto mask_half = [&](int h, uint32_t (&rr)[2][32]) {
            if (draft) {
#pragma unroll
              for (int e = 0; e < 64; ++e)
                if (!((see[2 * h + (e >> 5)] >> (e & 31)) & 1u)) rr[e >> 5][e & 31] = 0xff800000u;  // -inf
            } else {
#pragma unroll
              for (int e = 0; e < 64; ++e)
                if (h * 64 + e < first_key) rr[e >> 5][e & 31] = 0xff800000u;
            }
          };
          float mx8[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) mx8[e] = -INFINITY;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t rr[2][32];
            tmem_ld_32x32b_x32(scol + h * 64, rr[0]);
            tmem_ld_32x32b_x32(scol + h * 64 + 32, rr[1]);
            tmem_wait_ld();
            if (masked) mask_half(h, rr);
#pragma unroll
            for (int e = 0; e < 64; ++e) mx8[e & 7] = fmaxf(mx8[e & 7], __uint_as_float(rr[e >> 5][e & 31]));
          }
          const float mx = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                                 fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
          const float m_new = fmaxf(m_used, mx);
          bool need = false;
          if (m_used == -INFINITY)
            m_used = m_new;  // O and l are still zero for this row
          else
            need = m_new > m_used + thresh;
          if (!first && __any_sync(0xffffffffu, need)) {
            // the stream's last P V came before this S, so it has landed
            const float alpha = need ? ex2f((m_used - m_new) * p.scale_log2) : 1.0f;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t rr[32];
              tmem_ld_32x32b_x32(ocol + w * D + c * 32, rr);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) rr[e] = __float_as_uint(__uint_as_float(rr[e]) * alpha);
              tmem_st_32x32b_x32(ocol + w * D + c * 32, rr);
            }
            tmem_wait_st();
            if (need) {
              l *= alpha;
              m_used = m_new;
            }
          }
          const float ms = m_used == -INFINITY ? 0.0f : m_used * p.scale_log2;
          float ls8[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t rr[2][32], pk[32];
            tmem_ld_32x32b_x32(scol + h * 64, rr[0]);
            tmem_ld_32x32b_x32(scol + h * 64 + 32, rr[1]);
            tmem_wait_ld();
            if (masked) mask_half(h, rr);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              float q[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                q[e] = ex2f(fmaf(__uint_as_float(rr[c >> 2][(c & 3) * 8 + e]), p.scale_log2, -ms));
                ls8[e] += q[e];
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) pk[4 * c + e] = Half<F16>::pack2(q[2 * e], q[2 * e + 1]);
            }
            tmem_st_32x32b_x32(scol + h * 32, pk);
          }
          l += ((ls8[0] + ls8[1]) + (ls8[2] + ls8[3])) + ((ls8[4] + ls8[5]) + (ls8[6] + ls8[7]));
          tmem_wait_st();
        }
        first = false;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bar->p_full[w]));
      }
      if (!ok) break;
      // ---- the piece's result
      const int cnt[2] = {sg.two ? sg.n : (sg.n + 1) / 2, sg.two ? sg.n : sg.n / 2};
      const bool whole = sg.n == sg.units_t;
      float f0 = 1.0f, f1 = 0.0f;  // weights of the two streams (one row tile: joined)
      // a stream without tiles in the next piece may post for it while the other
      // still reads for this one: two buffers
      float* xv = xval + (n & 1) * 512;
      xv[(w * 128 + r) * 2] = m_used;
      xv[(w * 128 + r) * 2 + 1] = l;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bar->xbar));
      bool landed = mbar_wait(smem_u32(&bar->xbar), (uint32_t)n & 1, ctl);
      for (int v = 0; v < 2; ++v)
        if (cnt[v] > 0) {
          if (!sg.two || v == w) landed = landed && mbar_wait(smem_u32(&bar->o_full[v]), (uint32_t)go[v] & 1, ctl);
          ++go[v];
        }
      if (__any_sync(0xffffffffu, !landed)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (!sg.two) {
        const float ma = xv[r * 2], la = xv[r * 2 + 1], mb = xv[(128 + r) * 2], lb = xv[(128 + r) * 2 + 1];
        m_used = fmaxf(ma, mb);
        f0 = ma == -INFINITY ? 0.0f : ex2f((ma - m_used) * p.scale_log2);
        f1 = mb == -INFINITY ? 0.0f : ex2f((mb - m_used) * p.scale_log2);
        l = la * f0 + lb * f1;
      }
      // one row tile: each stream takes half of the columns of both O
      const int c_lo = sg.two ? 0 : w * (D / 64), c_hi = sg.two ? D / 32 : (w + 1) * (D / 64);
      const float inv = l > 0.0f ? 1.0f / l : 0.0f;
      const int64_t prow = ((int64_t)blockIdx.x * 2 + (x == x_begin ? 0 : 1)) * 256 + (sg.two ? w * 128 : 0) + r;
      if (!whole && c_lo == 0) {
        float* ml = p.part + (int64_t)gridDim.x * 512 * D + prow * 2;
        ml[0] = depth >= 0 ? m_used : -INFINITY;
        ml[1] = depth >= 0 ? l : 0.0f;
      }
#pragma unroll 1
      for (int c = c_lo; c < c_hi; ++c) {
        uint32_t ra[32];
        float v[32];
        if (sg.two || cnt[0] > 0) {
          tmem_ld_32x32b_x32(ocol + (sg.two ? w * D : 0) + c * 32, ra);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = f0 != 0.0f ? __uint_as_float(ra[e]) * f0 : 0.0f;
        }
        if (!sg.two && cnt[1] > 0) {
          tmem_ld_32x32b_x32(ocol + D + c * 32, ra);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = f1 != 0.0f ? fmaf(__uint_as_float(ra[e]), f1, v[e]) : v[e];
        }
        if (!live_row) continue;
        if (whole) {
          uint4* dst = reinterpret_cast<uint4*>(
              p.out + (((int64_t)sg.b * p.N + node) * p.H + sg.g * p.G + r % p.G) * D + c * 32);
          const float k = depth >= 0 ? inv : 0.0f;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint4 pk;
            pk.x = depth >= 0 ? Half<F16>::pack2(v[8 * q] * k, v[8 * q + 1] * k) : 0u;
            pk.y = depth >= 0 ? Half<F16>::pack2(v[8 * q + 2] * k, v[8 * q + 3] * k) : 0u;
            pk.z = depth >= 0 ? Half<F16>::pack2(v[8 * q + 4] * k, v[8 * q + 5] * k) : 0u;
            pk.w = depth >= 0 ? Half<F16>::pack2(v[8 * q + 6] * k, v[8 * q + 7] * k) : 0u;
            dst[q] = pk;
          }
        } else if (depth >= 0) {
          float4* dst = reinterpret_cast<float4*>(p.part + prow * D + c * 32);
#pragma unroll
          for (int q = 0; q < 8; ++q) dst[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bar->o_free));
      gt += sg.n;
      x += sg.n;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, TMEM_COLS);
}

// Joins the pieces of each cut unit.  CTA column c does so for the unit whose
// second piece is CTA c's first; blockIdx.y deals its rows.  One warp a row.
template <int D, bool F16>
__global__ void __launch_bounds__(256) tree_tc_merge_kernel(const Params p, int ctas) {
  extern __shared__ int64_t pre[];
  fill_prefix(p, pre);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x;
  const int64_t total = pre[p.B];
  const int64_t x = cta_begin(total, c, ctas);
  if (x >= cta_begin(total, c + 1, ctas)) return;
  const Seg sg = seg_at(p, pre, x, total);
  if (sg.t0 == 0) return;  // a unit starts here
  // first CTA of the unit: c is its second iff the CTA before c (with work) holds the unit's start
  int c0 = c - 1;
  while (c0 > 0 && cta_begin(total, c0, ctas) == x) --c0;  // CTAs without work
  if (cta_begin(total, c0, ctas) > sg.u0) return;
  const int64_t u_end = sg.u0 + sg.units_t;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int W = (p.N + 31) / 32;
  constexpr int PER = D / 32;
  const int rows = sg.two ? 256 : 128;
  for (int rr = blockIdx.y * 8 + warp; rr < rows; rr += gridDim.y * 8) {
    const int r = rr & 127;
    const int node = (2 * sg.pair + (rr >> 7)) * p.npt + r / p.G;
    if (r >= p.G * p.npt || node >= p.N) continue;
    const bool used = (p.mask[((int64_t)sg.b * p.N + node) * W + (node >> 5)] >> (node & 31)) & 1u;
    float acc[PER], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = 0.0f;
    const float* ml = p.part + (int64_t)ctas * 512 * D;
    for (int k = c0; used && k < ctas; ++k) {
      const int64_t kb = cta_begin(total, k, ctas);
      if (kb >= u_end) break;
      if (cta_begin(total, k + 1, ctas) == kb) continue;
      const int64_t prow = ((int64_t)k * 2 + (kb >= sg.u0 ? 0 : 1)) * 256 + rr;
      const float mk = ml[prow * 2], lk = ml[prow * 2 + 1];
      if (mk == -INFINITY) continue;
      const float mn = fmaxf(m, mk);
      const float a = m == -INFINITY ? 0.0f : ex2f((m - mn) * p.scale_log2), b = ex2f((mk - mn) * p.scale_log2);
      const float* src = p.part + prow * D + lane * PER;
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[e] = acc[e] * a + src[e] * b;
      l = l * a + lk * b;
      m = mn;
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    uint32_t* dst = reinterpret_cast<uint32_t*>(
        p.out + (((int64_t)sg.b * p.N + node) * p.H + sg.g * p.G + r % p.G) * D + lane * PER);
#pragma unroll
    for (int e = 0; e < PER / 2; ++e) dst[e] = Half<F16>::pack2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  }
}

template <int D, bool F16>
nc_status launch_t(const CUtensorMap& mq, const CUtensorMap& mc, const CUtensorMap& md, const Params& p, int ctas,
                   cudaStream_t stream) {
  using G = Geo<D>;
  if (cudaFuncSetAttribute(tree_tc_kernel<D, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM_BYTES) !=
      cudaSuccess)
    return NC_ERR_CUDA;
  tree_tc_kernel<D, F16><<<ctas, NUM_THREADS, G::SMEM_BYTES, stream>>>(mq, mc, md, p);
  if (cudaGetLastError() != cudaSuccess) return NC_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas, 8);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = (size_t)(p.B + 1) * 8;
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;  // its prologue overlaps the products
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_tc_merge_kernel<D, F16>, p, ctas) == cudaSuccess ? NC_OK : NC_ERR_CUDA;
}

}  // namespace tree_tc

bool tree_attention_tc_fits(int B, int N, int H, int Hkv, int window) {
  return B <= tree_tc::kMaxB && H / Hkv <= tree_tc::BM && (window <= 0 || window > tree_tc::BKV);
}

size_t tree_attention_tc_bytes(int D) { return (size_t)device_sm_count() * 512 * (D + 2) * 4; }

nc_status tree_attention_tc_launch(const uint16_t* q, int64_t q_stride, const uint16_t* kv, const uint16_t* cache,
                                   const int32_t* lens, const uint32_t* mask, uint16_t* out, int B, int N, int H,
                                   int Hkv, int D, int T_max, int window, bool f16, void* workspace,
                                   uint32_t* dev_status, cudaStream_t stream) {
  using namespace tree_tc;
  Params p{};
  p.lens = lens;
  p.mask = mask;
  p.out = out;
  p.part = static_cast<float*>(workspace);
  p.B = B;
  p.N = N;
  p.H = H;
  p.Hkv = Hkv;
  p.T_max = T_max;
  p.win = window > 0 ? window : 0x3fffffff;
  p.G = H / Hkv;
  p.npt = BM / p.G;
  p.tiles_r = (N + p.npt - 1) / p.npt;
  p.pairs = (p.tiles_r + 1) / 2;
  p.scale_log2 = 1.4426950408889634f / sqrtf((float)D);
  p.dev_status = dev_status;
  p.limit_ns = kWaitLimitNs;
  CUtensorMap mq, mc, md;
  const uint64_t pos = (uint64_t)2 * Hkv * D * 2;  // bytes of one position
  {
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)H, (uint64_t)N, (uint64_t)B};
    const uint64_t strides[3] = {(uint64_t)D * 2, (uint64_t)q_stride * 2, (uint64_t)N * q_stride * 2};
    const uint32_t box[4] = {64, (uint32_t)p.G, (uint32_t)p.npt, 1};
    if (!encode_tensor_map(&mq, f16, 4, q, dims, strides, box)) return NC_ERR_CUDA;
  }
  const uint32_t box[4] = {64, 1, BKV, 1};
  {
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)2 * Hkv, (uint64_t)T_max, (uint64_t)B};
    const uint64_t strides[3] = {(uint64_t)D * 2, pos, (uint64_t)T_max * pos};
    if (!encode_tensor_map(&mc, f16, 4, cache, dims, strides, box)) return NC_ERR_CUDA;
  }
  {
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)2 * Hkv, (uint64_t)N, (uint64_t)B};
    const uint64_t strides[3] = {(uint64_t)D * 2, pos, (uint64_t)N * pos};
    if (!encode_tensor_map(&md, f16, 4, kv, dims, strides, box)) return NC_ERR_CUDA;
  }
  // no more CTAs than the longest rows have tiles
  const int keys = window > 0 && window - 1 < T_max ? window - 1 : T_max;
  const int64_t most = (int64_t)B * Hkv * p.pairs * ((keys + BKV - 1) / BKV + 1);
  const int ctas = (int)(most < device_sm_count() ? most : device_sm_count());
  if (D == 128)
    return f16 ? launch_t<128, true>(mq, mc, md, p, ctas, stream) : launch_t<128, false>(mq, mc, md, p, ctas, stream);
  return f16 ? launch_t<64, true>(mq, mc, md, p, ctas, stream) : launch_t<64, false>(mq, mc, md, p, ctas, stream);
}

}  // namespace nc
