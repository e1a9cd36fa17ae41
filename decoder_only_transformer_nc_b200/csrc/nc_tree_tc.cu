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
// by more than 2^8, as in the other attention kernels.  P enters P V in 16 bits (the
// row's sum keeps it in fp32), in fp16 times a power of two (see log2_lift).
// Measured, in a graph: 32 rows of 64 nodes, 16 heads on 4, 3000 to 8100 positions
// of 128: 112 us for 385 MB and 93 GFLOP (59 us at the copy rate, 57 us at the tensor
// rate, which no overlap takes below the larger): 3.4 TB/s and 830 TFLOP/s.  The
// tensor pipe is 49 % busy, the exponentials' 50 %; the rest is the chain of one
// stream's tile (S, maximum and weights, P, P V), which two streams cover in part:
// a third would need more tensor memory than 512 columns hold.  8 rows of 32 nodes,
// 900 to 1990 positions: 20 us for 26 MB; some 10 us are start, plan, first loads and
// the merge.
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
constexpr int kMaxB = 1024;      // rows whose tile counts a CTA keeps: 8 KB beside the tiles' 192 (D = 128)
constexpr float kRescaleLog2 = 8.0f;
// In fp16 weights are held times 2^7: with the 2^8 that they may grow they stay under
// 65504, and one is lost below 2^-32 of the largest, not 2^-25: 2^22 keys of those weigh
// no more than half a rounding step of fp16 (at 2^-25 they would weigh an eighth).
// bf16 has fp32's range, for the weights and for V, which may leave no room for a factor.
constexpr float log2_lift(bool f16) { return f16 ? 7.0f : 0.0f; }

template <int D>
struct Geo {
  static constexpr int KA = D / 64;
  static constexpr int TILE = KA * ATOM;        // one Q, K or V tile
  static constexpr int OFF_K = 2 * TILE;        // after the two Q tiles
  static constexpr int OFF_V = OFF_K + 2 * TILE;
  static constexpr int OFF_BAR = OFF_V + 2 * TILE;
  static constexpr int OFF_X = OFF_BAR + 256;   // (max, sum) of both streams, by piece parity [2][2][128][2]
  static constexpr int OFF_SEE = OFF_X + 2 * 2 * 128 * 2 * 4;  // visible drafted keys of every softmax thread
  static constexpr int OFF_PRE = OFF_SEE + 256 * 16;
  static constexpr int SMEM_BYTES = OFF_PRE + (2 * kMaxB + 1) * 4;
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
  float* part;  // [CTAs][2 pieces][2 row tiles]: O [D / 4][128 rows][4], then max and sum [128][2]
  int B, N, H, Hkv, T_max, win;
  int G, npt, tiles_r, pairs;  // query heads a kv head, nodes a row tile, row tiles, pairs of them
  float scale_log2;
  uint32_t* dev_status;
  uint64_t limit_ns;
};

// A unit's first scores, last products and result take about as long as this many
// more tiles; the deal counts them at its end, where they are no work.
constexpr int kUnitCost = 2;

struct Row {  // one cache row's committed keys
  int len, lo, n_c;
};

__device__ __forceinline__ Row row_of(const Params& p, int len) {
  Row r;
  r.len = len;
  r.lo = max(0, len - p.win + 1);
  r.n_c = (r.len - r.lo + BKV - 1) / BKV;
  return r;
}

// The work in shared memory: pre[b] = linear index of row b's first tile (its
// units one after another, kUnitCost tiles of nothing behind each), pre[B] = all
// of them, len[b] = the clamped lengths.  (Fewer than 2^31: tree_attention_tc_fits.)
struct Plan {
  int* pre;
  int* len;
};

__device__ __forceinline__ Plan make_plan(const Params& p, int* mem) {
  const Plan pl{mem, mem + p.B + 1};
  const int upr = p.Hkv * p.pairs;
  for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
    const int len = min(max(p.lens[b], 0), p.T_max);
    pl.len[b] = len;
    pl.pre[b + 1] = (row_of(p, len).n_c + 1 + kUnitCost) * upr;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int run = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      int v = b0 + lane < p.B ? pl.pre[b0 + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
      }
      if (b0 + lane < p.B) pl.pre[b0 + lane + 1] = run + v;
      run += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) pl.pre[0] = 0;
  }
  __syncthreads();
  return pl;
}

// First tile of CTA c: the tiles are dealt as evenly as they go.
struct Deal {
  int q, r;
  __device__ Deal(int total, int ctas) : q(total / ctas), r(total % ctas) {}
  __device__ __forceinline__ int begin(int c) const { return c * q + min(c, r); }
};

struct Seg {
  int b, g, pair;  // the unit
  int t0, n;       // its tiles [t0, t0 + n) (n = 0: none, only the cost behind them) ...
  int units_t;     // ... of this many
  int next;        // linear index behind the piece
  bool two;        // two row tiles (streams share the key tiles)
  int u0;          // linear index of the unit's first tile
};

// The piece of work at linear tile x (< end).
__device__ __forceinline__ Seg seg_at(const Params& p, const int* pre, int x, int end) {
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
  const int span = (pre[lo + 1] - pre[lo]) / upr;
  s.units_t = span - kUnitCost;
  const int rem = x - pre[lo], u = rem / span;
  s.t0 = rem - u * span;
  s.pair = u % p.pairs;
  s.g = u / p.pairs;
  s.next = min(x + span - s.t0, end);
  s.n = max(min(s.units_t - s.t0, end - x), 0);
  s.two = 2 * s.pair + 1 < p.tiles_r;
  s.u0 = x - s.t0;
  return s;
}

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One lane of the (whole) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t got;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(got));
  return got != 0;
}

// A matrix descriptor from its low word: the high word (stride 1024, version,
// swizzle) is the same for all tiles here.  The issuing thread is one of a warp
// that works alone, so the few instructions a descriptor costs count: an MMA of
// 128 x 128 x 16 lasts 64 cycles.
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) {
  constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "n"(hi));
  return r;
}

// 32 lanes x 16 consecutive columns: thread i writes lane (base lane + i).
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32"
      " [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Inverse: thread i gets lane (base lane + i).
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32"
      " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ uint64_t pack_u32x2(uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint64_t pack_f32x2(float a, float b) {
  return pack_u32x2(__float_as_uint(a), __float_as_uint(b));
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
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
  uint4* see_s = reinterpret_cast<uint4*>(sm + G::OFF_SEE);
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
  const Plan pl = make_plan(p, reinterpret_cast<int*>(sm + G::OFF_PRE));  // ends with __syncthreads
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;
  const WaitCtl ctl{&bar->abort_flag, p.dev_status, p.limit_ns};
  const Deal deal(pl.pre[p.B], gridDim.x);
  const int x_begin = deal.begin(blockIdx.x), x_end = deal.begin(blockIdx.x + 1);

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer
      uint32_t outstanding = 0, out_phase = 0;  // bits 0,1: K slots; 2: Q; 3,4: V slots
      int gt = 0, n = 0;                        // tiles and pieces done before
      bool ok = true;
      for (int x = x_begin; x < x_end && ok;) {
        const Seg sg = seg_at(p, pl.pre, x, x_end);
        x = sg.next;
        if (sg.n == 0) continue;
        const Row rw = row_of(p, pl.len[sg.b]);
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
        ++n;
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
    // ---------------- MMA issuer.  The whole warp walks the loop, one lane issues:
    // the operands stay warp-uniform.
    int gt = 0, n = 0;
    int gp[2] = {0, 0};  // P V products issued for each stream
    bool ok = true;
    for (int x = x_begin; x < x_end && ok;) {
      const Seg sg = seg_at(p, pl.pre, x, x_end);
      x = sg.next;
      if (sg.n == 0) continue;
      const int sn = __shfl_sync(0xffffffffu, sg.n, 0);
      const bool two = __shfl_sync(0xffffffffu, (int)sg.two, 0) != 0;
      if (!mbar_wait(smem_u32(&bar->q_full), n & 1, ctl)) break;
      tc_fence_after();
      const int steps = two ? sn : (sn + 1) / 2;
      bool freed = n == 0;
      for (int i = 0; i <= steps && ok; ++i) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int tp = two ? i - 1 : 2 * (i - 1) + w;  // tile of PV_w(i - 1)
          if (ok && i > 0 && tp < sn) {
            const int gi = gt + tp, st = gi & 1;
            ok = mbar_wait(smem_u32(&bar->v_full[st]), (uint32_t)(gi >> 1) & 1, ctl) &&
                 mbar_wait(smem_u32(&bar->p_full[w]), (uint32_t)gp[w] & 1, ctl) &&
                 (freed || mbar_wait(smem_u32(&bar->o_free), (uint32_t)(n - 1) & 1, ctl));
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            freed = true;
            ++gp[w];
            tc_fence_after();
            const uint32_t vlo = (uint32_t)sw128_desc(s_v + st * G::TILE, ATOM, 1024);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < BKV / 16; ++k)
                umma_f16_ts(tmem + O_COL + w * D, tmem + w * BKV + 8 * k, desc_of(vlo + k * (2048 >> 4)), IDESC_PV,
                            (i > 1 || k > 0) ? 1u : 0u);
              if (!two || w == 1) umma_commit(smem_u32(&bar->v_empty[st]));
              if (two ? i == steps : tp + 2 >= sn) umma_commit(smem_u32(&bar->o_full[w]));
            }
            __syncwarp();
          }
          const int ts = two ? i : 2 * i + w;  // tile of S_w(i)
          if (ok && i < steps && ts < sn) {
            const int gi = gt + ts, st = gi & 1;
            ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar->k_full[st]), (uint32_t)(gi >> 1) & 1, ctl));
            if (!ok) break;
            tc_fence_after();
            const uint32_t qlo = (uint32_t)sw128_kmajor_desc(s_q + (two ? w * G::TILE : 0));
            const uint32_t klo = (uint32_t)sw128_kmajor_desc(s_k + st * G::TILE);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = ((k >> 2) * ATOM + (k & 3) * 32) >> 4;
                umma_f16(tmem + w * BKV, desc_of(qlo + off), desc_of(klo + off), IDESC_S, k > 0 ? 1u : 0u);
              }
              umma_commit(smem_u32(&bar->s_full[w]));
              if (!two || w == 1) umma_commit(smem_u32(&bar->k_empty[st]));
              if (ts == sn - 1 && (!two || w == 1)) umma_commit(smem_u32(&bar->q_empty));
            }
            __syncwarp();
          }
        }
      }
      gt += sn;
      ++n;
    }
    if (elect_one()) umma_commit(smem_u32(&bar->drain));
    __syncwarp();
    int zero = 0;
    const WaitCtl dctl{&zero, nullptr, p.limit_ns};
    mbar_wait(smem_u32(&bar->drain), 0, dctl);
  } else {
    // ---------------- softmax streams
    const int w = (int)(warp - 2) / 4;  // this warp's stream
    const uint32_t quarter = warp & 3u;
    const int r = (int)(quarter * 32 + lane);  // this thread's row of the tile
    const uint32_t lane_off = (quarter * 32u) << 16;
    const uint32_t scol = tmem + lane_off + w * BKV, ocol = tmem + lane_off + O_COL;
    const float lift = log2_lift(F16) / p.scale_log2, thresh = kRescaleLog2 / p.scale_log2 + lift;
    const int W = (p.N + 31) / 32;
    int gt = 0, n = 0, gs = 0, go[2] = {0, 0};
    bool ok = true;
    for (int x = x_begin; x < x_end && ok;) {
      const Seg sg = seg_at(p, pl.pre, x, x_end);
      const bool first_piece = x == x_begin;
      x = sg.next;
      if (sg.n == 0) continue;
      const Row rw = row_of(p, pl.len[sg.b]);
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
      // For the drafted tile: whether the row has unused nodes, and this thread's visible
      // keys (in shared memory: registers are short in the loop).
      bool hole = false;
      if (sg.t0 + sg.n > rw.n_c) {
        uint32_t used[4];
        uint32_t word[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k * 32 + (int)lane < p.N) word[k] = p.mask[((int64_t)sg.b * p.N + k * 32 + (int)lane) * W + k];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          used[k] = __ballot_sync(0xffffffffu, (word[k] >> lane) & 1u);
          const int left = p.N - 32 * k;
          const uint32_t nodes = left <= 0 ? 0u : left >= 32 ? 0xffffffffu : (1u << left) - 1u;
          hole = hole || (used[k] & nodes) != nodes;
          see[k] &= used[k];
        }
        see_s[(w * 128 + r)] = make_uint4(see[0], see[1], see[2], see[3]);
      }
      const bool live_warp = __any_sync(0xffffffffu, depth >= 0);
      const int tmin = depth >= 0 ? rw.len + depth - p.win + 1 : 0;  // first visible position (unused rows: any)
      float m_used = -INFINITY, l = 0.0f;  // m_used: a maximum so far, less lift
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
          if (hole) {
            const int gi = gt + j, st = gi & 1;
            if (__any_sync(0xffffffffu, !mbar_wait(smem_u32(&bar->v_full[st]), (uint32_t)(gi >> 1) & 1, ctl))) {
              ok = false;
              break;
            }
            bool mine = false;
#pragma unroll
            for (int k = 0; k < 4; ++k) mine = mine || (k == (int)quarter && r < p.N && !((p.mask[((int64_t)sg.b * p.N + r) * W + k] >> lane) & 1u));
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
          // A tile with hidden keys gets -inf over their scores in tensor memory first,
          // so the common path below carries no masks.
          int first_key = 0;  // committed tile: first visible column
          if (!draft) {
            const int start = min(rw.lo + t * BKV, rw.len - BKV);
            first_key = max(rw.lo + t * BKV, tmin) - start;
          }
          if (__any_sync(0xffffffffu, draft || first_key > 0)) {
#pragma unroll 1
            for (int c = 0; c < BKV / 32; ++c) {
              const int fk = first_key - c * 32;
              const uint32_t vis = draft ? reinterpret_cast<const uint32_t*>(see_s + w * 128 + r)[c]
                                         : (fk <= 0 ? 0xffffffffu : fk >= 32 ? 0u : 0xffffffffu << fk);
              uint32_t rr[32];
              tmem_ld_32x32b_x32(scol + c * 32, rr);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((vis >> e) & 1u)) rr[e] = 0xff800000u;  // -inf
              tmem_st_32x32b_x32(scol + c * 32, rr);
            }
            tmem_wait_st();
          }
          // The weights against the maximum so far, the tile's own maximum on the side;
          // P stays in registers (64) until that is known to be at most 2^8 above, else
          // O is rescaled and the weights are made again (the first tile of a piece
          // always: its first maximum).  Scores 16 at a time, the next on their way.
          uint32_t pk[BKV / 2];
          float mx = -INFINITY, lt = 0.0f;
          auto weigh = [&](float m) {
            const float ms = m == -INFINITY ? 0.0f : m * p.scale_log2;
            // two at a time (packed fp32 multiply-adds and sums)
            const uint64_t sc2 = pack_f32x2(p.scale_log2, p.scale_log2), ms2 = pack_f32x2(-ms, -ms);
            uint64_t ls4[4] = {0ull, 0ull, 0ull, 0ull};  // pairs of zeros
            float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            uint32_t sr[2][16];
            tmem_ld_32x32b_x16(scol, sr[0]);
#pragma unroll
            for (int c = 0; c < BKV / 16; ++c) {
              tmem_wait_ld();
              if (c + 1 < BKV / 16) tmem_ld_32x32b_x16(scol + (c + 1) * 16, sr[(c + 1) & 1]);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const uint32_t s0 = sr[c & 1][2 * e], s1 = sr[c & 1][2 * e + 1];
                mx4[e & 3] = fmaxf(fmaxf(mx4[e & 3], __uint_as_float(s0)), __uint_as_float(s1));
                float a, b;
                unpack_f32x2(fma_f32x2(pack_u32x2(s0, s1), sc2, ms2), a, b);
                a = ex2f(a);
                b = ex2f(b);
                ls4[e & 3] = add_f32x2(ls4[e & 3], pack_f32x2(a, b));
                pk[c * 8 + e] = Half<F16>::pack2(a, b);
              }
            }
            mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
            float a, b;
            unpack_f32x2(add_f32x2(add_f32x2(ls4[0], ls4[1]), add_f32x2(ls4[2], ls4[3])), a, b);
            lt = a + b;
          };
          if (first) {  // only the maximum is wanted of this pass
            float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
            for (int c = 0; c < BKV / 32; ++c) {
              uint32_t rr[32];
              tmem_ld_32x32b_x32(scol + c * 32, rr);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) mx4[e & 3] = fmaxf(mx4[e & 3], __uint_as_float(rr[e]));
            }
            m_used = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) - lift;
          }
#pragma unroll 1
          for (;;) {
            weigh(m_used);
            // a row that has seen nothing yet (O and l are zero) takes any maximum
            const bool need = mx > m_used + thresh || (m_used == -INFINITY && mx != -INFINITY);
            if (!__any_sync(0xffffffffu, need)) break;
            // the stream's last P V came before this S, so it has landed
            const float alpha = need && m_used != -INFINITY ? ex2f((m_used - (mx - lift)) * p.scale_log2) : 1.0f;
            if (!first) {
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
            }
            l *= alpha;
            if (need) m_used = mx - lift;
          }
          l += lt;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t q[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) q[e] = pk[c * 16 + e];
            tmem_st_32x32b_x16(scol + c * 16, q);
          }
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
      // pieces: four columns of a warp's 32 rows are neighbours, so its stores are whole lines
      float* part = p.part + (((int64_t)blockIdx.x * 2 + (first_piece ? 0 : 1)) * 2 + (sg.two ? w : 0)) * ((D + 2) * 128);
      if (!whole && c_lo == 0)
        *reinterpret_cast<float2*>(part + D * 128 + r * 2) =
            make_float2(depth >= 0 ? m_used : -INFINITY, depth >= 0 ? l : 0.0f);
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
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *reinterpret_cast<float4*>(part + ((c * 8 + q) * 128 + r) * 4) =
                make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bar->o_free));
      gt += sg.n;
      ++n;
    }
  }

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the merge's plan may be made now
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, TMEM_COLS);
}

// Joins the pieces of each cut unit.  CTA column c does so for the unit whose
// second piece is CTA c's first; blockIdx.y deals its rows and columns: a warp
// takes 32 rows (a row a lane, as the pieces are stored) and 16 columns.
template <int D, bool F16>
__global__ void __launch_bounds__(256) tree_tc_merge_kernel(const Params p, int ctas) {
  extern __shared__ int mem[];
  const Plan pl = make_plan(p, mem);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x;
  const int total = pl.pre[p.B];
  const Deal deal(total, ctas);
  const int x = deal.begin(c);
  if (x >= deal.begin(c + 1)) return;
  const Seg sg = seg_at(p, pl.pre, x, total);
  // Every CTA has a tile or more once c has one (the first ones get the extra
  // tiles), so the piece before this one is CTA c - 1's.
  if (sg.t0 == 0 || sg.n == 0 || deal.begin(c - 1) > sg.u0) return;
  const int u_end = sg.u0 + sg.units_t;
  const int lane = threadIdx.x & 31;
  int k_end = c + 1;  // past the last piece's CTA
  while (k_end < ctas && deal.begin(k_end) < u_end && deal.begin(k_end + 1) > deal.begin(k_end)) ++k_end;
  constexpr int CG = D / 16;  // column groups
  const int jobs = (sg.two ? 8 : 4) * CG;
  for (int job = blockIdx.y * 8 + (threadIdx.x >> 5); job < jobs; job += gridDim.y * 8) {
    const int rg = job / CG, cg = job - rg * CG;
    const int r = (rg & 3) * 32 + lane;
    const int node = (2 * sg.pair + (rg >> 2)) * p.npt + r / p.G;
    const bool in = r < p.G * p.npt && node < p.N;
    // piece k of the unit: CTA k's first piece unless the unit starts inside CTA k's work
    auto piece = [&](int k) {
      return p.part + (((int64_t)k * 2 + (deal.begin(k) >= sg.u0 ? 0 : 1)) * 2 + (rg >> 2)) * ((D + 2) * 128);
    };
    float acc[16], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.0f;
    for (int k0 = c - 1; k0 < k_end; k0 += 3) {  // three pieces' loads in flight
      float4 v[3][4];
      float2 ml[3];
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        ml[i] = make_float2(-INFINITY, 0.0f);
        if (k0 + i < k_end) {
          const float* src = piece(k0 + i);
          ml[i] = *reinterpret_cast<const float2*>(src + D * 128 + r * 2);
#pragma unroll
          for (int q = 0; q < 4; ++q) v[i][q] = *reinterpret_cast<const float4*>(src + ((cg * 4 + q) * 128 + r) * 4);
        }
      }
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        // rows of a piece that saw nothing (and rows that are no node's) hold anything
        if (in && ml[i].x != -INFINITY) {
          const float mn = fmaxf(m, ml[i].x);
          const float a = m == -INFINITY ? 0.0f : ex2f((m - mn) * p.scale_log2), b = ex2f((ml[i].x - mn) * p.scale_log2);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            acc[4 * q] = fmaf(acc[4 * q], a, v[i][q].x * b);
            acc[4 * q + 1] = fmaf(acc[4 * q + 1], a, v[i][q].y * b);
            acc[4 * q + 2] = fmaf(acc[4 * q + 2], a, v[i][q].z * b);
            acc[4 * q + 3] = fmaf(acc[4 * q + 3], a, v[i][q].w * b);
          }
          l = fmaf(l, a, ml[i].y * b);
          m = mn;
        }
      }
    }
    if (!in) continue;
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    uint4* dst = reinterpret_cast<uint4*>(
        p.out + (((int64_t)sg.b * p.N + node) * p.H + sg.g * p.G + r % p.G) * D + cg * 16);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      uint4 pk;
      pk.x = Half<F16>::pack2(acc[8 * q] * inv, acc[8 * q + 1] * inv);
      pk.y = Half<F16>::pack2(acc[8 * q + 2] * inv, acc[8 * q + 3] * inv);
      pk.z = Half<F16>::pack2(acc[8 * q + 4] * inv, acc[8 * q + 5] * inv);
      pk.w = Half<F16>::pack2(acc[8 * q + 6] * inv, acc[8 * q + 7] * inv);
      dst[q] = pk;
    }
  }
}

template <int D, bool F16>
nc_status launch_t(const CUtensorMap& mq, const CUtensorMap& mc, const CUtensorMap& md, const Params& p, int ctas,
                   cudaStream_t stream) {
  using G = Geo<D>;
  static bool attr_done[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !attr_done[dev]) {
    if (cudaFuncSetAttribute(tree_tc_kernel<D, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM_BYTES) !=
        cudaSuccess)
      return NC_ERR_CUDA;
    if (dev < 64) attr_done[dev] = true;
  }
  tree_tc_kernel<D, F16><<<ctas, NUM_THREADS, G::SMEM_BYTES, stream>>>(mq, mc, md, p);
  if (cudaGetLastError() != cudaSuccess) return NC_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas, 8);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = (size_t)(2 * p.B + 1) * 4;
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;  // its prologue overlaps the products
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_tc_merge_kernel<D, F16>, p, ctas) == cudaSuccess ? NC_OK : NC_ERR_CUDA;
}

}  // namespace tree_tc

// At most 2^15 units of at most 2^22 / 128 + 3 tiles: linear tile indices fit 32 bits.
bool tree_attention_tc_fits(int B, int N, int H, int Hkv, int window) {
  const int G = H / Hkv;
  if (G > tree_tc::BM) return false;
  const int tiles_r = (N + tree_tc::BM / G - 1) / (tree_tc::BM / G);
  return B <= tree_tc::kMaxB && (int64_t)B * Hkv * ((tiles_r + 1) / 2) <= (1 << 15) && (window <= 0 || window > tree_tc::BKV);
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
  const int64_t most = (int64_t)B * Hkv * p.pairs * ((keys + BKV - 1) / BKV + 1);  // (without kUnitCost)
  const int ctas = (int)(most < device_sm_count() ? most : device_sm_count());
  if (D == 128)
    return f16 ? launch_t<128, true>(mq, mc, md, p, ctas, stream) : launch_t<128, false>(mq, mc, md, p, ctas, stream);
  return f16 ? launch_t<64, true>(mq, mc, md, p, ctas, stream) : launch_t<64, false>(mq, mc, md, p, ctas, stream);
}

}  // namespace nc
