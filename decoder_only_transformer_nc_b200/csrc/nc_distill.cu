// Distillation from a teacher's K largest logits a row: the loss and the
// gradient with respect to the student's raw logits.
//
//   l = cap tanh(z / cap) (cap = 0: l = z), p = softmax(l / tau) over V,
//   q = softmax(t / tau) over the row's teacher entries,
//   loss = tau^2 sum_k q_k (log q_k - log p_{i_k}),
//   dz_i = w tau (p_i - sum_{k: i_k = i} q_k) (1 - (l_i / cap)^2).
//
// An entry with index -1 is unused (rows with fewer teacher entries than K); an
// index outside [-1, V) is flagged and unused.  A row with no entry has loss 0
// and gradient 0.  Softmax statistics and sums are fp32 in a fixed order; exponentials and
// reciprocals are the hardware's (2^-22 relative) and the scale cap log2(e) / tau is rounded
// once, which leaves the loss within some 5e-7 of the 64-bit one (fp32 with exp: 1e-7).
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "nc_half.cuh"
#include "nc_internal.h"
#include "nc_ptx.cuh"

namespace nc {
namespace {

constexpr int kThreads = 256;           // that hold the row
constexpr int kBlock = kThreads + 32;  // and a warp for the teacher's entries
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// The maximum over the warp (NaN gives way).
__device__ __forceinline__ float warp_max_redux(float v) {
  float m;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}

// Pairs of fp32: the kernel is bound by the instructions it issues.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t pair(const float2& v) { return *reinterpret_cast<const uint64_t*>(&v); }
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh(u).  Up to |u| = 1.5, where nearly all logits are under their cap, the
// continued fraction u / (1 + s / (3 + s / (5 + s / (7 + s / (9 + s / 11))))),
// s = u^2, as a quotient of polynomials: within 3e-8 there, one reciprocal.
// Beyond, 1 - 2 / (e^2u + 1), whose absolute error is that of its 1.
constexpr float kNear = 1.5f;
__device__ __forceinline__ float tanh_far(float u) {
  return copysignf(fmaf(-2.0f, rcp(1.0f + ex2(2.0f * kLog2e * fabsf(u))), 1.0f), u);
}

// tanh(z / cap) with the quotient's coefficients in terms of z.
struct Tanh {
  float inv_cap, near, a1, a2, b1, b2, b3;
  float2 pi, pa1, pa2, pb1, pb2, pb3;  // each twice, for pairs
  explicit Tanh(float cap) {
    inv_cap = 1.0f / cap;
    near = kNear * cap;
    const float c2 = inv_cap * inv_cap;
    a1 = 1260.0f / 10395.0f * (c2 * inv_cap);
    a2 = 21.0f / 10395.0f * (c2 * c2 * inv_cap);
    b1 = 4725.0f / 10395.0f * c2;
    b2 = 210.0f / 10395.0f * (c2 * c2);
    b3 = 1.0f / 10395.0f * (c2 * c2 * c2);
    pi = make_float2(inv_cap, inv_cap);
    pa1 = make_float2(a1, a1);
    pa2 = make_float2(a2, a2);
    pb1 = make_float2(b1, b1);
    pb2 = make_float2(b2, b2);
    pb3 = make_float2(b3, b3);
  }
  __device__ __forceinline__ float close(float z) const {
    const float s = z * z;
    const float a = fmaf(fmaf(a2, s, a1), s, inv_cap);
    const float b = fmaf(fmaf(fmaf(b3, s, b2), s, b1), s, 1.0f);
    return z * a * rcp(b);
  }
  __device__ __forceinline__ float operator()(float z) const {
    return fabsf(z) <= near ? close(z) : tanh_far(z * inv_cap);
  }
  __device__ __forceinline__ uint64_t close2(uint64_t z) const {
    const uint64_t s = mul2(z, z);
    const uint64_t a = fma2(fma2(pair(pa2), s, pair(pa1)), s, pair(pi));
    const float2 b = unpair(fma2(fma2(fma2(pair(pb3), s, pair(pb2)), s, pair(pb1)), s, pair(1.0f, 1.0f)));
    return mul2(mul2(z, a), pair(rcp(b.x), rcp(b.y)));
  }
  // four at a time; the far form only where some lane of the warp needs it
  __device__ __forceinline__ float4 operator()(const float4& z) const {
    const float2 t01 = unpair(close2(pair(z.x, z.y))), t23 = unpair(close2(pair(z.z, z.w)));
    float4 t = make_float4(t01.x, t01.y, t23.x, t23.y);
    const float m = fmaxf(fmaxf(fabsf(z.x), fabsf(z.y)), fmaxf(fabsf(z.z), fabsf(z.w)));
    if (!(m <= near)) {
      if (!(fabsf(z.x) <= near)) t.x = tanh_far(z.x * inv_cap);
      if (!(fabsf(z.y) <= near)) t.y = tanh_far(z.y * inv_cap);
      if (!(fabsf(z.z) <= near)) t.z = tanh_far(z.z * inv_cap);
      if (!(fabsf(z.w) <= near)) t.w = tanh_far(z.w * inv_cap);
    }
    return t;
  }
};

struct DistillParams {
  const float* z;         // [M][V]
  const int32_t* idx;     // [M][K]
  const float* teacher;   // [M][K]
  const float* weight;    // [M] or null
  float* loss;            // [M]
  void* dz;               // [M][V] or null
  int V, K;
  float tau, inv_tau, kx;  // kx: x (log2) of t or z, that is cap log2(e) / tau or log2(e) / tau
  Tanh tanh_of;            // on the host, so its coefficients are constant operands, not registers
  uint32_t* status;
};

// (maximum, sum) of the parts of a softmax that the first n <= 8 lanes hold (log2
// domain), in a fixed tree, in every one of the first 8 lanes.
__device__ __forceinline__ float2 join8(float2 v) {
  const float m = warp_max_redux(v.x);
  float s = m == -INFINITY ? 0.0f : v.y * ex2(v.x - m);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return make_float2(m, s);
}

// A row is dealt over the CTAs of a cluster (one CTA up to 8192 logits), every
// thread holding its REGS groups of four logits (in registers, with a gradient half
// of them in shared memory) from the one read to the gradient's store, so z and dz
// cross the memory bus once.  Four or five CTAs of 256 threads share an SM, at
// different points of different rows: one loads while another computes or stores.
// The threads' (maximum, sum) are joined over the block and, through distributed
// shared memory, over the cluster, in a fixed order.
//
// Measured, in a graph: 4096 rows of 32768 logits, K = 64, bf16 gradient: 176 us for
// 807 MB, which take 123 us at the copy rate (4.6 TB/s, 70 %).  The three special
// functions a logit (two exponentials and the quotient of tanh) take 89 us on their
// own, and the issue slots are 63 % busy.  2048 rows without a gradient: 60 us for
// 269 MB (41 us).  Fetching the next rows into L2 ahead of time changed nothing.
//
// The teacher's entries are the business of a warp of its own: with K = 64 beside 8192
// logits, eight warps repeating it took as many instructions as the row.  That warp
// takes longer than the row from K = 128 or so (4096 rows without a gradient: 117 us
// at K = 64, 330 at 512).
// REGS = 0: rows of more than 65536 logits, one CTA each, read again from L2 for each
// use.  1024 rows of 131072, K = 64: 377 us with a bf16 gradient (floor 123 at the copy
// rate), 173 without (82); 8 rows of them take 151 us, of 65536 logits 7 us.
// Groups of four start at 16-byte boundaries of z's row; the row's ends and a dz that
// is not aligned alike go by single elements.  2048 rows of 32767 logits without a
// gradient take 86 us (106 while every group was tested for the ends), those of 32768
// 61: the odd ones start anywhere, which takes a fifth CTA a row.
// DZ: 0 none, 1 fp32, 2 bf16, 3 fp16
struct Shared {
  float2 part[8], part_w[kThreads / 32];
  uint64_t bar;  // the cluster's parts have arrived
};

// bar.sync / bar.arrive on a barrier of the CTA that not all its threads take part in
__device__ __forceinline__ void named_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ void named_arrive(int id, int n) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// Built-in indices that are read anew: what depends on them is computed where it is
// used, not kept in registers (or spilled) from the row's loads to the gradient's
// stores.
__device__ __forceinline__ uint32_t fresh_tid() {
  uint32_t v;
  asm volatile("mov.u32 %0, %%tid.x;" : "=r"(v));
  return v;
}
__device__ __forceinline__ uint32_t fresh_row() {
  uint32_t v;
  asm volatile("mov.u32 %0, %%ctaid.y;" : "=r"(v));
  return v;
}
__device__ __forceinline__ uint32_t fresh_rank() {
  uint32_t v;
  asm volatile("mov.u32 %0, %%ctaid.x;" : "=r"(v));
  return v;
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// Of a thread's groups, how many are in registers, and the CTAs that share an SM.
// With a gradient, half of the eight are in shared memory: with all of them in registers four
// CTAs fit an SM, and spill (225 us for 4096 rows of 32768 logits, K = 64, bf16 gradient;
// so 201).  Without, the row's values are needed once less (59 us for 2048 rows, 65).
constexpr int held(int dz, int regs) { return dz != 0 && regs == 8 ? 4 : regs; }
constexpr int resident(int dz, int regs) { return regs != 8 ? 1 : dz != 0 ? 5 : 4; }

constexpr int kTwice = 1 << 30;  // marks an index of the table (below 2^24)

// FULL: every thread has REGS whole groups (no test of a group's place).
template <int DZ, bool CAP, int REGS, bool FULL>
__device__ __forceinline__ void distill_part(const DistillParams& p, int slice, int slots, float* mem, Shared& sh) {
  // mem: the groups not in registers; the teacher's [K] logits, [K] z at the entry,
  // [K] indices; [K] the entries of this CTA's positions, [K] their gradients; [slots]
  constexpr int HELD = held(DZ, REGS);
  float4* own = reinterpret_cast<float4*>(mem) + threadIdx.x;  // this thread's, kThreads apart
  float* q_s = mem + (REGS - HELD) * kThreads * 4;
  float* z_s = q_s + p.K;
  int32_t* i_s = reinterpret_cast<int32_t*>(z_s + p.K);
  int32_t* list = i_s + p.K;
  float* g_s = reinterpret_cast<float*>(i_s + 2 * p.K);
  int32_t* table = i_s + 3 * p.K;
  const int64_t row = blockIdx.y;
  const int rank = blockIdx.x, CS = gridDim.x;  // the cluster spans the grid's x
  const int V = p.V, K = p.K, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float* zr = p.z + row * V;
  const int off = (int)((reinterpret_cast<uintptr_t>(zr) >> 2) & 3);  // logit 0 is position off
  const float* z = zr - off;
  const int end = off + V;
  const int s0 = rank * slice, s1 = min(end, s0 + slice);  // this CTA's positions
  const Tanh& tanh_of = p.tanh_of;
  const float kx = p.kx;
  auto load = [&](int j) { return __ldcs(reinterpret_cast<const float4*>(z + j)); };
  constexpr int STEP = kThreads * 4;
  const int j_first = s0 + tid * 4;
  // Whole groups of four from position `lo` on; this thread has the first nr (0 or
  // less: none) but for one before lo.  What is left of the row's ends, up to three
  // logits each, is dealt to the first six threads, one each (`edge` at je).
  const int lo = off > 0 ? 4 : 0;
  const int nr = warp == kThreads / 32 ? 0 : (min(s0 + slice, end & ~3) - j_first + STEP - 1) / STEP;
  int je = -1;
  float edge = -INFINITY;
  if (!FULL && tid < 6) {
    const int tail = end & ~3;
    if (tid < 3) {
      if (s0 == 0 && off > 0 && off + tid < min(4, end)) je = off + tid;
    } else if (tail >= lo && tail >= s0 && tail < s0 + slice && tail + tid - 3 < end) {
      je = tail + tid - 3;
    }
    if (je >= 0) edge = z[je];
  }
  float4 keep[HELD > 0 ? HELD : 1];
  if constexpr (REGS > 0) {
#pragma unroll
    for (int r = HELD; r < REGS; ++r)
      if (FULL ? warp < kThreads / 32 : r < nr) cp_async16(own + (r - HELD) * kThreads, z + j_first + r * STEP);
#pragma unroll
    for (int r = 0; r < HELD; ++r)
      if (FULL ? warp < kThreads / 32 : r < nr && (r > 0 || j_first >= lo)) keep[r] = load(j_first + r * STEP);
  }
  // f(position, four values); WRITE: f changes them
  auto each = [&](int j_first, auto write, auto f) {
    if constexpr (REGS > 0) {
      constexpr bool WRITE = decltype(write)::value;
#pragma unroll
      for (int r = 0; r < HELD; ++r)
        if (FULL || (r < nr && (r > 0 || j_first >= lo))) f(j_first + r * STEP, keep[r]);
      if (WRITE && REGS > HELD) asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
      for (int r = HELD; r < REGS; ++r)
        if (FULL || r < nr) {
          float4 v = own[(r - HELD) * kThreads];
          f(j_first + r * STEP, v);
          if (WRITE) own[(r - HELD) * kThreads] = v;
        }
    } else {
#pragma unroll 1
      for (int j = j_first, r = 0; r < nr; ++r, j += STEP) {
        if (j < lo) continue;
        float4 v = load(j);
        f(j, v);
      }
    }
  };

  // the teacher's softmax, while the row is on its way
  const bool helper = warp == kThreads / 32;
  bool t_any = true;  // the helper's
  float t_lse = 0.0f;
  int n_here = 0;  // entries of this CTA's positions
  if (helper) {
    float tm = -INFINITY;
    for (int k0 = 0; k0 < K; k0 += 32) {
      const int k = k0 + lane;
      int i = -1;
      if (k < K) {
        i = p.idx[row * K + k];
        if (i < -1 || i >= V) {
          if (p.status) atomicOr(p.status, NC_DEV_TARGET_RANGE);
          i = -1;
        }
        const float t = i < 0 ? -INFINITY : p.teacher[row * K + k] * p.inv_tau;
        z_s[k] = i < 0 ? 0.0f : zr[i];
        i_s[k] = i;
        q_s[k] = t;
        tm = fmaxf(tm, t);
      }
      if (DZ != 0) {
        const bool here = i >= 0 && off + i >= s0 && off + i < s1;
        const uint32_t bal = __ballot_sync(0xffffffffu, here);
        if (here) list[n_here + __popc(bal & ((1u << lane) - 1u))] = k;
        n_here += __popc(bal);
      }
    }
    tm = warp_max_redux(tm);
    const bool any = tm != -INFINITY;
    float ts = 0.0f;
    for (int k = lane; k < K; k += 32) ts += any ? expf(q_s[k] - tm) : 0.0f;
    ts = warp_sum(ts);
    t_any = any;
    t_lse = any ? tm + logf(ts) : 0.0f;
  }

  // the student's softmax: with registers, t takes the place of z
  float2 ms = make_float2(-INFINITY, 0.0f);
  const uint64_t kx2 = pair(kx, kx);
  auto exps = [&](const float4& v, uint64_t minus_m, uint64_t& e01, uint64_t& e23) {
    const float2 a = unpair(fma2(pair(v.x, v.y), kx2, minus_m)), b = unpair(fma2(pair(v.z, v.w), kx2, minus_m));
    e01 = pair(ex2(a.x), ex2(a.y));
    e23 = pair(ex2(b.x), ex2(b.y));
  };
  if (!helper) {
    each(j_first, std::true_type{}, [&](int, float4& v) {
      if (CAP) v = tanh_of(v);
      const float m = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
      if (REGS > 0) {
        ms.x = fmaxf(ms.x, m);
      } else {
        const float mn = fmaxf(ms.x, m * kx);
        if (mn != -INFINITY) {
          uint64_t e01, e23;
          exps(v, pair(-mn, -mn), e01, e23);
          const float2 s = unpair(add2(e01, e23));
          ms = make_float2(mn, ms.y * ex2(ms.x - mn) + (s.x + s.y));
        }
      }
    });
    if (!FULL && je >= 0) {
      if (CAP) edge = tanh_of(edge);
      if (REGS > 0) {
        ms.x = fmaxf(ms.x, edge);
      } else {
        const float mn = fmaxf(ms.x, edge * kx);
        if (mn != -INFINITY) ms = make_float2(mn, ms.y * ex2(ms.x - mn) + ex2(fmaf(edge, kx, -mn)));
      }
    }
    const float m = warp_max_redux(ms.x) * (REGS > 0 ? kx : 1.0f);
    if constexpr (REGS > 0) {
      if (m != -INFINITY) {
        const uint64_t minus_m = pair(-m, -m);
        uint64_t sum = 0ull;  // a pair of zeros
        each(j_first, std::false_type{}, [&](int, float4& v) {
          uint64_t e01, e23;
          exps(v, minus_m, e01, e23);
          sum = add2(sum, add2(e01, e23));
        });
        const float2 s = unpair(sum);
        ms.y = s.x + s.y;
        if (!FULL && je >= 0) ms.y += ex2(fmaf(edge, kx, -m));
      }
    } else {
      ms.y = ms.x == -INFINITY ? 0.0f : ms.y * ex2(ms.x - m);
    }
    ms = make_float2(m, warp_sum(ms.y));
    if (lane == 0) sh.part_w[warp] = ms;
  }
  auto part_of = [&](const float2* v, int n) { return lane < n ? v[lane] : make_float2(-INFINITY, 0.0f); };
  // The row's warps meet (the helper is not waited for), and warp 0 sends the CTA's
  // part to every CTA of the cluster; each waits for all of them to arrive.
  if (!helper) {
    named_sync(1, kThreads);
    if (warp == 0) {
      ms = join8(part_of(sh.part_w, kThreads / 32));
      asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // every CTA of the cluster runs
      if (lane < CS)
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(
                         mapa_shared(smem_u32(&sh.part[rank]), lane)),
                     "l"(((uint64_t)__float_as_uint(ms.y) << 32) | __float_as_uint(ms.x)),
                     "r"(mapa_shared(smem_u32(&sh.bar), lane))
                     : "memory");
    }
  }
  if (warp != 0) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  {
    // A part that comes too late to count is still waited for, as long again: it lands in
    // this CTA's shared memory, which must be there.
    bool late = false;
    if (!mbar_try_wait_cluster(smem_u32(&sh.bar), 0)) {
      const uint64_t t0 = global_timer_ns();
      uint64_t waited = 0;
      for (uint32_t it = 1; waited <= 2 * kWaitLimitNs && !mbar_try_wait_cluster(smem_u32(&sh.bar), 0); ++it)
        if ((it & 255u) == 0u) waited = global_timer_ns() - t0;
      late = waited > kWaitLimitNs;
    }
    if (__any_sync(0xffffffffu, late)) {  // this warp writes nothing (others may have seen the parts in time)
      if (lane == 0 && p.status) atomicOr(p.status, NC_DEV_TIMEOUT);
      if (DZ != 0 && !helper) named_arrive(2, kBlock);
      return;
    }
  }
  ms = join8(part_of(sh.part, CS));
  const float xm = ms.x, xs = __shfl_sync(0xffffffffu, ms.y, 0);

  auto store_loss = [&] {  // the helper's
    const float xlse = logf(xs);
    float loss = 0.0f;
    for (int k = lane; k < K; k += 32) {
      const float lq = q_s[k] - t_lse, q = t_any ? expf(lq) : 0.0f;
      if (q > 0.0f) {
        const float t = CAP ? tanh_of(z_s[k]) : z_s[k];
        loss = fmaf(q, lq - (fmaf(t, kx, -xm) * 0.6931471805599453f - xlse), loss);
      }
    }
    loss = warp_sum(loss);
    if (lane == 0) p.loss[blockIdx.y] = t_any ? p.tau * p.tau * loss : 0.0f;
  };
  auto slope = [&](float t) { return CAP ? fmaf(-t, t, 1.0f) : 1.0f; };
  if constexpr (DZ != 0) {
    const int64_t row = fresh_row();
    const int rank = fresh_rank(), tid = fresh_tid(), lane = tid & 31;
    const int off = (int)((reinterpret_cast<uintptr_t>(p.z + row * p.V) >> 2) & 3), end = off + p.V;
    const int s0 = rank * slice, s1 = min(end, s0 + slice), j_first = s0 + tid * 4;
    const float wp = p.tau * (p.weight ? p.weight[row] : 1.0f) / xs;
    constexpr int ES = DZ == 1 ? 4 : 2;
    uint8_t* dr = static_cast<uint8_t*>(p.dz) + row * V * ES - (int64_t)off * ES;  // position 0
    const bool vec = (reinterpret_cast<uintptr_t>(dr) & (4 * ES - 1)) == 0;
    auto store1 = [&](int j, float v) {
      if constexpr (DZ == 1)
        reinterpret_cast<float*>(dr)[j] = v;
      else
        reinterpret_cast<uint16_t*>(dr)[j] = (uint16_t)Half<DZ == 3>::pack2(v, 0.0f);
    };
    if (!helper) {
      each(j_first, std::false_type{}, [&](int j, float4& v) {
        const float4 t = CAP && REGS == 0 ? tanh_of(v) : v;
        uint64_t e01, e23;
        exps(t, pair(-xm, -xm), e01, e23);
        auto scaled = [&](uint64_t e, uint64_t u) {  // w tau / sum (1 - u^2) e
          const uint64_t w2 = pair(wp, wp);
          return unpair(mul2(e, CAP ? fma2(mul2(u, pair(-wp, -wp)), u, w2) : w2));
        };
        const float2 d01 = scaled(e01, pair(t.x, t.y)), d23 = scaled(e23, pair(t.z, t.w));
        const float4 d = make_float4(d01.x, d01.y, d23.x, d23.y);
        if (vec) {
          if constexpr (DZ == 1)
            __stcs(reinterpret_cast<float4*>(dr + (int64_t)j * 4), d);
          else
            __stcs(reinterpret_cast<uint2*>(dr + (int64_t)j * 2),
                   make_uint2(Half<DZ == 3>::pack2(d.x, d.y), Half<DZ == 3>::pack2(d.z, d.w)));
        } else {
          store1(j, d.x);
          store1(j + 1, d.y);
          store1(j + 2, d.z);
          store1(j + 3, d.w);
        }
      });
      if (!FULL && je >= 0) store1(je, ex2(fmaf(edge, kx, -xm)) * (wp * slope(edge)));
      named_arrive(2, kBlock);
    } else {
      // the entries' gradients, while the row is stored; then they go over it
      const float tlse = t_lse, w = p.tau * (p.weight ? p.weight[row] : 1.0f), inv = 1.0f / xs;
      const int n = t_any ? n_here : 0;
      __syncwarp();
      auto insert = [&](int i) {  // into a table of 2 K slots or more
        for (int h = i;; ++h) {
          const int was = atomicCAS(&table[h & (slots - 1)], -1, i);
          if (was == -1) return;
          if ((was & ~kTwice) == i) {
            atomicOr(&table[h & (slots - 1)], kTwice);
            return;
          }
        }
      };
      auto is_twice = [&](int i) {
        int h = i;
        while ((table[h & (slots - 1)] & ~kTwice) != i) ++h;
        return (table[h & (slots - 1)] & kTwice) != 0;
      };
      if (n > 32) {
        for (int k = lane; k < slots; k += 32) table[k] = -1;
        __syncwarp();
        for (int e = lane; e < n; e += 32) insert(i_s[list[e]]);
        __syncwarp();
      }
      uint32_t mine = 0u;  // the lane's entries that are stored, 32 of them at most
      for (int e0 = 0, turn = 0; e0 < n; e0 += 32, ++turn) {
        const bool in = e0 + lane < n;
        const int k = in ? list[e0 + lane] : 0, i = in ? i_s[k] : -1 - lane;
        float q = in ? expf(q_s[k] - tlse) : 0.0f;
        bool first = in;
        const bool twice = n > 32 ? in && is_twice(i) : (__match_any_sync(0xffffffffu, i) & ~(1u << lane)) != 0u;
        // an index given more than once: the sum over its entries, stored by the first
        for (uint32_t bal = __ballot_sync(0xffffffffu, twice); bal != 0u; bal &= bal - 1u) {
          const int s = __ffs(bal) - 1, is = __shfl_sync(0xffffffffu, i, s);
          float sum = 0.0f;
          int least = n;
          for (int f = lane; f < n; f += 32)
            if (i_s[list[f]] == is) {
              sum += expf(q_s[list[f]] - tlse);
              least = min(least, f);
            }
          sum = warp_sum(sum);
          least = __reduce_min_sync(0xffffffffu, least);
          if (lane == s) {
            q = sum;
            first = least == e0 + lane;
          }
        }
        if (in) {
          const float t = CAP ? tanh_of(z_s[k]) : z_s[k];
          g_s[e0 + lane] = (ex2(fmaf(t, kx, -xm)) * inv - q) * w * slope(t);
        }
        if (first) mine |= 1u << turn;
      }
      if (rank == 0) store_loss();
      named_sync(2, kBlock);
      for (int e = lane; mine != 0u; e += 32, mine >>= 1)
        if (mine & 1u) store1(off + i_s[list[e]], g_s[e]);
      if (!t_any)  // no entry: no gradient
        for (int j = max(s0, off) + lane; j < s1; j += 32) store1(j, 0.0f);
    }
  } else {
    if (helper && rank == 0) store_loss();
  }
}

template <int DZ, bool CAP, int REGS>
__global__ void __launch_bounds__(kBlock, resident(DZ, REGS))
    distill_kernel(const DistillParams p, int slice, int slots) {
  extern __shared__ __align__(16) float mem[];
  __shared__ Shared sh;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&sh.bar), 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(smem_u32(&sh.bar), gridDim.x * 8);
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int off = (int)((reinterpret_cast<uintptr_t>(p.z + (int64_t)blockIdx.y * p.V) >> 2) & 3);
  const int s0 = blockIdx.x * slice;
  if (REGS == 8 && s0 >= off && s0 + REGS * 4 * kThreads <= off + p.V)
    distill_part<DZ, CAP, REGS, true>(p, slice, slots, mem, sh);
  else
    distill_part<DZ, CAP, REGS, false>(p, slice, slots, mem, sh);
}

template <int DZ, bool CAP, int REGS>
nc_status launch_r(const DistillParams& p, int M, int cs, int slice, cudaStream_t stream) {
  for (int m0 = 0; m0 < M; m0 += 65535) {  // rows on the grid's y
    DistillParams q = p;
    const int64_t at = m0;
    q.z += at * p.V;
    q.idx += at * p.K;
    q.teacher += at * p.K;
    if (q.weight) q.weight += at;
    q.loss += at;
    if (q.dz) q.dz = static_cast<uint8_t*>(p.dz) + at * p.V * (DZ == 1 ? 4 : 2);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(cs, M - m0 < 65535 ? M - m0 : 65535);
    cfg.blockDim = dim3(kBlock);
    int slots = 2;
    while (slots < 2 * p.K) slots *= 2;
    cfg.dynamicSmemBytes = (size_t)((REGS - held(DZ, REGS)) * kThreads * 4 + 5 * p.K + slots) * 4;
    cfg.stream = stream;
    cudaLaunchAttribute a{};
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim.x = cs;
    a.val.clusterDim.y = 1;
    a.val.clusterDim.z = 1;
    cfg.attrs = &a;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, distill_kernel<DZ, CAP, REGS>, q, slice, slots) != cudaSuccess) return NC_ERR_CUDA;
  }
  return NC_OK;
}

template <int DZ, bool CAP>
nc_status launch_t(const DistillParams& p, int M, cudaStream_t stream) {
  // groups of four positions in the worst row's alignment
  const bool even = p.V % 4 == 0 && aligned16(p.z);
  const int groups = even ? p.V / 4 : (p.V + 6) / 4;
  if (groups <= kThreads) return launch_r<DZ, CAP, 1>(p, M, 1, 4 * kThreads, stream);
  if (groups <= 4 * kThreads) return launch_r<DZ, CAP, 4>(p, M, 1, 16 * kThreads, stream);
  const int cs = (groups + 8 * kThreads - 1) / (8 * kThreads);
  if (cs <= 8) return launch_r<DZ, CAP, 8>(p, M, cs, 32 * kThreads, stream);
  return launch_r<DZ, CAP, 0>(p, M, 1, 4 * groups, stream);
}

template <int DZ>
nc_status launch_c(const DistillParams& p, int M, float cap, cudaStream_t stream) {
  return cap > 0.0f ? launch_t<DZ, true>(p, M, stream) : launch_t<DZ, false>(p, M, stream);
}

}  // namespace

nc_status distill_topk_launch(const float* z, const int32_t* idx, const float* teacher, const float* weight,
                              float* loss, void* dz, int dz_kind, int M, int V, int K, float tau, float cap,
                              uint32_t* dev_status, cudaStream_t stream) {
  if (M == 0) return NC_OK;
  const DistillParams p{z, idx, teacher, weight, loss, dz, V, K, tau, 1.0f / tau, (cap > 0.0f ? cap : 1.0f) / tau * kLog2e,
                        Tanh(cap > 0.0f ? cap : 1.0f), dev_status};
  switch (dz_kind) {
    case 0: return launch_c<0>(p, M, cap, stream);
    case 1: return launch_c<1>(p, M, cap, stream);
    case 2: return launch_c<2>(p, M, cap, stream);
    default: return launch_c<3>(p, M, cap, stream);
  }
}

}  // namespace nc
