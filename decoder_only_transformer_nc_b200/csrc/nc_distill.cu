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
// and gradient 0.  Softmax statistics and sums are fp32 in a fixed order.
#include <cuda_runtime.h>

#include <cstdint>

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
  explicit Tanh(float cap) {
    inv_cap = 1.0f / cap;
    near = kNear * cap;
    const float c2 = inv_cap * inv_cap;
    a1 = 1260.0f / 10395.0f * (c2 * inv_cap);
    a2 = 21.0f / 10395.0f * (c2 * c2 * inv_cap);
    b1 = 4725.0f / 10395.0f * c2;
    b2 = 210.0f / 10395.0f * (c2 * c2);
    b3 = 1.0f / 10395.0f * (c2 * c2 * c2);
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
  // four at a time; the far form only where some lane of the warp needs it
  __device__ __forceinline__ float4 operator()(const float4& z) const {
    float4 t = make_float4(close(z.x), close(z.y), close(z.z), close(z.w));
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

// (maximum, sum) of two parts of a softmax, log2 domain.
__device__ __forceinline__ float2 join(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  if (m == -INFINITY) return make_float2(m, 0.0f);
  return make_float2(m, fmaf(a.y, ex2(a.x - m), b.y * ex2(b.x - m)));
}

// A row is dealt over the CTAs of a cluster (one CTA up to 8192 logits), every
// thread holding its REGS groups of four logits in registers from the one read
// to the gradient's store, so z and dz cross the memory bus once.  Four CTAs of
// 256 threads share an SM, at different points of different rows: one loads
// while another computes or stores.  The threads' (maximum, sum) are joined over
// the block and, through distributed shared memory, over the cluster, in a fixed
// order.  The teacher's entries are the business of a warp of its own: with K = 64 beside
// 8192 logits, eight warps repeating it took as many instructions as the row.
// REGS = 0: longer rows, one CTA, read again from L2 for each use.
// Groups of four start at 16-byte boundaries of z's row (the ends and a dz that is
// not aligned alike go by single elements).
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

// FULL: every thread has REGS whole groups (no test of a group's place).
template <int DZ, bool CAP, int REGS, bool FULL>
__device__ __forceinline__ void distill_part(const DistillParams& p, int slice, int slots, float* q_s, Shared& sh) {
  //  // [K] logits, then probabilities; [K] z of the entry; [K] indices; [slots]
  float* z_s = q_s + p.K;
  int32_t* i_s = reinterpret_cast<int32_t*>(z_s + p.K);
  int32_t* table = i_s + p.K;
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
  auto load = [&](int j) -> float4 {
    if (FULL || (j >= off && j + 4 <= end)) return __ldcs(reinterpret_cast<const float4*>(z + j));
    float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    if (j >= off && j < end) v.x = z[j];
    if (j + 1 >= off && j + 1 < end) v.y = z[j + 1];
    if (j + 2 >= off && j + 2 < end) v.z = z[j + 2];
    if (j + 3 >= off && j + 3 < end) v.w = z[j + 3];
    return v;
  };
  constexpr int STEP = kThreads * 4;
  const int j_first = s0 + tid * 4;
  // groups of this thread (0 or less: none)
  const int nr = warp == kThreads / 32 ? 0 : (s1 - j_first + STEP - 1) / STEP;
  float4 keep[REGS > 0 ? REGS : 1];
  if constexpr (REGS > 0) {
#pragma unroll
    for (int r = 0; r < REGS; ++r)
      if (FULL ? warp < kThreads / 32 : r < nr) keep[r] = load(j_first + r * STEP);
  }
  auto each = [&](auto f) {
    if constexpr (REGS > 0) {
#pragma unroll
      for (int r = 0; r < REGS; ++r)
        if (FULL || r < nr) f(j_first + r * STEP, keep[r]);
    } else {
#pragma unroll 1
      for (int j = j_first, r = 0; r < nr; ++r, j += STEP) {
        float4 v = load(j);
        f(j, v);
      }
    }
  };

  // the teacher's softmax, while the row is on its way
  const bool helper = warp == kThreads / 32;
  bool t_any = true, t_twice = false;  // the helper's
  float t_lse = 0.0f;
  if (helper) {
    float tm = -INFINITY;
    for (int k = lane; k < slots; k += 32) table[k] = -1;
    for (int k = lane; k < K; k += 32) {
      int i = p.idx[row * K + k];
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
    tm = warp_max(tm);
    const bool any = tm != -INFINITY;
    float ts = 0.0f;
    for (int k = lane; k < K; k += 32) ts += any ? expf(q_s[k] - tm) : 0.0f;
    ts = warp_sum(ts);
    bool twice = false;
    if (DZ != 0) {  // is an index given more than once?  (a table of 2 K slots or more)
      __syncwarp();
      for (int k = lane; k < K; k += 32) {
        const int i = i_s[k];
        for (int h = i; i >= 0; ++h) {
          const int was = atomicCAS(&table[h & (slots - 1)], -1, i);
          twice = twice || was == i;
          if (was == -1 || was == i) break;
        }
      }
      twice = __any_sync(0xffffffffu, twice);
    }
    t_any = any;
    t_twice = twice;
    t_lse = any ? tm + logf(ts) : 0.0f;
  }

  // the student's softmax: with registers, t takes the place of z
  float2 ms = make_float2(-INFINITY, 0.0f);
  auto sum4 = [&](const float4& v, float m) {
    return (ex2(fmaf(v.x, kx, -m)) + ex2(fmaf(v.y, kx, -m))) + (ex2(fmaf(v.z, kx, -m)) + ex2(fmaf(v.w, kx, -m)));
  };
  if (!helper) {
    each([&](int j, float4& v) {
      if (CAP) {
        v = tanh_of(v);
        if (!FULL && (j < off || j + 4 > end)) {  // positions outside the row stay -inf
          if (j < off || j >= end) v.x = -INFINITY;
          if (j + 1 < off || j + 1 >= end) v.y = -INFINITY;
          if (j + 2 < off || j + 2 >= end) v.z = -INFINITY;
          if (j + 3 < off || j + 3 >= end) v.w = -INFINITY;
        }
      }
      const float m = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
      if (REGS > 0) {
        ms.x = fmaxf(ms.x, m);
      } else {
        const float mn = fmaxf(ms.x, m * kx);
        if (mn != -INFINITY) ms = make_float2(mn, ms.y * ex2(ms.x - mn) + sum4(v, mn));
      }
    });
    if constexpr (REGS > 0) {
      ms.x *= kx;
      if (ms.x != -INFINITY) each([&](int, float4& v) { ms.y += sum4(v, ms.x); });
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      ms = join(ms, make_float2(__shfl_xor_sync(0xffffffffu, ms.x, o), __shfl_xor_sync(0xffffffffu, ms.y, o)));
    if (lane == 0) sh.part_w[warp] = ms;
  }
  auto join_lanes = [&](const float2* v, int n) {  // n <= 8 parts, in a fixed tree
    float2 x = lane < n ? v[lane] : make_float2(-INFINITY, 0.0f);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
      x = join(x, make_float2(__shfl_xor_sync(0xffffffffu, x.x, o), __shfl_xor_sync(0xffffffffu, x.y, o)));
    return make_float2(__shfl_sync(0xffffffffu, x.x, 0), __shfl_sync(0xffffffffu, x.y, 0));
  };
  // The row's warps meet (the helper is not waited for), and warp 0 sends the CTA's
  // part to every CTA of the cluster; each waits for all of them to arrive.
  if (!helper) {
    named_sync(1, kThreads);
    if (warp == 0) {
      ms = join_lanes(sh.part_w, kThreads / 32);
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
    bool late = false;
    if (!mbar_try_wait_cluster(smem_u32(&sh.bar), 0)) {
      const uint64_t t0 = global_timer_ns();
      for (uint32_t it = 1; !late && !mbar_try_wait_cluster(smem_u32(&sh.bar), 0); ++it)
        if ((it & 255u) == 0u) late = global_timer_ns() - t0 > kWaitLimitNs;
    }
    if (__any_sync(0xffffffffu, late)) {  // a CTA of the cluster never came: nothing is written
      if (lane == 0 && p.status) atomicOr(p.status, NC_DEV_TIMEOUT);
      if (DZ != 0 && !helper) named_arrive(2, kBlock);
      return;
    }
  }
  ms = join_lanes(sh.part, CS);
  const float xm = ms.x, xs = ms.y;

  auto slope = [&](float t) { return CAP ? fmaf(-t, t, 1.0f) : 1.0f; };
  if constexpr (DZ != 0) {
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
      each([&](int j, float4& v) {
        const float4 t = CAP && REGS == 0 ? tanh_of(v) : v;
        const float4 d = make_float4(ex2(fmaf(t.x, kx, -xm)) * (wp * slope(t.x)), ex2(fmaf(t.y, kx, -xm)) * (wp * slope(t.y)),
                                     ex2(fmaf(t.z, kx, -xm)) * (wp * slope(t.z)), ex2(fmaf(t.w, kx, -xm)) * (wp * slope(t.w)));
        if (vec && (FULL || (j >= off && j + 4 <= end))) {
          if constexpr (DZ == 1)
            __stcs(reinterpret_cast<float4*>(dr + (int64_t)j * 4), d);
          else
            __stcs(reinterpret_cast<uint2*>(dr + (int64_t)j * 2),
                   make_uint2(Half<DZ == 3>::pack2(d.x, d.y), Half<DZ == 3>::pack2(d.z, d.w)));
        } else {
          if (j >= off && j < end) store1(j, d.x);
          if (j + 1 >= off && j + 1 < end) store1(j + 1, d.y);
          if (j + 2 >= off && j + 2 < end) store1(j + 2, d.z);
          if (j + 3 >= off && j + 3 < end) store1(j + 3, d.w);
        }
      });
      named_arrive(2, kBlock);
    } else {
      named_sync(2, kBlock);  // the row is stored; the teacher's entries go over it
      const float tlse = t_lse, w = p.tau * (p.weight ? p.weight[row] : 1.0f), inv = 1.0f / xs;
      if (!t_any)  // no entry: no gradient
        for (int j = max(s0, off) + lane; j < s1; j += 32) store1(j, 0.0f);
      const bool twice = t_twice;
      for (int k = lane; k < K && t_any; k += 32) {
        const int i = i_s[k];
        if (i < 0 || off + i < s0 || off + i >= s1) continue;
        float q = expf(q_s[k] - tlse);
        bool first = true;
        if (twice) {  // its first entry stores for all
          q = 0.0f;
          for (int j = 0; j < K; ++j)
            if (i_s[j] == i) {
              first = first && j >= k;
              q += expf(q_s[j] - tlse);
            }
        }
        const float t = CAP ? tanh_of(z_s[k]) : z_s[k];
        if (first) store1(off + i, (ex2(fmaf(t, kx, -xm)) * inv - q) * w * slope(t));
      }
    }
  }
  if (helper && rank == 0) {
    const bool any = t_any;
    const float tlse = t_lse, xlse = logf(xs);
    float loss = 0.0f;
    for (int k = lane; k < K; k += 32) {
      const float lq = q_s[k] - tlse, q = any ? expf(lq) : 0.0f;
      if (q > 0.0f) {
        const float t = CAP ? tanh_of(z_s[k]) : z_s[k];
        loss = fmaf(q, lq - (fmaf(t, kx, -xm) * 0.6931471805599453f - xlse), loss);
      }
    }
    loss = warp_sum(loss);
    if (lane == 0) p.loss[row] = any ? p.tau * p.tau * loss : 0.0f;
  }
}

template <int DZ, bool CAP, int REGS>
__global__ void __launch_bounds__(kBlock, REGS == 8 ? 4 : 1)
    distill_kernel(const DistillParams p, int slice, int slots) {
  extern __shared__ float q_s[];
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
    distill_part<DZ, CAP, REGS, true>(p, slice, slots, q_s, sh);
  else
    distill_part<DZ, CAP, REGS, false>(p, slice, slots, q_s, sh);
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
    cfg.dynamicSmemBytes = (size_t)(3 * p.K + slots) * 4;
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
