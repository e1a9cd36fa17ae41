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

constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

struct DistillParams {
  const float* z;         // [M][V]
  const int32_t* idx;     // [M][K]
  const float* teacher;   // [M][K]
  const float* weight;    // [M] or null
  float* loss;            // [M]
  void* dz;               // [M][V] or null
  int V, K;
  float cap, tau;
  uint32_t* status;
};

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

template <bool MAX>
__device__ __forceinline__ float block_all(float v, float* red) {
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = MAX ? warp_max(v) : warp_sum(v);
  __syncthreads();
  if (lane == 0) red[w] = v;
  __syncthreads();
  float t = lane < kThreads / 32 ? red[lane] : (MAX ? -INFINITY : 0.0f);
  return MAX ? warp_max(t) : warp_sum(t);
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

// tanh(u).  Up to |u| = 0.55, where most logits are under their cap, the odd
// series u - u^3/3 + 2 u^5/15 - ... to u^13 (the next term is 8e-7 of u there):
// no special-function unit, which would bound these passes.  Beyond, 1 - 2 /
// (e^2u + 1), whose absolute error is that of its 1.
__device__ __forceinline__ float tanh_small(float u) {
  const float s = u * u;
  float r = 3.5921280365724810e-03f;               // 21844 / 6081075
  r = fmaf(r, s, -8.8632355299021966e-03f);        // -1382 / 155925
  r = fmaf(r, s, 2.1869488536155203e-02f);         // 62 / 2835
  r = fmaf(r, s, -5.3968253968253971e-02f);        // -17 / 315
  r = fmaf(r, s, 1.3333333333333333e-01f);         // 2 / 15
  r = fmaf(r, s, -3.3333333333333331e-01f);        // -1 / 3
  return fmaf(r * s, u, u);
}
__device__ __forceinline__ float tanh_any(float u) {
  return copysignf(fmaf(-2.0f, rcp(1.0f + ex2(2.0f * kLog2e * fabsf(u))), 1.0f), u);
}

// The four logits' tanh; the slow form only where some lane of the warp needs it.
__device__ __forceinline__ void tanh4(const float4& z, float inv_cap, float (&t)[4]) {
  const float u[4] = {z.x * inv_cap, z.y * inv_cap, z.z * inv_cap, z.w * inv_cap};
#pragma unroll
  for (int e = 0; e < 4; ++e) t[e] = tanh_small(u[e]);
  const float m = fmaxf(fmaxf(fabsf(u[0]), fabsf(u[1])), fmaxf(fabsf(u[2]), fabsf(u[3])));
  if (!(m <= 0.55f)) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (!(fabsf(u[e]) <= 0.55f)) t[e] = tanh_any(u[e]);
  }
}

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
// order.  REGS = 0: longer rows, one CTA, read again from L2 for each use.
// Groups of four start at 16-byte boundaries of z's row (the ends and a dz that is
// not aligned alike go by single elements).
// DZ: 0 none, 1 fp32, 2 bf16, 3 fp16
template <int DZ, bool CAP, int REGS>
__global__ void __launch_bounds__(kThreads, REGS == 8 ? 4 : 1) distill_kernel(const DistillParams p, int slice) {
  extern __shared__ float q_s[];  // [K] probabilities, then [K] indices
  __shared__ float red[32];
  __shared__ float2 part[8], part_w[kThreads / 32];
  int32_t* i_s = reinterpret_cast<int32_t*>(q_s + p.K);
  const int64_t row = blockIdx.y;
  const int rank = blockIdx.x, CS = gridDim.x;  // the cluster spans the grid's x
  const int V = p.V, K = p.K, tid = threadIdx.x;
  const float* zr = p.z + row * V;
  const int off = (int)((reinterpret_cast<uintptr_t>(zr) >> 2) & 3);  // logit 0 is position off
  const float* z = zr - off;
  const int end = off + V;
  const int s0 = rank * slice, s1 = min(end, s0 + slice);  // this CTA's positions
  if (CS > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const float inv_tau = 1.0f / p.tau;
  const float cap = p.cap, inv_cap = CAP ? 1.0f / cap : 0.0f;
  const float kx = (CAP ? cap : 1.0f) * inv_tau * kLog2e;  // x (log2) of t or z
  auto load = [&](int j) -> float4 {
    if (j >= off && j + 4 <= end) return __ldcs(reinterpret_cast<const float4*>(z + j));
    float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    if (j >= off && j < end) v.x = z[j];
    if (j + 1 >= off && j + 1 < end) v.y = z[j + 1];
    if (j + 2 >= off && j + 2 < end) v.z = z[j + 2];
    if (j + 3 >= off && j + 3 < end) v.w = z[j + 3];
    return v;
  };
  constexpr int STEP = kThreads * 4;
  const int j_first = s0 + tid * 4;
  float4 keep[REGS > 0 ? REGS : 1];
  if constexpr (REGS > 0) {
#pragma unroll
    for (int r = 0; r < REGS; ++r)
      if (j_first + r * STEP < s1) keep[r] = load(j_first + r * STEP);
  }
  auto each = [&](auto f) {
    if constexpr (REGS > 0) {
#pragma unroll
      for (int r = 0; r < REGS; ++r)
        if (j_first + r * STEP < s1) f(j_first + r * STEP, keep[r]);
    } else {
#pragma unroll 1
      for (int j = j_first; j < s1; j += STEP) {
        float4 v = load(j);
        f(j, v);
      }
    }
  };

  // teacher's softmax (every CTA for itself), while the row is on its way
  float tm = -INFINITY;
  for (int k = tid; k < K; k += kThreads) {
    int i = p.idx[row * K + k];
    if (i < -1 || i >= V) {
      if (p.status) atomicOr(p.status, NC_DEV_TARGET_RANGE);
      i = -1;
    }
    const float t = i < 0 ? -INFINITY : p.teacher[row * K + k] * inv_tau;
    i_s[k] = i;
    q_s[k] = t;
    tm = fmaxf(tm, t);
  }
  tm = block_all<true>(tm, red);
  const bool any = tm != -INFINITY;
  float ts = 0.0f;
  for (int k = tid; k < K; k += kThreads) ts += any ? expf(q_s[k] - tm) : 0.0f;
  ts = block_all<false>(ts, red);
  const float tlse = any ? tm + logf(ts) : 0.0f;

  // the student's softmax: with registers, t takes the place of z
  float2 ms = make_float2(-INFINITY, 0.0f);
  each([&](int j, float4& v) {
    if (CAP) {
      float t[4];
      tanh4(v, inv_cap, t);
      if (j < off || j + 4 > end) {  // positions outside the row stay -inf
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (j + q < off || j + q >= end) t[q] = -INFINITY;
      }
      v = make_float4(t[0], t[1], t[2], t[3]);
    }
    if (REGS > 0) {
      ms.x = fmaxf(ms.x, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)));
    } else {
      const float m = fmaxf(ms.x, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)) * kx);
      if (m != -INFINITY)
        ms = make_float2(m, ms.y * ex2(ms.x - m) + ((ex2(fmaf(v.x, kx, -m)) + ex2(fmaf(v.y, kx, -m))) +
                                                    (ex2(fmaf(v.z, kx, -m)) + ex2(fmaf(v.w, kx, -m)))));
    }
  });
  if constexpr (REGS > 0) {
    ms.x *= kx;
    if (ms.x != -INFINITY)
      each([&](int, float4& v) {
        ms.y += (ex2(fmaf(v.x, kx, -ms.x)) + ex2(fmaf(v.y, kx, -ms.x))) +
                (ex2(fmaf(v.z, kx, -ms.x)) + ex2(fmaf(v.w, kx, -ms.x)));
      });
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    ms = join(ms, make_float2(__shfl_xor_sync(0xffffffffu, ms.x, o), __shfl_xor_sync(0xffffffffu, ms.y, o)));
  if ((tid & 31) == 0) part_w[tid >> 5] = ms;
  __syncthreads();
  ms = part_w[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) ms = join(ms, part_w[w]);
  if (CS > 1) {
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // every CTA of the cluster runs
    if (tid < CS)
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(mapa_shared(smem_u32(&part[rank]), tid)),
                   "f"(ms.x), "f"(ms.y)
                   : "memory");
    cluster_sync();
    ms = part[0];
    for (int c = 1; c < CS; ++c) ms = join(ms, part[c]);
  }
  const float xm = ms.x, xs = ms.y, xlse = logf(xs);

  // x of one logit read again (the teacher's entries)
  auto one = [&](float v, float& t) -> float {
    const float u = v * inv_cap;
    t = CAP ? (fabsf(u) <= 0.55f ? tanh_small(u) : tanh_any(u)) : v;
    return fmaf(t, kx, -xm);
  };
  float loss = 0.0f;
  for (int k = tid; k < K; k += kThreads) {
    const int i = i_s[k];
    const float lq = q_s[k] - tlse, q = any ? expf(lq) : 0.0f;
    if (rank == 0 && q > 0.0f) {
      float t;
      loss = fmaf(q, lq - (one(zr[i], t) * 0.6931471805599453f - xlse), loss);
    }
    q_s[k] = q;
  }
  if (rank == 0) {
    loss = block_all<false>(loss, red);
    if (tid == 0) p.loss[row] = any ? p.tau * p.tau * loss : 0.0f;
  }

  if constexpr (DZ != 0) {
    const float w = any ? p.tau * (p.weight ? p.weight[row] : 1.0f) : 0.0f;
    const float inv = any ? 1.0f / xs : 0.0f;
    const float wp = w * inv;
    constexpr int ES = DZ == 1 ? 4 : 2;
    uint8_t* dr = static_cast<uint8_t*>(p.dz) + row * V * ES - (int64_t)off * ES;  // position 0
    const bool vec = (reinterpret_cast<uintptr_t>(dr) & (4 * ES - 1)) == 0;
    auto store1 = [&](int j, float v) {
      if constexpr (DZ == 1)
        reinterpret_cast<float*>(dr)[j] = v;
      else
        reinterpret_cast<uint16_t*>(dr)[j] = (uint16_t)Half<DZ == 3>::pack2(v, 0.0f);
    };
    auto slope = [&](float t) { return CAP ? fmaf(-t, t, 1.0f) : 1.0f; };
    each([&](int j, float4& v) {
      float t[4] = {v.x, v.y, v.z, v.w};
      if (CAP && REGS == 0) tanh4(v, inv_cap, t);
      float d[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) d[q] = any ? ex2(fmaf(t[q], kx, -xm)) * wp * slope(t[q]) : 0.0f;
      if (vec && j >= off && j + 4 <= end) {
        if constexpr (DZ == 1)
          __stcs(reinterpret_cast<float4*>(dr + (int64_t)j * 4), make_float4(d[0], d[1], d[2], d[3]));
        else
          __stcs(reinterpret_cast<uint2*>(dr + (int64_t)j * 2),
                 make_uint2(Half<DZ == 3>::pack2(d[0], d[1]), Half<DZ == 3>::pack2(d[2], d[3])));
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (j + q >= off && j + q < end) store1(j + q, d[q]);
      }
    });
    __syncthreads();
    for (int k = tid; k < K; k += kThreads) {
      const int i = i_s[k];
      if (i < 0 || off + i < s0 || off + i >= s1) continue;
      float q = 0.0f;  // an index given more than once: its first entry stores for all
      bool first = true;
      for (int j = 0; j < K; ++j)
        if (i_s[j] == i) {
          first = first && j >= k;
          q += q_s[j];
        }
      float t;
      const float x = one(zr[i], t);
      if (first) store1(off + i, any ? (ex2(x) * inv - q) * w * slope(t) : 0.0f);
    }
  }
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
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)p.K * 8;
    cfg.stream = stream;
    cudaLaunchAttribute a{};
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim.x = cs;
    a.val.clusterDim.y = 1;
    a.val.clusterDim.z = 1;
    cfg.attrs = &a;
    cfg.numAttrs = cs > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, distill_kernel<DZ, CAP, REGS>, q, slice) != cudaSuccess) return NC_ERR_CUDA;
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
  if (cs <= 8) return launch_r<DZ, CAP, 8>(p, M, cs, (groups + cs - 1) / cs * 4, stream);
  return launch_r<DZ, CAP, 0>(p, M, 1, 4 * groups, stream);
}

template <int DZ>
nc_status launch_c(const DistillParams& p, int M, cudaStream_t stream) {
  return p.cap > 0.0f ? launch_t<DZ, true>(p, M, stream) : launch_t<DZ, false>(p, M, stream);
}

}  // namespace

nc_status distill_topk_launch(const float* z, const int32_t* idx, const float* teacher, const float* weight,
                              float* loss, void* dz, int dz_kind, int M, int V, int K, float tau, float cap,
                              uint32_t* dev_status, cudaStream_t stream) {
  if (M == 0) return NC_OK;
  const DistillParams p{z, idx, teacher, weight, loss, dz, V, K, cap, tau, dev_status};
  switch (dz_kind) {
    case 0: return launch_c<0>(p, M, stream);
    case 1: return launch_c<1>(p, M, stream);
    case 2: return launch_c<2>(p, M, stream);
    default: return launch_c<3>(p, M, stream);
  }
}

}  // namespace nc
