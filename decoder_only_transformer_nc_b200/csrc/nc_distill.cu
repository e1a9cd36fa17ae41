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

namespace nc {
namespace {

constexpr int kThreads = 512;

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

// DZ: 0 none, 1 fp32, 2 bf16, 3 fp16
template <int DZ>
__global__ void __launch_bounds__(kThreads) distill_kernel(const DistillParams p) {
  extern __shared__ float q_s[];  // [K] probabilities, then [K] indices
  __shared__ float red[32];
  int32_t* i_s = reinterpret_cast<int32_t*>(q_s + p.K);
  const int64_t row = blockIdx.x;
  const int V = p.V, K = p.K;
  const float* z = p.z + row * V;
  const float cap = p.cap, inv_tau = 1.0f / p.tau;
  const float inv_cap = cap > 0.0f ? 1.0f / cap : 0.0f;
  auto tanh_of = [&](float v) { return tanhf(v * inv_cap); };

  // teacher's softmax
  float tm = -INFINITY;
  for (int k = threadIdx.x; k < K; k += kThreads) {
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
  for (int k = threadIdx.x; k < K; k += kThreads) ts += any ? expf(q_s[k] - tm) : 0.0f;
  ts = block_all<false>(ts, red);
  const float tlse = any ? tm + logf(ts) : 0.0f;

  // student's softmax
  float xm = -INFINITY;
  for (int i = threadIdx.x; i < V; i += kThreads) xm = fmaxf(xm, z[i]);
  xm = block_all<true>(xm, red);
  xm = (cap > 0.0f ? cap * tanh_of(xm) : xm) * inv_tau;
  float xs = 0.0f;
  for (int i = threadIdx.x; i < V; i += kThreads) {
    const float x = (cap > 0.0f ? cap * tanh_of(z[i]) : z[i]) * inv_tau;
    xs += expf(x - xm);
  }
  xs = block_all<false>(xs, red);
  const float xlse = logf(xs);

  float loss = 0.0f;
  for (int k = threadIdx.x; k < K; k += kThreads) {
    const int i = i_s[k];
    const float lq = q_s[k] - tlse, q = any ? expf(lq) : 0.0f;
    if (q > 0.0f) {
      const float x = (cap > 0.0f ? cap * tanh_of(z[i]) : z[i]) * inv_tau;
      loss = fmaf(q, lq - ((x - xm) - xlse), loss);
    }
    q_s[k] = q;
  }
  loss = block_all<false>(loss, red);
  if (threadIdx.x == 0) p.loss[row] = any ? p.tau * p.tau * loss : 0.0f;

  if constexpr (DZ != 0) {
    const float w = any ? p.tau * (p.weight ? p.weight[row] : 1.0f) : 0.0f;
    const float inv = 1.0f / xs;
    auto grad = [&](float v, float q) {
      const float t = cap > 0.0f ? tanh_of(v) : 0.0f;
      const float x = (cap > 0.0f ? cap * t : v) * inv_tau;
      const float d = any ? (expf(x - xm) * inv - q) * w : 0.0f;
      return d * fmaf(-t, t, 1.0f);
    };
    auto store = [&](int i, float v) {
      if constexpr (DZ == 1) {
        static_cast<float*>(p.dz)[row * V + i] = v;
      } else {
        static_cast<uint16_t*>(p.dz)[row * V + i] = (uint16_t)Half<DZ == 3>::pack2(v, 0.0f);
      }
    };
    for (int i = threadIdx.x; i < V; i += kThreads) store(i, grad(z[i], 0.0f));
    __syncthreads();
    for (int k = threadIdx.x; k < K; k += kThreads) {
      const int i = i_s[k];
      if (i < 0) continue;
      float q = 0.0f;  // an index given more than once: its first entry stores for all
      bool first = true;
      for (int j = 0; j < K; ++j)
        if (i_s[j] == i) {
          first = first && j >= k;
          q += q_s[j];
        }
      if (first) store(i, grad(z[i], q));
    }
  }
}

}  // namespace

nc_status distill_topk_launch(const float* z, const int32_t* idx, const float* teacher, const float* weight,
                              float* loss, void* dz, int dz_kind, int M, int V, int K, float tau, float cap,
                              uint32_t* dev_status, cudaStream_t stream) {
  if (M == 0) return NC_OK;
  const DistillParams p{z, idx, teacher, weight, loss, dz, V, K, cap, tau, dev_status};
  const int smem = K * 8;
  switch (dz_kind) {
    case 0: distill_kernel<0><<<M, kThreads, smem, stream>>>(p); break;
    case 1: distill_kernel<1><<<M, kThreads, smem, stream>>>(p); break;
    case 2: distill_kernel<2><<<M, kThreads, smem, stream>>>(p); break;
    default: distill_kernel<3><<<M, kThreads, smem, stream>>>(p); break;
  }
  return cudaGetLastError() == cudaSuccess ? NC_OK : NC_ERR_CUDA;
}

}  // namespace nc
