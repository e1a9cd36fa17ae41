// Sampling a token a row from the logits with temperature, top-k, top-p and
// min-p, from given random numbers: the step between a decode step's logits and
// the next step's tokens.
//
//   w_i = exp((l_i - max l) / T)
//   order: logit descending, index ascending
//   keep the first top_k; of these the shortest prefix whose mass reaches top_p
//   of theirs (at least one); of these the ones with w_i >= min_p
//   token = the first kept index, in index order, whose running mass exceeds
//   u times the kept mass; logprob = log(w_token / kept mass)
//
// A token's index changes when a running sum is misplaced by one border, so the
// weights are computed in fp64 and summed as 64-bit integers in units of 2^-sh
// (sh = 62 less the bits of V, 51 at most: V weights of 1 do not overflow): integer sums do not
// depend on their order, so neither the split of a row over threads nor a race
// changes a result.  A weight below half a unit counts as 0.
#include <cuda_runtime.h>

#include <cstdint>

#include "nc_internal.h"

namespace nc {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

struct SampleParams {
  const float* logits;  // [M][ld]
  int64_t ld;
  const float* u;            // [M]
  const float* temperature;  // [M] or null (1)
  const int32_t* top_k;      // [M] or null (off)
  const float* top_p;        // [M] or null (off)
  const float* min_p;        // [M] or null (off)
  int32_t* tokens;           // [M]
  float* logprob;            // [M] or null
  int V, sh;
};

// Order-preserving map of a logit to 32 bits; -0 equals +0, NaN is below
// everything (key 0).
__device__ __forceinline__ uint32_t key_of(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float((key >> 31) ? (key & 0x7fffffffu) : ~key);
}

// exp((l - mx) / T) in units of 2^-sh, rounded to the nearest: 2^y with
// y = (l - mx) log2(e) / T split into the nearest integer and a remainder in
// [-1/2, 1/2], whose exponential is the Taylor series of e^(f ln 2) to the
// 11th power (remainder 7e-15).  c = log2(e) / T.  The row's maximum counts 1
// whatever it is (also +inf), -inf and NaN count 0.
__device__ __forceinline__ int64_t weight_of(float l, float mx, double c, int sh) {
  if (l == mx) return (int64_t)1 << sh;
  const double d = (double)l - (double)mx;
  const double y = d * c;
  if (!(y > -(double)(sh + 2))) return 0;  // NaN, -inf and what rounds to 0
  constexpr double kMagic = 6755399441055744.0;  // 1.5 2^52: adding it rounds to an integer
  const double t = y + kMagic;
  const int n = (int)__double2loint(t);
  const double f = y - (t - kMagic);
  // ln(2)^k / k!
  double r = 4.4455382718708116e-10 * f + 7.0549116208011233e-09;
  r = fma(r, f, 1.0178086009239699e-07);
  r = fma(r, f, 1.3215486790144309e-06);
  r = fma(r, f, 1.5252733804059840e-05);
  r = fma(r, f, 1.5403530393381609e-04);
  r = fma(r, f, 1.3333558146428443e-03);
  r = fma(r, f, 9.6181291076284772e-03);
  r = fma(r, f, 5.5504108664821580e-02);
  r = fma(r, f, 2.4022650695910071e-01);
  r = fma(r, f, 6.9314718055994531e-01);
  r = fma(r, f, 1.0);
  const double s = __hiloint2double(__double2hiint(r) + ((n + sh) << 20), __double2loint(r));  // r 2^(n + sh)
  return __double2ll_rn(s);
}

template <typename T, typename F>
__device__ __forceinline__ T block_reduce(T v, T* red, F f) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[threadIdx.x & 31];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

struct Add {
  __device__ int64_t operator()(int64_t a, int64_t b) const { return a + b; }
};
struct MaxU64 {
  __device__ uint64_t operator()(uint64_t a, uint64_t b) const { return a > b ? a : b; }
};

// One CTA a row; every warp owns a contiguous segment of the row for the steps
// that depend on the index order.
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleParams p) {
  __shared__ int64_t red[kWarps];
  __shared__ int64_t seg[kWarps];
  const int row = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float* x = p.logits + (int64_t)row * p.ld;
  const int V = p.V, sh = p.sh;

  // the largest logit, its lowest index
  uint64_t best = 0;
  for (int i = tid; i < V; i += kThreads) {
    const uint64_t e = ((uint64_t)key_of(x[i]) << 32) | (uint32_t)~i;
    best = e > best ? e : best;
  }
  best = block_reduce(best, reinterpret_cast<uint64_t*>(red), MaxU64{});
  const uint32_t kmax = (uint32_t)(best >> 32);
  const int arg = (int)~(uint32_t)best;
  if (kmax <= key_of(-INFINITY)) {  // nothing can be sampled: every logit is -inf or NaN
    if (tid == 0) {
      p.tokens[row] = -1;
      if (p.logprob) p.logprob[row] = -INFINITY;
    }
    return;
  }
  const float mx = value_of(kmax);
  const float T = p.temperature ? p.temperature[row] : 1.0f;
  if (!(T > 0.0f)) {  // greedy
    if (tid == 0) {
      p.tokens[row] = arg;
      if (p.logprob) p.logprob[row] = 0.0f;
    }
    return;
  }
  const double c = 1.4426950408889634 / (double)T;
  const int k = p.top_k ? p.top_k[row] : 0;
  const float tp = p.top_p ? p.top_p[row] : 1.0f;
  const float mp = p.min_p ? p.min_p[row] : 0.0f;
  // kept: key > cut, and of those with key == cut the first `ties` in index order
  uint32_t cut = 0;
  int64_t ties = V;
  if (k > 0 && k < V) {
    // the largest key with at least k elements at or above it
    uint32_t lo = 0, hi = kmax;
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo) / 2 + 1;
      int64_t n = 0;
      for (int i = tid; i < V; i += kThreads) n += key_of(x[i]) >= mid;
      n = block_reduce(n, red, Add{});
      if (n >= k)
        lo = mid;
      else
        hi = mid - 1;
    }
    cut = lo;
    int64_t above = 0;
    for (int i = tid; i < V; i += kThreads) above += key_of(x[i]) > cut;
    ties = k - block_reduce(above, red, Add{});
  }
  if (!(tp >= 1.0f)) {
    // mass of the first top_k; ties weigh the same
    int64_t z = 0;
    for (int i = tid; i < V; i += kThreads)
      if (key_of(x[i]) > cut) z += weight_of(x[i], mx, c, sh);
    z = block_reduce(z, red, Add{});
    int64_t nt = 0;
    for (int i = tid; i < V; i += kThreads) nt += key_of(x[i]) == cut;
    nt = block_reduce(nt, red, Add{});
    z += (nt < ties ? nt : ties) * weight_of(value_of(cut), mx, c, sh);
    const double want = (tp > 0.0f ? (double)tp : 0.0) * (double)z;
    // the smallest key whose predecessors (larger keys) have less than `want`
    uint32_t lo = cut, hi = kmax;
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo) / 2;
      int64_t s = 0;
      for (int i = tid; i < V; i += kThreads)
        if (key_of(x[i]) > mid) s += weight_of(x[i], mx, c, sh);
      s = block_reduce(s, red, Add{});
      if ((double)s < want)
        hi = mid;
      else
        lo = mid + 1;
    }
    // of its ties, those whose predecessors have less than `want`
    int64_t s = 0;
    for (int i = tid; i < V; i += kThreads)
      if (key_of(x[i]) > lo) s += weight_of(x[i], mx, c, sh);
    s = block_reduce(s, red, Add{});
    const int64_t w = weight_of(value_of(lo), mx, c, sh);
    int64_t r = V;
    if (w > 0) {
      const double q = ceil((want - (double)s) / (double)w);
      r = q < 1.0 ? 1 : (q > (double)V ? V : (int64_t)q);
    }
    ties = lo == cut ? (ties < r ? ties : r) : r;
    cut = lo;
  }
  // min-p: a weight below it is dropped
  const int64_t wmin = mp > 0.0f ? __double2ll_ru((double)fminf(mp, 1.0f) * (double)((int64_t)1 << sh)) : 0;

  // mass of every warp's segment
  const int per = (V + kWarps - 1) / kWarps, a0 = warp * per, a1 = min(V, a0 + per);
  int n = 0;
  for (int i = a0 + lane; i < a1; i += 32) n += key_of(x[i]) == cut;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  __syncthreads();
  if (lane == 0) seg[warp] = n;
  __syncthreads();
  int64_t tie0 = 0;  // ties before this warp's segment
  for (int w = 0; w < warp; ++w) tie0 += seg[w];
  // weight of element i (0 where not kept); seen: ties before this lane's element
  auto kept = [&](int i, int64_t& seen) -> int64_t {
    const bool in = i < a1;
    const float l = in ? x[i] : -INFINITY;
    const uint32_t key = in ? key_of(l) : 0u;
    const bool tie = in && key == cut;
    const uint32_t bal = __ballot_sync(0xffffffffu, tie);
    const int64_t before = seen + __popc(bal & ((1u << lane) - 1u));
    seen += __popc(bal);
    if (!in || !(key > cut || (tie && before < ties))) return 0;
    const int64_t w = weight_of(l, mx, c, sh);
    return w >= wmin ? w : 0;
  };
  int64_t mass = 0, seen = tie0;
  for (int i = a0; i < a1; i += 32) mass += kept(i + lane, seen);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, o);
  __syncthreads();
  if (lane == 0) seg[warp] = mass;
  __syncthreads();
  int64_t total = 0, before = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += seg[w];
    total += seg[w];
  }
  const float u = p.u[row];
  const double target = (u > 0.0f ? (double)u : 0.0) * (double)total;
  // u >= 1: the last kept token
  const bool last = target >= (double)total;
  const bool mine = last ? mass > 0 && before + mass == total
                         : (double)before <= target && (double)(before + mass) > target;
  if (!mine) return;  // one warp goes on
  int64_t run = before;
  seen = tie0;
  int pick = -1;
  for (int i = a0; i < a1; i += 32) {
    int64_t w = kept(i + lane, seen), cum = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t t = __shfl_up_sync(0xffffffffu, cum, o);
      if (lane >= o) cum += t;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, w > 0 && (last || (double)(run + cum) > target));
    if (hit) {
      pick = i + (last ? 31 - __clz(hit) : __ffs(hit) - 1);
      if (!last) break;
    }
    run += __shfl_sync(0xffffffffu, cum, 31);
  }
  if (lane == 0) {
    p.tokens[row] = pick;
    if (p.logprob) {
      const double z = log((double)total) - (double)sh * 0.6931471805599453;
      p.logprob[row] = (float)((x[pick] == mx ? 0.0 : ((double)x[pick] - (double)mx) / (double)T) - z);
    }
  }
}

}  // namespace

nc_status sample_launch(const float* logits, int64_t ld, const float* u, const float* temperature,
                        const int32_t* top_k, const float* top_p, const float* min_p, int32_t* tokens,
                        float* logprob, int M, int V, cudaStream_t stream) {
  if (M == 0) return NC_OK;
  int bits = 0;  // V <= 2^bits
  while (((int64_t)1 << bits) < V) ++bits;
  const int sh = 62 - bits < 51 ? 62 - bits : 51;
  const SampleParams p{logits, ld, u, temperature, top_k, top_p, min_p, tokens, logprob, V, sh};
  sample_kernel<<<M, kThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? NC_OK : NC_ERR_CUDA;
}

}  // namespace nc
