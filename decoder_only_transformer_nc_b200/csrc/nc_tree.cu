// A tree of drafted tokens over the KV cache: ancestor masks, the attention of
// all its nodes in one pass, and the accepted path with its keys and values
// moved into the cache (speculative decoding over the cache of nc_decode.cu).
//
// Node i < N <= 128 of row b has the ancestor words mask[b][i]: bit j set where
// j is i itself or an ancestor of i.  depth_i = popcount - 1; the node sits at
// position p_i = len_b + depth_i, len_b being the committed positions of the
// row.  It attends over the committed keys t < len_b with p_i - t < window and
// over the drafted keys j of its mask words with depth_i - depth_j < window.
// A node whose own bit is clear is unused: its output is 0 and its drafted K/V
// are never read.
#include <cuda_runtime.h>

#include <cstdint>

#include "nc_half.cuh"
#include "nc_internal.h"
#include "nc_mma.cuh"

namespace nc {
namespace {

constexpr int kMaxNodes = kTreeMaxNodes;
constexpr int kMaxWords = kMaxNodes / 32;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// mask[b][i] = bit i | the words of i's parent, by walking up from i: a walk
// that leaves [0, i), or does not end at a root (-1), makes the node unused
// (all words 0).  One CTA a row, one thread a node.
__global__ void __launch_bounds__(kMaxNodes) tree_mask_kernel(const int32_t* __restrict__ parents,
                                                              uint32_t* __restrict__ mask, int N) {
  __shared__ int32_t par[kMaxNodes];
  const int b = blockIdx.x, i = threadIdx.x;
  if (i < N) par[i] = parents[(int64_t)b * N + i];
  __syncthreads();
  if (i >= N) return;
  uint32_t w[kMaxWords] = {};
  int at = i;
  while (at >= 0) {  // par[at] < at or the walk ends: at most N steps
#pragma unroll
    for (int k = 0; k < kMaxWords; ++k)
      if (k == (at >> 5)) w[k] |= 1u << (at & 31);
    const int up = par[at];
    at = up < at ? up : -2;
  }
  const int W = (N + 31) / 32;
#pragma unroll
  for (int k = 0; k < kMaxWords; ++k)
    if (k < W) mask[((int64_t)b * N + i) * W + k] = at == -1 ? w[k] : 0u;
}

// ---------------------------------------------------------------- attention
// Rows of one kv head: R = node * G + (query head in the group), so the heads
// that share K/V also share each K/V tile.  A CTA of four warps takes 16 * RW
// rows; its 4 / RW key-warps take each their own share of every 64-key tile and
// keep the running maximum and sum of their rows (fp32, log2 domain), which are
// merged at the end.  The tiles of one (row, kv head) -- committed keys from
// the window's first on, then the drafted ones -- are split over the CTAs of a
// cluster, which merge their partial results through distributed shared
// memory: one launch, no workspace, a fixed order of sums.
// K/V tiles arrive by 16-byte asynchronous copies, kStages deep.  What is left of
// its time is latency, not bytes: 8 us (in a graph) for 4 nodes over 300 positions of
// 10 heads of 128, whose K/V takes 0.24 us to read; 17 us for 16 rows of 27 nodes, 12
// heads of 64 and a window of 512, 27 MB or 4.2 us (tensor pipe 10 %, DRAM 16 %: three or
// four tiles a CTA, each of them waited for at a barrier).  The products
// run on m16n8k16 with fp32 accumulation; P enters P V in the 16-bit format of
// the inputs (half a step of each weight, relative; the row's sum keeps them in
// fp32), as in the attention kernels of the whole forward; in fp16, whose numbers end
// at 2^-24, times 2^15: the weights of a long cache may all be below that beside one
// large one.  (nc_decode_step's attention keeps its weights in fp32.)
constexpr int kTK = 64;      // keys per tile
constexpr int kStages = 3;   // tiles in flight
// fp16: weights (at most 1) times 2^15 stay under 65504.  bf16 has fp32's range, for the
// weights and for V, which may leave no room for a factor.
constexpr float lift(bool f16) { return f16 ? 15.0f : 0.0f; }

struct TreeAttnParams {
  const uint16_t* q;      // [B][N] rows of H heads, q_stride elements apart
  int64_t q_stride;
  const uint16_t* kv;     // [B][N][2][Hkv][D]
  const uint16_t* cache;  // [B][T_max][2][Hkv][D]
  const int32_t* lens;    // [B]
  const uint32_t* mask;   // [B][N][W]
  uint16_t* out;          // [B][N][H][D]
  int N, H, Hkv, T_max, window;  // window <= 0: none
  float scale_log2;
};

template <int D, bool F16, int RW>
__global__ void __launch_bounds__(128) tree_attn_kernel(const TreeAttnParams p) {
  using namespace wmma16;
  constexpr int KW = 4 / RW;         // key-warps
  constexpr int WK = kTK / KW;       // keys of a tile per warp
  constexpr int LD = D + 8;
  constexpr int NT = WK / 8;         // n8 tiles per warp
  constexpr int ROWS = 16 * RW;
  extern __shared__ __align__(16) uint16_t smem[];  // [kStages][K kTK x LD | V kTK x LD]
  __shared__ uint32_t mw[kMaxNodes * kMaxWords];
  __shared__ int depth_s[kMaxNodes];  // -1: unused

  const int CS = gridDim.x;
  const int rank = blockIdx.x;  // the cluster spans the grid's x
  const int g = blockIdx.y % p.Hkv, tile_r = blockIdx.y / p.Hkv, b = blockIdx.z;
  const int G = p.H / p.Hkv, N = p.N, W = (N + 31) / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rw = warp % RW, kw = warp / RW;

  for (int e = threadIdx.x; e < N * W; e += 128) mw[e] = p.mask[(int64_t)b * N * W + e];
  __syncthreads();
  for (int i = threadIdx.x; i < N; i += 128) {
    int c = 0;
    for (int k = 0; k < W; ++k) c += __popc(mw[i * W + k]);
    depth_s[i] = (mw[i * W + (i >> 5)] >> (i & 31)) & 1u ? c - 1 : -1;
  }
  __syncthreads();

  const int len = min(max(p.lens[b], 0), p.T_max);
  const int win = p.window > 0 ? p.window : 0x3fffffff;
  const int lo = max(0, len - win + 1);  // the root's first visible key: no node sees an earlier one
  const int nc = len - lo;               // committed keys, then N drafted ones
  const int nkeys = nc + N;
  const int ntiles = (nkeys + kTK - 1) / kTK;
  const int t_begin = (int)((int64_t)ntiles * rank / CS), t_end = (int)((int64_t)ntiles * (rank + 1) / CS);

  const int64_t pos_stride = 2 * (int64_t)p.Hkv * D;
  const uint16_t* cbase = p.cache + ((int64_t)b * p.T_max + lo) * pos_stride + (int64_t)g * D;
  const uint16_t* dbase = p.kv + (int64_t)b * N * pos_stride + (int64_t)g * D;
  auto issue = [&](int t) {
    uint16_t* st = smem + (t % kStages) * (2 * kTK * LD);
    constexpr int PARTS = 2 * D / 8;
    for (int e = threadIdx.x; e < kTK * PARTS; e += 128) {
      const int r = e / PARTS, part = e % PARTS;
      const int kv = part / (D / 8), off = (part % (D / 8)) * 8;
      const int v = t * kTK + r;
      const bool drafted = v >= nc;
      const bool ok = v < nkeys && (!drafted || depth_s[v - nc] >= 0);
      const uint16_t* src = (drafted ? dbase + (int64_t)(ok ? v - nc : 0) * pos_stride : cbase + (int64_t)v * pos_stride) +
                            (int64_t)kv * p.Hkv * D + off;
      cp_async16(st + (kv * kTK + r) * LD + off, src, ok);
    }
  };

  // this thread's two rows of the fragments
  const int row0 = tile_r * ROWS + rw * 16 + (lane >> 2);
  int node[2], dep[2], tmin[2];  // tmin: first visible virtual committed key
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int R = row0 + 8 * h;
    node[h] = R / G;
    dep[h] = node[h] < N ? depth_s[node[h]] : -1;
    tmin[h] = dep[h] < 0 ? 0x7fffffff : max(0, len + dep[h] - win + 1 - lo);
  }
  // Q fragments, straight from global memory (rows past the end: zeros)
  uint32_t qf[D / 16][4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int R = row0 + 8 * h;
    const bool ok = dep[h] >= 0;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(
        p.q + ((int64_t)b * N + (ok ? node[h] : 0)) * p.q_stride + (int64_t)(g * G + (ok ? R % G : 0)) * D);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      qf[k][h] = ok ? src[k * 8 + (lane & 3)] : 0u;
      qf[k][2 + h] = ok ? src[k * 8 + 4 + (lane & 3)] : 0u;
    }
  }
  float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
  for (int d = 0; d < D / 8; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[d][e] = 0.0f;

#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) {
    if (t_begin + i < t_end) issue(t_begin + i);
    cp_async_commit();
  }
  for (int t = t_begin; t < t_end; ++t) {
    cp_async_wait<kStages - 2>();
    __syncthreads();  // tile t has landed for every thread; tile t - 1's stage is free
    if (t + kStages - 1 < t_end) issue(t + kStages - 1);
    cp_async_commit();
    const uint32_t sk = smem_u32(smem + (t % kStages) * (2 * kTK * LD)), sv = sk + kTK * LD * 2;
    float s[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int n = 0; n < NT / 2; ++n) {
        uint32_t bf[4];
        load_b_nk<LD>(bf, sk, kw * WK + n * 16, k * 16, lane);
        mma16816<F16>(s[2 * n], qf[k], bf[0], bf[1]);
        mma16816<F16>(s[2 * n + 1], qf[k], bf[2], bf[3]);
      }
    // visibility: a tile of committed keys that every node sees needs no test
    const int v0 = t * kTK + kw * WK;
    const bool clean = v0 + WK <= nc && lo + v0 >= len + N - win;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x = s[n][e] * p.scale_log2;
        if (!clean) {
          const int h = e >> 1, v = v0 + n * 8 + (lane & 3) * 2 + (e & 1);
          bool see;
          if (v < nc) {
            see = v >= tmin[h];
          } else {
            const int j = v - nc;
            see = dep[h] >= 0 && j < N && ((mw[node[h] * W + (j >> 5)] >> (j & 31)) & 1u) && depth_s[j] >= 0 &&
                  dep[h] - depth_s[j] < win;
          }
          x = see ? x : -INFINITY;
        } else if (dep[e >> 1] < 0) {
          x = -INFINITY;
        }
        s[n][e] = x;
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float mx = m[h];
#pragma unroll
      for (int n = 0; n < NT; ++n) mx = fmaxf(mx, fmaxf(s[n][2 * h], s[n][2 * h + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float ms = mx == -INFINITY ? 0.0f : mx;  // nothing visible yet: every p is 0
      const float a = ex2(m[h] - ms), mp = ms - lift(F16);  // the sum and O carry the factor too
      float ps = 0.0f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        s[n][2 * h] = ex2(s[n][2 * h] - mp);
        s[n][2 * h + 1] = ex2(s[n][2 * h + 1] - mp);
        ps += s[n][2 * h] + s[n][2 * h + 1];
      }
      l[h] = fmaf(l[h], a, ps);
      m[h] = mx;
#pragma unroll
      for (int d = 0; d < D / 8; ++d) {
        o[d][2 * h] *= a;
        o[d][2 * h + 1] *= a;
      }
    }
#pragma unroll
    for (int n = 0; n < NT / 2; ++n) {
      uint32_t pf[4];
      pf[0] = Half<F16>::pack2(s[2 * n][0], s[2 * n][1]);
      pf[1] = Half<F16>::pack2(s[2 * n][2], s[2 * n][3]);
      pf[2] = Half<F16>::pack2(s[2 * n + 1][0], s[2 * n + 1][1]);
      pf[3] = Half<F16>::pack2(s[2 * n + 1][2], s[2 * n + 1][3]);
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        uint32_t bf[4];
        load_b_kn<LD>(bf, sv, kw * WK + n * 16, d * 16, lane);
        mma16816<F16>(o[2 * d], pf, bf[0], bf[1]);
        mma16816<F16>(o[2 * d + 1], pf, bf[2], bf[3]);
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();  // every tile is consumed: the stages hold the partial results now

  // partials: om [KW][ROWS][D] fp32, then (m, l) [KW][ROWS][2]
  constexpr int OLD = D + 4;
  float* om = reinterpret_cast<float*>(smem);
  float* ml = om + KW * ROWS * OLD;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = kw * ROWS + rw * 16 + (lane >> 2) + 8 * h;
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    if ((lane & 3) == 0) {
      ml[2 * r] = m[h];
      ml[2 * r + 1] = l[h];
    }
#pragma unroll
    for (int d = 0; d < D / 8; ++d)
      *reinterpret_cast<float2*>(om + r * OLD + d * 8 + (lane & 3) * 2) = make_float2(o[d][2 * h], o[d][2 * h + 1]);
  }
  if (CS > 1)
    cluster_sync();
  else
    __syncthreads();
  // the rows are dealt over the cluster; a row's D values over D / 4 threads
  const uint32_t om_u = smem_u32(om), ml_u = smem_u32(ml);
  const int live = min(ROWS, N * G - tile_r * ROWS);
  for (int e = threadIdx.x; e < (ROWS / CS + 1) * (D / 4); e += 128) {
    const int r = rank + (e / (D / 4)) * CS, d4 = e % (D / 4);
    if (r >= live) continue;
    float mm = -INFINITY;
    for (int c = 0; c < CS; ++c) {
      const uint32_t base = mapa_shared(ml_u, c);
#pragma unroll
      for (int k = 0; k < KW; ++k) mm = fmaxf(mm, ld_cluster_f32(base + (k * ROWS + r) * 8));
    }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float ll = 0.0f;
    if (mm != -INFINITY) {
      for (int c = 0; c < CS; ++c) {
        const uint32_t base = mapa_shared(ml_u, c), ob = mapa_shared(om_u, c);
#pragma unroll
        for (int k = 0; k < KW; ++k) {
          const float f = ex2(ld_cluster_f32(base + (k * ROWS + r) * 8) - mm);
          ll = fmaf(ld_cluster_f32(base + (k * ROWS + r) * 8 + 4), f, ll);
          const float4 v = ld_cluster_f32x4(ob + ((k * ROWS + r) * OLD + d4 * 4) * 4);
          acc.x = fmaf(v.x, f, acc.x);
          acc.y = fmaf(v.y, f, acc.y);
          acc.z = fmaf(v.z, f, acc.z);
          acc.w = fmaf(v.w, f, acc.w);
        }
      }
    }
    const float inv = mm != -INFINITY ? 1.0f / ll : 0.0f;
    const int R = tile_r * ROWS + r;
    uint16_t* dst = p.out + (((int64_t)b * N + R / G) * p.H + g * G + R % G) * D + d4 * 4;
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(Half<F16>::pack2(acc.x * inv, acc.y * inv), Half<F16>::pack2(acc.z * inv, acc.w * inv));
  }
  if (CS > 1) cluster_sync();  // no CTA leaves while another reads its partials
}

template <int D, bool F16, int RW>
nc_status tree_attn_run(const TreeAttnParams& p, int B, cudaStream_t stream) {
  constexpr int ROWS = 16 * RW;
  constexpr int smem = kStages * 2 * kTK * (D + 8) * 2;
  static_assert(smem >= 4 / RW * ROWS * (D + 4 + 2) * 4, "the partial results reuse the stages");
  auto* fn = tree_attn_kernel<D, F16, RW>;
  static bool attr_done[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !attr_done[dev]) {
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return NC_ERR_CUDA;
    if (dev < 64) attr_done[dev] = true;
  }
  const int G = p.H / p.Hkv;
  const int row_tiles = (p.N * G + ROWS - 1) / ROWS;
  const int base = row_tiles * p.Hkv * B;
  int keys = p.T_max;
  if (p.window > 0 && p.window - 1 < keys) keys = p.window - 1;
  const int tiles = (keys + p.N + kTK - 1) / kTK;
  // split the keys until the CTAs fill the device as often as their shared memory
  // lets them share an SM, down to one tile a CTA
  const int64_t slots = (int64_t)device_sm_count() * (227 * 1024 / (smem + 4096));
  int cs = 1;
  while (cs < 8 && cs * 2 <= tiles && (int64_t)base * cs * 2 <= slots) cs *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(cs, row_tiles * p.Hkv, B);
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = cs;
  at.val.clusterDim.y = 1;
  at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p) == cudaSuccess ? NC_OK : NC_ERR_CUDA;
}

template <int D, bool F16>
nc_status tree_attn_rows(const TreeAttnParams& p, int B, cudaStream_t stream) {
  const int rows = p.N * (p.H / p.Hkv);
  if (rows <= 16) return tree_attn_run<D, F16, 1>(p, B, stream);
  if (rows <= 32) return tree_attn_run<D, F16, 2>(p, B, stream);
  return tree_attn_run<D, F16, 4>(p, B, stream);
}

// ---------------------------------------------------------------- acceptance
// The accepted path of row b: the root (node 0), then from each accepted node
// its first child whose drafted token is the token sampled at that node.  Every
// CTA walks the path of its row by itself (a warp, up to four nodes a lane; a
// step is a compare and a ballot), so the copies of a layer wait for no other
// launch; the CTAs of layer 0 also write the path.  The walk and the launch are all
// there is to it: 3.4 us for a row of 8 nodes and 20 layers, 5.0 us for 32 rows of 64
// nodes and 26 layers, whose 17 MB take 2.6 us.
__global__ void __launch_bounds__(256) tree_accept_kernel(
    const int32_t* __restrict__ tokens, const int32_t* __restrict__ parents, const uint32_t* __restrict__ mask,
    const int32_t* __restrict__ sampled, const int32_t* __restrict__ lens, const uint4* __restrict__ kv,
    uint4* __restrict__ cache, int32_t* __restrict__ path, int32_t* __restrict__ count, int32_t* __restrict__ next,
    int32_t* __restrict__ lens_out, int32_t* __restrict__ hist, int B, int N, int L, int T_max, int width16) {
  __shared__ int32_t path_s[kMaxNodes];
  __shared__ int count_s;
  const int b = blockIdx.x, layer = blockIdx.y;
  const int len0 = lens[b];
  const int len = min(max(len0, 0), T_max);
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x, W = (N + 31) / 32;
    int32_t tok[kMaxWords], par[kMaxWords], smp[kMaxWords];
#pragma unroll
    for (int k = 0; k < kMaxWords; ++k) {
      const int j = k * 32 + lane;
      const int64_t at = (int64_t)b * N + j;
      // a node whose own bit is clear is unused
      const bool used = j < N && ((mask[at * W + k] >> lane) & 1u);
      tok[k] = j < N ? tokens[at] : 0;
      smp[k] = j < N ? sampled[at] : 0;
      par[k] = used ? parents[at] : -2;
    }
    const bool root = __shfl_sync(0xffffffffu, par[0] != -2, 0);
    const int32_t tok0 = __shfl_sync(0xffffffffu, tok[0], 0);
    int at = root ? 0 : -1, n = 0;
    int32_t nxt = tok0;
    while (at >= 0 && len + n < T_max) {  // indices grow along a path: at most N steps
      if (lane == 0) path_s[n] = at;
      ++n;
      int32_t s = 0;
#pragma unroll
      for (int k = 0; k < kMaxWords; ++k) {
        const int32_t v = __shfl_sync(0xffffffffu, smp[k], at & 31);
        if (k == (at >> 5)) s = v;
      }
      nxt = s;
      int child = -1;
#pragma unroll
      for (int k = kMaxWords - 1; k >= 0; --k) {
        const uint32_t hit = __ballot_sync(0xffffffffu, par[k] == at && tok[k] == s && k * 32 + lane > at);
        if (hit) child = k * 32 + __ffs(hit) - 1;
      }
      at = child;
    }
    if (lane == 0) {
      count_s = n;
      if (layer == 0) {
        count[b] = n;
        next[b] = nxt;
        lens_out[b] = len + n;
      }
    }
  }
  __syncthreads();
  const int n = count_s;
  if (layer == 0)
    for (int i = threadIdx.x; i < N; i += blockDim.x) {
      path[(int64_t)b * N + i] = i < n ? path_s[i] : -1;
      if (hist && i < n) hist[(int64_t)b * T_max + len + i] = tokens[(int64_t)b * N + path_s[i]];
    }
  if (layer >= L) return;
  const uint4* src = kv + ((int64_t)layer * B + b) * N * width16;
  uint4* dst = cache + (((int64_t)layer * B + b) * T_max + len) * width16;
  for (int e = threadIdx.x; e < n * width16; e += blockDim.x) {
    const int r = e / width16, c = e - r * width16;
    dst[e] = src[(int64_t)path_s[r] * width16 + c];
  }
}

// ---------------------------------------------------------------- the step's row kernels
// Depth of a node from its mask words; -1 if it is unused.
__device__ __forceinline__ int node_depth(const uint32_t* __restrict__ words, int i, int W) {
  int c = 0;
  for (int k = 0; k < W; ++k) c += __popc(words[k]);
  return (words[i >> 5] >> (i & 31)) & 1u ? c - 1 : -1;
}

// One warp a node; the smear gate's weight enters as bf16, as in the whole forward.
__global__ void __launch_bounds__(256) tree_embedding_kernel(
    const int32_t* __restrict__ tokens, const int32_t* __restrict__ parents, const uint32_t* __restrict__ mask,
    const int32_t* __restrict__ lens, const int32_t* __restrict__ hist, const float* __restrict__ wte,
    const float* __restrict__ gate, float* __restrict__ x, float* __restrict__ x0, int M, int N, int C, int V,
    int T_max, uint32_t* __restrict__ dev_status) {
  const int r = (int)(((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5);
  const int lane = threadIdx.x & 31;
  if (r >= M) return;
  const int b = r / N, i = r - b * N, W = (N + 31) / 32;
  const bool used = (mask[(int64_t)r * W + (i >> 5)] >> (i & 31)) & 1u;
  int tok = used ? tokens[r] : 0;
  if (tok < 0 || tok >= V) {
    if (lane == 0 && dev_status) atomicOr(dev_status, NC_DEV_TOKEN_RANGE);
    tok = 0;
  }
  const float4* e = reinterpret_cast<const float4*>(wte + (int64_t)tok * C);
  const float4* ep = e;
  const int n4 = C / 4;
  float sg = 0.0f;
  if (gate && used) {
    const int par = parents[r];  // in [-1, i) for a used node
    const int len = min(max(lens[b], 0), T_max);
    int ptok = -1;
    if (par >= 0)
      ptok = tokens[b * (int64_t)N + par];
    else if (len > 0)
      ptok = hist[(int64_t)b * T_max + len - 1];
    if (par >= 0 || len > 0) {
      if (ptok < 0 || ptok >= V) ptok = 0;
      ep = reinterpret_cast<const float4*>(wte + (int64_t)ptok * C);
      const float4* g4 = reinterpret_cast<const float4*>(gate);
      float dot = 0.0f;
      for (int c = lane; c < n4; c += 32) {
        const float4 a = e[c], g = g4[c];
        dot = fmaf(a.x, __bfloat162float(__float2bfloat16_rn(g.x)), dot);
        dot = fmaf(a.y, __bfloat162float(__float2bfloat16_rn(g.y)), dot);
        dot = fmaf(a.z, __bfloat162float(__float2bfloat16_rn(g.z)), dot);
        dot = fmaf(a.w, __bfloat162float(__float2bfloat16_rn(g.w)), dot);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      sg = 1.0f / (1.0f + expf(-dot));
    }
  }
  float4* dst = reinterpret_cast<float4*>(x + (int64_t)r * C);
  float4* dst0 = x0 ? reinterpret_cast<float4*>(x0 + (int64_t)r * C) : nullptr;
  for (int c = lane; c < n4; c += 32) {
    float4 a = e[c];
    if (sg != 0.0f) {
      const float4 p = ep[c];
      a.x = fmaf(sg, p.x, a.x);
      a.y = fmaf(sg, p.y, a.y);
      a.z = fmaf(sg, p.z, a.z);
      a.w = fmaf(sg, p.w, a.w);
    }
    dst[c] = a;
    if (dst0) dst0[c] = a;
  }
}

// As the finish of a decode step (nc_decode.cu), at each node's own position:
// columns 2i, 2i + 1 of a q or k head are the RoPE pair.  One warp per (node,
// head); lane l holds columns l * DW ...
template <int DW, bool F16>
__global__ void __launch_bounds__(256) tree_qkv_finish_kernel(
    const float* __restrict__ acc, const uint32_t* __restrict__ mask, const int32_t* __restrict__ lens,
    uint16_t* __restrict__ q, uint16_t* __restrict__ kv, const float* __restrict__ rope, int M, int N, int H, int Hkv,
    int T_max, float eps, uint32_t* __restrict__ dev_status, DecodeVe ve) {
  constexpr int D = DW * 32;
  const int heads = H + 2 * Hkv;
  const int64_t wid = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (wid >= (int64_t)M * heads) return;
  const int r = (int)(wid / heads), hd = (int)(wid - (int64_t)r * heads);
  const int b = r / N, W = (N + 31) / 32;
  const float* src = acc + wid * D + lane * DW;
  float v[DW];
#pragma unroll
  for (int d = 0; d < DW; ++d) v[d] = src[d];
  if (hd < H + Hkv) {
    const int depth = max(node_depth(mask + (int64_t)r * W, r - b * N, W), 0);
    const int pos = min(min(max(lens[b], 0), T_max) + depth, T_max - 1);  // past the cache: never accepted
    const float* cs = rope + (int64_t)pos * (D / 2);
    const float* sn = rope + ((int64_t)T_max + pos) * (D / 2);
    float ss = 0.0f;
#pragma unroll
    for (int p = 0; p < DW / 2; ++p) {
      const int i = lane * (DW / 2) + p;
      const float c = cs[i], sv = sn[i];
      const float a = v[2 * p], bb = v[2 * p + 1];
      v[2 * p] = a * c - bb * sv;
      v[2 * p + 1] = a * sv + bb * c;
      ss = fmaf(v[2 * p], v[2 * p], ss);
      ss = fmaf(v[2 * p + 1], v[2 * p + 1], ss);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float rs = rsqrtf(ss * (1.0f / D) + eps);
#pragma unroll
    for (int d = 0; d < DW; ++d) v[d] *= rs;
  } else if (ve.table) {
    const int g = hd - H - Hkv;
    int tok = ve.tokens[r];
    if (tok < 0 || tok >= ve.V) tok = 0;  // flagged by the embedding kernel
    const float* e = ve.table + ((int64_t)tok * Hkv + g) * D + lane * DW;
    const float gt = ve.gate[g];
#pragma unroll
    for (int d = 0; d < DW; ++d) v[d] = fmaf(gt, e[d], v[d]);
  }
  uint32_t pk[DW / 2];
  float vmax = 0.0f;
#pragma unroll
  for (int p = 0; p < DW / 2; ++p) {
    pk[p] = Half<F16>::pack2(v[2 * p], v[2 * p + 1]);
    vmax = fmaxf(vmax, fmaxf(fabsf(v[2 * p]), fabsf(v[2 * p + 1])));
  }
  if (F16 && dev_status && vmax > 65504.0f) atomicOr(dev_status, NC_DEV_F16_RANGE);
  uint16_t* dst = hd < H ? q + ((int64_t)r * H + hd) * D + lane * DW
                         : kv + ((int64_t)r * 2 * Hkv + (hd - H)) * D + lane * DW;
  if constexpr (DW == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pk[0], pk[1]);
  else
    *reinterpret_cast<uint32_t*>(dst) = pk[0];
}

}  // namespace

nc_status tree_embedding_launch(const int32_t* tokens, const int32_t* parents, const uint32_t* mask,
                                const int32_t* lens, const int32_t* hist, const float* wte, const float* smear_gate,
                                float* x, float* x0, int B, int N, int C, int V, int T_max, uint32_t* dev_status,
                                cudaStream_t stream) {
  const int M = B * N;
  if (M == 0) return NC_OK;
  if (C % 4 || (smear_gate && !hist)) return NC_ERR_SHAPE;
  tree_embedding_kernel<<<(unsigned)((M + 7) / 8), 256, 0, stream>>>(tokens, parents, mask, lens, hist, wte,
                                                                     smear_gate, x, x0, M, N, C, V, T_max, dev_status);
  return cudaGetLastError() == cudaSuccess ? NC_OK : NC_ERR_CUDA;
}

nc_status tree_qkv_finish_launch(const float* acc, const uint32_t* mask, const int32_t* lens, uint16_t* q,
                                 uint16_t* kv, const float* rope, int B, int N, int H, int Hkv, int D, int T_max,
                                 float eps, bool f16, uint32_t* dev_status, DecodeVe ve, cudaStream_t stream) {
  const int M = B * N;
  if (M == 0) return NC_OK;
  const unsigned grid = (unsigned)(((int64_t)M * (H + 2 * Hkv) + 7) / 8);
  auto go = [&](auto* fn) {
    fn<<<grid, 256, 0, stream>>>(acc, mask, lens, q, kv, rope, M, N, H, Hkv, T_max, eps, dev_status, ve);
  };
  if (D == 128)
    f16 ? go(tree_qkv_finish_kernel<4, true>) : go(tree_qkv_finish_kernel<4, false>);
  else
    f16 ? go(tree_qkv_finish_kernel<2, true>) : go(tree_qkv_finish_kernel<2, false>);
  return cudaGetLastError() == cudaSuccess ? NC_OK : NC_ERR_CUDA;
}

nc_status tree_mask_launch(const int32_t* parents, uint32_t* mask, int B, int N, cudaStream_t stream) {
  if (B == 0) return NC_OK;
  tree_mask_kernel<<<B, kMaxNodes, 0, stream>>>(parents, mask, N);
  return cudaGetLastError() == cudaSuccess ? NC_OK : NC_ERR_CUDA;
}

// Which kernel: the tcgen05 one starts later (about 10 us for next to nothing,
// this file's 7.5) and reads the keys faster, and a row tile costs it the same
// whether 4 or 128 of its rows are there.  Measured, us, this file's / tcgen05, at
// D = 128: 8 rows of the cache, 4 kv heads, 200 / 1000 / 4000 keys: 16 rows a kv
// head 9.1 / 14.8, 14.0 / 17.0, 27.0 / 23.4; 64 rows 12.6 / 15.0, 18.7 / 17.3,
// 41.6 / 23.9; 128 rows 14.8 / 15.7, 31.7 / 17.9, 73.4 / 25.3; 16 rows of the
// cache, 12 kv heads, 32 rows: 19.3 / 24.3, 55.6 / 35.4, 180 / 80.  The lengths
// are not known here; half of what the cache may hold stands for them.  What that
// costs: more than 32 rows over lengths that stay short, whatever T_max, take the
// tcgen05 kernel at 200 keys of 64 rows 14.5 / 15.4 (D = 128) and 11.3 / 14.5 (64),
// of 128 rows 15.0 / 16.1 and 11.5 / 14.9 (T_max 512 to 4096); the kernels meet at
// some 500 keys, for 64 rows of D = 64 between 1000 and 4000.
// The tcgen05 kernel is out where a CTA's plan would not hold the rows of the cache
// (more than 1024), a group has more than 128 heads or the window is 128 keys or less.
static bool use_tc(int B, int N, int H, int Hkv, int D, int T_max, int window) {
  const int rows = N * (H / Hkv);
  const int keys = window > 0 && window < T_max ? window : T_max;
  return (rows > 32 || (rows > 16 && keys >= 1536) || keys >= 4096 * 128 / D) &&
         tree_attention_tc_fits(B, N, H, Hkv, window);
}

size_t tree_attention_bytes(int B, int N, int H, int Hkv, int D, int T_max, int window) {
  return use_tc(B, N, H, Hkv, D, T_max, window) ? tree_attention_tc_bytes(D) : 0;
}

nc_status tree_attention_launch(const uint16_t* q, int64_t q_stride, const uint16_t* kv, const uint16_t* cache,
                                const int32_t* lens, const uint32_t* mask, uint16_t* out, int B, int N, int H,
                                int Hkv, int D, int T_max, int window, bool f16, void* workspace,
                                uint32_t* dev_status, cudaStream_t stream) {
  if (B == 0) return NC_OK;
  if (use_tc(B, N, H, Hkv, D, T_max, window))
    return tree_attention_tc_launch(q, q_stride, kv, cache, lens, mask, out, B, N, H, Hkv, D, T_max, window, f16,
                                    workspace, dev_status, stream);
  const TreeAttnParams p{q, q_stride, kv, cache, lens, mask, out, N, H, Hkv, T_max, window,
                         1.4426950408889634f / sqrtf((float)D)};
  if (D == 128) return f16 ? tree_attn_rows<128, true>(p, B, stream) : tree_attn_rows<128, false>(p, B, stream);
  return f16 ? tree_attn_rows<64, true>(p, B, stream) : tree_attn_rows<64, false>(p, B, stream);
}

nc_status tree_accept_launch(const int32_t* tokens, const int32_t* parents, const uint32_t* mask,
                             const int32_t* sampled, const int32_t* lens, const uint16_t* kv, uint16_t* cache,
                             int32_t* path, int32_t* count, int32_t* next, int32_t* lens_out, int32_t* hist, int B,
                             int N, int L, int T_max, int width, cudaStream_t stream) {
  if (B == 0) return NC_OK;
  tree_accept_kernel<<<dim3(B, L > 0 ? L : 1), 256, 0, stream>>>(
      tokens, parents, mask, sampled, lens, reinterpret_cast<const uint4*>(kv), reinterpret_cast<uint4*>(cache), path,
      count, next, lens_out, hist, B, N, L, T_max, width / 8);
  return cudaGetLastError() == cudaSuccess ? NC_OK : NC_ERR_CUDA;
}

}  // namespace nc
