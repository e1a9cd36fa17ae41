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
// A token's index changes when a running sum is misplaced by one border.  The
// definition here is in integers: a weight is computed in fp64 and rounded to
// units of 2^-sh (sh = 62 less the bits of V, 51 at most: V weights of 1 do not
// overflow), and sums are exact whatever their order.  A row is first tried
// with fp32 weights, whose sums carry a bound of their error and of what rounding
// all V weights to units may change (V 2^-(sh + 1) of the mass: 1.2e-10 at V = 2^15,
// 1.9e-9 at 2^17, 1.2e-7 at 2^20): where no border (of top-p's share, of min-p, of the
// token's own interval) lies within it, the integers would give the same token; only
// else are they computed.
//
// What bounds it: up to some hundred rows, latency (passes of a row that end at a
// barrier, and code that is met for the first time: a row of 32768 logits, top-k 50
// and top-p 0.95, takes 14 us, 0.02 us of them at the copy rate); from there, the
// instructions of a pass.  1024 rows of 32749 logits, one pass: 58 us in a graph for
// 134 MB (2.3 TB/s, 35 % of a copy); two waves of four rows an SM, with the search of the token's
// segment behind each row.  The same with top-p 0.95, whose cut lies among thousands of
// tokens (a histogram and a pass more): 230 us, a row alone 36 us.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <type_traits>

#include "nc_internal.h"
#include "nc_ptx.cuh"

namespace nc {
namespace {

// Filters: a histogram of the logits (kBins equal bins from the maximum down)
// finds the bin where top-k cuts and a bracket of bins where top-p does; the
// tokens of those bins, at most one a thread, are sorted and cut exactly.
constexpr int kBins = 2048;

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
  int half;  // the histogram keeps a bin's mass as two sums of this many bits a token
};

// The share of the mass by which sums of units and of true weights may differ: half a
// unit a token, and 1e-9 for the fp64 sums and the integers' own exponential.
__device__ __forceinline__ double slack_of(const SampleParams& p) {
  return fma((double)p.V, __hiloint2double((1022 - p.sh) << 20, 0), 1e-9);
}

// Two units: by so much rounding a weight and min-p to units may part them.
__device__ __forceinline__ float two_units(const SampleParams& p) { return __int_as_float((128 - p.sh) << 23); }

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

// 2^(j / 32)
__constant__ double kExp2[32] = {
    1, 1.0218971486541166, 1.0442737824274138, 1.0671404006768237,
    1.0905077326652577, 1.1143867425958924, 1.1387886347566916, 1.1637248587775775,
    1.189207115002721, 1.215247359980469, 1.241857812073484, 1.2690509571917332,
    1.2968395546510096, 1.3252366431597413, 1.3542555469368927, 1.383909881963832,
    1.4142135623730951, 1.4451808069770467, 1.4768261459394993, 1.5091644275934228,
    1.5422108254079407, 1.5759808451078865, 1.6104903319492543, 1.6457554781539649,
    1.681792830507429, 1.7186192981224779, 1.7562521603732995, 1.7947090750031072,
    1.8340080864093424, 1.8741676341103, 1.9152065613971474, 1.9571441241754002};

// fp64 of an fp32 value, on the bits: the conversion instruction runs at a few
// values a cycle and bounded these passes.  Zero and subnormals come out below
// 2^-126 in size too, infinities and NaN as something finite.
__device__ __forceinline__ double wide(float x) {
  const int u = __float_as_int(x);
  return __hiloint2double(((u >> 3) & (int)0x8fffffffu) + (896 << 20), u << 29);
}

// The same of a weight, which is not negative.
__device__ __forceinline__ double wide_weight(float x) {
  const int u = __float_as_int(x);
  return __hiloint2double((u >> 3) + (896 << 20), u << 29);
}

// A sum of fp32 weights in fp64.  Four are added up first, unless one may be the
// maximum's (of weight `big` or more): what is beside it counts in full (the
// logprob of a token that is nearly certain).
struct Sum {
  double v = 0.0;
  __device__ __forceinline__ void add(float a, float b, float c, float d, float big = 1.0f) {
    const float x = (a + b) + (c + d);
    if (x < big)
      v += wide_weight(x);
    else
      v += (wide_weight(a) + wide_weight(b)) + (wide_weight(c) + wide_weight(d));
  }
};

// A row's exponential: exp((l - mx) / T) in units of 2^-sh, rounded to nearest.
// 2^y, y = (l - mx) log2(e) / T, in fp64: y = (32 n + j) / 32 + f with |f| <=
// 1/64, 2^f by the Taylor series of e^(f ln 2) to the 5th power (remainder
// 2.2e-15) times 2^(j/32).  The maximum counts 1 whatever it is (also +inf);
// -inf and NaN count 0.
struct Expo {
  float mx, c32, least;  // c32: log2(e) / T; y below `least` rounds to 0
  double mxd, c;
  int shx;               // sh << 20
  const double* tab;     // kExp2 in shared memory

  __device__ Expo(float mx_, double c_, int sh, const double* tab_)
      : mx(mx_), c32((float)c_), least(-(float)(sh + 1)), mxd(mx_ == INFINITY ? 0.0 : (double)mx_), c(c_),
        shx(sh << 20), tab(tab_) {}

  static constexpr int64_t kRaw0 = 0x4330000000000000ll;  // the bits of 2^52: what 0 looks like

  // The weight as the low bits of 2^52 + weight: sums of these are exact too.
  __device__ __forceinline__ int64_t raw(float l) const {
    const bool counts = l == mx || (l - mx) * c32 > least;
    const double d = l == mx ? 0.0 : wide(l) - mxd;
    constexpr double kMagic = 6755399441055744.0 / 32;  // 1.5 2^52 / 32: adding it rounds to 1/32
    const double t = fma(d, c, kMagic);
    const int nj = __double2loint(t);
    const double f = fma(d, c, kMagic - t);
    // ln(2)^k / k!
    double r = 1.3333558146428443e-03;
    r = fma(r, f, 9.618129107628477e-03);
    r = fma(r, f, 5.550410866482158e-02);
    r = fma(r, f, 2.402265069591007e-01);
    r = fma(r, f, 6.931471805599453e-01);
    r = fma(r, f, 1.0);
    r *= tab[nj & 31];
    // r 2^(n + sh) <= 2^51, rounded to an integer by adding 2^52
    const int hi = __double2hiint(r) + ((nj & ~31) << 15) + shx;
    return __double_as_longlong(__hiloint2double(counts ? hi : 0, __double2loint(r)) + 4503599627370496.0);
  }
  __device__ __forceinline__ int64_t operator()(float l) const { return raw(l) - kRaw0; }
};

// The same as an fp32 number (1 for the maximum).  l log2(e) / T = n + f, the
// remainder f from the unrounded product; less the maximum's own n and f (phi)
// it is y without the rounding of l - mx, which for far tokens is an error in
// proportion to |y|.  2^(f - phi) by the hardware, n into the exponent.
struct Expo32 {
  float least, c_hi, c_lo, m0, phi;
  // Relative error of a weight: 2^-22 (2^f) and ln 2 times that of f - phi, at most 4
  // roundings of 2^-25; and of a sum of four, two roundings.
  static constexpr double kErr = 4.5e-7;
  static constexpr float kMagic = 12582912.0f;  // 1.5 2^23: the nearest integer in the low bits

  __device__ Expo32(float mx, double c, float T) {
    c_hi = (float)c;
    c_lo = (float)(c - (double)c_hi);
    least = mx - 69.3f * T;  // below it a weight is 2^-100: nothing beside 1
    m0 = 2.0f * kMagic - fmaf(mx, c_hi, kMagic);
    const float t = fmaf(mx, c_hi, m0);
    phi = (t - kMagic) + fmaf(mx, c_lo, fmaf(mx, c_hi, m0 - t));
  }
  Expo32() = default;
  // Against 2^n0 (n0 an integer) instead of the maximum, for scaled().
  __device__ static Expo32 against(float n0, float mx, double c, float T) {
    Expo32 w;
    w.c_hi = (float)c;
    w.c_lo = (float)(c - (double)w.c_hi);
    w.least = mx - 69.3f * T;
    w.m0 = kMagic - n0;
    return w;
  }
  __device__ __forceinline__ float scaled(float l) const {
    l = fmaxf(l, least);
    const float t = fmaf(l, c_hi, m0);
    float w;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(fmaf(l, c_lo, fmaf(l, c_hi, m0 - t))));
    return __int_as_float(__float_as_int(w) + (__float_as_int(t) << 23));
  }
  __device__ static bool usable(float mx, float T) {
    return T > 1e-20f && T < 1e20f && fabsf(mx) < 1e5f * T;
  }
  __device__ __forceinline__ float operator()(float l) const {
    l = fmaxf(l, least);  // also -inf and NaN
    const float t = fmaf(l, c_hi, m0);
    float w;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(fmaf(l, c_lo, fmaf(l, c_hi, m0 - t)) - phi));
    return __int_as_float(__float_as_int(w) + (__float_as_int(t) << 23));
  }
  // The weight to 2.5e-9 in fp64: l log2(e) / T = n + j / 32 + g, |g| <= 1/64, with
  // 2^(j / 32) in fp64 and 2^g - 1, at most 0.011, in fp32 (Taylor to the 4th power, the
  // rest 1e-12; three roundings of 2^-24 of it, two of 2^-31 of g).
  static constexpr double kErrFine = 3e-9;
  __device__ __forceinline__ double fine(float l, float n0, const double* tab) const {
    l = fmaxf(l, least);
    const float m = fmaf(-32.0f, n0, kMagic);
    const float t = fmaf(l, 32.0f * c_hi, m);
    const float g = fmaf(l, c_lo, fmaf(l, c_hi, (m - t) * 0.03125f));
    const int k = __float_as_int(t) - __float_as_int(kMagic);
    // ln(2)^i / i!
    float e = fmaf(9.618129e-3f, g, 5.5504109e-2f);
    e = fmaf(e, g, 2.4022651e-1f);
    e = fmaf(e, g, 6.9314718e-1f) * g;
    double w = tab[k & 31];
    w = __hiloint2double(__double2hiint(w) + ((k & ~31) << 15), __double2loint(w));
    return fma(w, wide(e), w);
  }
  // What a - s z (a: a sum of some of the weights that z sums) may be off by: the
  // errors of a count 1 - s times, those of the others s times; and the units' rounding.
  __device__ static double off_by(double s, double a, double z, double slack, double err = kErr) {
    return err * ((1.0 - s) * a + s * fmax(z - a, 0.0)) + slack * z;
  }
};

// One row as its CTA walks it: from a 16-byte boundary at or before its start
// (position off is token 0), in a contiguous segment per warp, which passes that
// depend on the index order rely on.
struct Row {
  const float* base;
  int off, end;    // tokens are the positions [off, end)
  int seg0, seg1;  // this warp's
  int per;         // positions a segment, a multiple of 128
};

__device__ __forceinline__ float4 load4(const Row& r, int j) {
  if (j >= r.off && j + 4 <= r.end) return *reinterpret_cast<const float4*>(r.base + j);
  float4 v = make_float4(NAN, NAN, NAN, NAN);
  if (j >= r.off && j < r.end) v.x = r.base[j];
  if (j + 1 >= r.off && j + 1 < r.end) v.y = r.base[j + 1];
  if (j + 2 >= r.off && j + 2 < r.end) v.z = r.base[j + 2];
  if (j + 3 >= r.off && j + 3 < r.end) v.w = r.base[j + 3];
  return v;
}

// f(position, four logits) for the warp's positions, each lane four neighbours
// at a time; positions outside the row come as NaN.  U loads are in flight.
template <int U, typename F>
__device__ __forceinline__ void walk4(const Row& r, F f) {
  int j0 = r.seg0 + (threadIdx.x & 31) * 4;
  if constexpr (U == 1) {  // long f: one copy of its code, the next load on its way
    float4 v;
    if (j0 < r.seg1) v = load4(r, j0);
#pragma unroll 1
    for (; j0 < r.seg1; j0 += 128) {
      const float4 w = v;
      if (j0 + 128 < r.seg1) v = load4(r, j0 + 128);
      f(j0, w);
    }
  } else {
#pragma unroll 1
    for (; j0 < r.seg1; j0 += 128 * U) {
      float4 v[U];
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (j0 + k * 128 < r.seg1) v[k] = load4(r, j0 + k * 128);
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (j0 + k * 128 < r.seg1) f(j0 + k * 128, v[k]);
    }
  }
}

template <int U, typename F>
__device__ __forceinline__ void walk(const Row& r, F f) {
  walk4<U>(r, [&](int j, const float4& v) {
    f(j, v.x);
    f(j + 1, v.y);
    f(j + 2, v.z);
    f(j + 3, v.w);
  });
}

// f(position, logit) says whether a token is listed; every warp keeps the first
// kOwn of its own in its part of `own`, without an atomic (the same counter for
// all costs about a hundred cycles a token), and puts them into list[] at the end.
// Returns how many there are (list holds the first cap).  For the whole block.
template <int NT, int U, typename F>
__device__ __forceinline__ int collect(const Row& r, uint64_t* own, uint64_t* list, int cap, int* total, F f) {
  constexpr int kOwn = 64;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int n = 0;  // the warp's
  uint64_t* mine = own + warp * kOwn;
  __syncthreads();
  if (threadIdx.x == 0) *total = 0;
  __syncthreads();
#pragma unroll 1
  for (int j0 = r.seg0; j0 < r.seg1; j0 += 128 * U) {
    float4 v[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int j = j0 + k * 128 + lane * 4;
      v[k] = j < r.seg1 ? load4(r, j) : make_float4(NAN, NAN, NAN, NAN);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int j = j0 + k * 128 + lane * 4;
      const bool t0 = f(v[k].x), t1 = f(v[k].y), t2 = f(v[k].z), t3 = f(v[k].w);
      if (!__any_sync(0xffffffffu, t0 || t1 || t2 || t3)) continue;
      const float l[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
      const bool t[4] = {t0, t1, t2, t3};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t bal = __ballot_sync(0xffffffffu, t[e]);
        const int at = n + __popc(bal & ((1u << lane) - 1u));
        if (t[e]) {
          const uint64_t code = ((uint64_t)key_of(l[e]) << 32) | (uint32_t)~(j + e);
          if (at < kOwn) {
            mine[at] = code;
          } else {
            const int g = atomicAdd(total, 1);
            if (g < cap) list[g] = code;
          }
        }
        n += __popc(bal);
      }
    }
  }
  const int keep = min(n, kOwn);
  int base = 0;
  if (lane == 0) base = atomicAdd(total, keep);
  base = __shfl_sync(0xffffffffu, base, 0);
  __syncwarp();
  for (int i = lane; i < keep; i += 32)
    if (base + i < cap) list[base + i] = mine[i];
  __syncthreads();
  return *total;
}

// Order of the tokens: larger first (logit, then lower index).
__device__ __forceinline__ uint64_t code_of(float l, int pos) {
  return ((uint64_t)key_of(l) << 32) | (uint32_t)~pos;
}

constexpr int kStageBytes = 180 * 1024;  // a staged row and the list before it
constexpr int kTopBins = 256;  // histogram of the threads' maxima

template <int NT>
struct Smem {
  double tab[32], c, slack;  // c: log2(e) / T
  int64_t red[32];
  float redf[2][32];
  int64_t seg[32];
  union {
    struct {
      uint32_t cnt[kBins], lo[kBins], hi[kBins];  // tokens; mass in 2^-(2 half), as hi 2^half + lo
    } h;
    struct {
      uint64_t buf[2 * NT];
      int64_t mass[NT];
      float logit[NT];
    } s;
  };
  uint64_t cand[NT];
  uint64_t bar[NT / 32];
  int ncand, bk, cnt_bk, b1, b2, cnt_b1, cnt_b2, pick;
};

struct Add {
  template <typename T>
  __device__ T operator()(T a, T b) const {
    return a + b;
  }
};
struct MinF {
  __device__ float operator()(float a, float b) const { return fminf(a, b); }
};
struct Min {
  __device__ int operator()(int a, int b) const { return min(a, b); }
};

template <int NT, typename T, typename F>
__device__ __forceinline__ T block_reduce(T v, int64_t* red, F f, T none) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) reinterpret_cast<T*>(red)[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  v = lane < NT / 32 ? reinterpret_cast<T*>(red)[lane] : none;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <typename T>
__device__ __forceinline__ T warp_scan(T v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

// Inclusive sums of one 64-bit value a thread over the first `threads` threads.
template <int NT, typename T>
__device__ __forceinline__ T block_scan(T v, int64_t* red, int threads = NT) {
  static_assert(sizeof(T) == 8, "red holds 64-bit values");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T* rd = reinterpret_cast<T*>(red);
  if (threadIdx.x < threads) v = warp_scan(v);
  __syncthreads();
  if (lane == 31) rd[warp] = threadIdx.x < threads ? v : T(0);
  __syncthreads();
  if (warp == 0 || threadIdx.x >= threads) return v;
  const T w = warp_scan(lane < warp ? rd[lane] : T(0));
  return v + __shfl_sync(0xffffffffu, w, 31);
}

struct Filter {
  int k;    // 0: off
  float p;  // >= 1: off
};

// The code of the last token that top-k and top-p keep, for any row: bisection
// over the keys, a pass of the row each.  For rows whose cut falls among more tokens
// of one bin than the block has threads (heavy ties, logits spread over hundreds).
template <int NT>
__device__ __noinline__ uint64_t cut_by_bisection(const Row r, const Filter f, const Expo weight, Smem<NT>& sm) {
  const uint32_t kmax = key_of(weight.mx);
  uint32_t cut = 0;
  int64_t ties = INT_MAX;
  auto count_from = [&](uint32_t key) {  // tokens at or above it
    int64_t n = 0;
    walk<2>(r, [&](int, float l) { n += key_of(l) >= key; });
    return block_reduce<NT>(n, sm.red, Add{}, (int64_t)0);
  };
  auto mass_above = [&](uint32_t key) {
    int64_t z = 0;
    walk<2>(r, [&](int, float l) {
      if (key_of(l) > key) z += weight(l);
    });
    return block_reduce<NT>(z, sm.red, Add{}, (int64_t)0);
  };
  if (f.k > 0) {
    uint32_t lo = 1, hi = kmax;  // the largest key with at least k tokens from it on
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo) / 2 + 1;
      if (count_from(mid) >= f.k)
        lo = mid;
      else
        hi = mid - 1;
    }
    cut = lo;
    ties = f.k - count_from(cut + 1);
  }
  if (!(f.p >= 1.0f)) {
    int64_t z = mass_above(cut);
    if (cut > 0) {
      const int64_t nt = count_from(cut) - count_from(cut + 1);
      z += (nt < ties ? nt : ties) * weight(value_of(cut));
    }
    const double want = (f.p > 0.0f ? (double)f.p : 0.0) * (double)z;
    uint32_t lo = cut, hi = kmax;  // the smallest key with less than `want` above it
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo) / 2;
      if ((double)mass_above(mid) < want)
        hi = mid;
      else
        lo = mid + 1;
    }
    const int64_t w = weight(value_of(lo));
    int64_t n = INT_MAX;  // of its ties, those with less than `want` before them
    if (w > 0) {
      const double q = ceil((want - (double)mass_above(lo)) / (double)w);
      n = q < 1.0 ? 1 : (q > (double)INT_MAX ? INT_MAX : (int64_t)q);
    }
    ties = lo == cut ? (ties < n ? ties : n) : n;
    cut = lo;
  }
  // the index of the last kept tie
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int n = 0;
  walk<2>(r, [&](int, float l) { n += l == l && key_of(l) == cut; });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  __syncthreads();
  if (lane == 0) sm.seg[warp] = n;
  if (threadIdx.x == 0) sm.pick = -1;
  __syncthreads();
  int64_t before = 0;
  for (int w = 0; w < warp; ++w) before += sm.seg[w];
  if (before < ties && ties <= before + n) {
    int64_t seen = before;
    for (int j = r.seg0; j < r.seg1 && seen < ties; j += 32) {
      const int i = j + lane;
      const bool tie = i >= r.off && i < r.end && i < r.seg1 && r.base[i] == r.base[i] && key_of(r.base[i]) == cut;
      uint32_t bal = __ballot_sync(0xffffffffu, tie);
      const int here = __popc(bal);
      if (seen + here >= ties) {
        for (int64_t q = seen + 1; q < ties; ++q) bal &= bal - 1;
        if (lane == 0) sm.pick = j + __ffs(bal) - 1;
      }
      seen += here;
    }
  }
  __syncthreads();
  const int at = sm.pick;
  return at >= 0 ? ((uint64_t)cut << 32) | (uint32_t)~at : (uint64_t)cut << 32;
}

// Bitonic sort of one value a thread, largest first, over the first P threads
// (a power of two; the others only keep step); buf: 2 NT values.
template <int NT>
__device__ __forceinline__ uint64_t block_sort(uint64_t v, int P, uint64_t* buf) {
  const int tid = threadIdx.x;
  const bool in = (tid & ~31) < P;  // the warp takes part
  int flip = 0;
#pragma unroll 1
  for (int k = 2; k <= P; k <<= 1)
#pragma unroll 1
    for (int j = k >> 1; j > 0; j >>= 1) {
      uint64_t o = 0;
      if (j >= 32) {
        uint64_t* b = buf + flip * NT;
        flip ^= 1;
        if (in) b[tid] = v;
        __syncthreads();
        if (in) o = b[tid ^ j];
      } else if (in) {
        o = __shfl_xor_sync(0xffffffffu, v, j);
      }
      const bool big = ((tid & j) == 0) == ((tid & k) == 0);
      v = (v > o) == big ? v : o;
    }
  return v;
}

__device__ __forceinline__ int pow2_from(int n) { return n <= 1 ? 1 : 1 << (32 - __clz(n - 1)); }

// The last steps where the n <= NT candidates (sm.cand) are known to hold every
// kept token: sorted by likelihood, cut, sorted by index, and the running mass
// tells the token.  k: how many top-k leaves.  Without top-k the mass that top-p
// is a share of is known to lie in [z_lo, z_hi]; false if that does not settle
// the cut.  Called by the whole block.
template <int NT>
__device__ __noinline__ bool pick_from_list(int n, int k, float tp, int64_t z_lo, int64_t z_hi, int64_t wmin, float u,
                                            const Expo weight, float T, Smem<NT>& sm, const SampleParams& p, int row,
                                            int off) {
  const int tid = threadIdx.x;
  const bool use_p = !(tp >= 1.0f);
  const int P = pow2_from(n);
  const uint64_t code = block_sort<NT>(tid < n ? sm.cand[tid] : 0ull, P, sm.s.buf);
  const float l = value_of((uint32_t)(code >> 32));
  int64_t w = tid < n ? weight(l) : 0;
  int64_t cum = block_scan<NT>(w, sm.red, (P + 31) & ~31);
  if (k < n) n = k;
  if (use_p && z_lo < 0) {  // top-k's mass
    if (tid == n - 1) sm.seg[0] = cum;
    __syncthreads();
    z_lo = z_hi = sm.seg[0];
  }
  const double pp = tp > 0.0f ? (double)tp : 0.0, b = (double)(cum - w);
  // top-p and min-p keep a first part of the order as well
  bool keep = tid < n && w >= wmin;
  if (use_p) {
    const bool open = (keep && tid > 0 && b >= pp * (double)z_lo && b < pp * (double)z_hi) ||
                      (tid == n - 1 && (double)cum < pp * (double)z_hi);  // the cut may lie past the list
    if (__syncthreads_or(open)) return false;
    keep = keep && (tid == 0 || b < pp * (double)z_lo);
  }
  n = __syncthreads_count(keep);
  if (tid == n - 1) sm.seg[0] = cum;  // the kept mass
  if (tid < n) {
    sm.s.mass[tid] = w;
    sm.s.logit[tid] = l;
  }
  // by index: ~position is in the code's low word, so largest first is index order
  const int Q = pow2_from(n);
  const uint64_t by_pos = block_sort<NT>(tid < n ? (code << 32) | (uint32_t)tid : 0ull, Q, sm.s.buf);
  __syncthreads();
  const int64_t total = sm.seg[0];
  const int rank = (int)(uint32_t)by_pos;
  w = tid < n ? sm.s.mass[rank] : 0;
  cum = block_scan<NT>(w, sm.red, (Q + 31) & ~31);
  const double target = (u > 0.0f ? (double)u : 0.0) * (double)total;
  const bool last = target >= (double)total;  // u >= 1: the last kept token
  if (tid < n && w > 0 && (last ? cum == total : (double)cum > target && (double)(cum - w) <= target)) {
    p.tokens[row] = (int)~(uint32_t)(by_pos >> 32) - off;
    if (p.logprob) {
      const float lt = sm.s.logit[rank];
      const double z = log((double)total) - (double)p.sh * 0.6931471805599453;
      p.logprob[row] = (float)((lt == weight.mx ? 0.0 : ((double)lt - (double)weight.mx) / (double)T) - z);
    }
  }
  return true;
}

// The row's token where the tokens from `least` on, at most kPart in a warp's
// segment, hold every kept one: one pass
// lists them in index order and sums the others' mass; the rest happens in
// registers, kPer tokens a thread with integer weights.  The cuts are bisections
// over the keys.  Only the others' mass is fp32 and in no units; false where its error leaves
// top-p's cut open, or where a cut lies past the list.  For the whole block.
constexpr int kPart = 256, kPer = kPart / 32;
template <int NT>
__device__ __noinline__ bool pick_from_top(const Row r, int k, float tp, float mp, float u, float T, float least, const Expo we,
                                           uint64_t* list, Smem<NT>& sm, const SampleParams& p, int row) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool use_p = !(tp >= 1.0f);
  const Expo32 wf(we.mx, we.c, T);
  uint64_t* mine = list + warp * kPart;
  int n = 0;
  Sum tail;
#pragma unroll 1
  for (int j0 = r.seg0; j0 < r.seg1; j0 += 128) {
    const int j = j0 + lane * 4;
    const float4 v = j < r.seg1 ? load4(r, j) : make_float4(NAN, NAN, NAN, NAN);
    const float l[4] = {v.x, v.y, v.z, v.w};
    uint32_t bal[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) bal[e] = __ballot_sync(0xffffffffu, l[e] >= least);
    if (use_p && k <= 0) {
      float w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w[e] = wf(l[e]);
        w[e] = l[e] >= least ? 0.0f : w[e];
      }
      tail.add(w[0], w[1], w[2], w[3]);
    }
    if (bal[0] | bal[1] | bal[2] | bal[3]) {  // of the 128, a lane's four are neighbours
      const uint32_t lt = (1u << lane) - 1u;
      int at = n + __popc(bal[0] & lt) + __popc(bal[1] & lt) + __popc(bal[2] & lt) + __popc(bal[3] & lt);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (l[e] >= least) {
          if (at < kPart) mine[at] = code_of(l[e], j + e);
          ++at;
        }
      n += __popc(bal[0]) + __popc(bal[1]) + __popc(bal[2]) + __popc(bal[3]);
    }
  }
  if (__syncthreads_or(n > kPart)) return false;
  uint32_t key[kPer];
  int64_t w[kPer], sum = 0;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int i = lane * kPer + e;
    key[e] = i < n ? (uint32_t)(mine[i] >> 32) : 0u;
    w[e] = i < n ? we(value_of(key[e])) : 0;
    sum += w[e];
  }
  const uint32_t kmax = key_of(we.mx), kmin = key_of(least);
  auto count_from = [&](uint32_t from) {
    int c = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) c += key[e] >= from;
    return block_reduce<NT>(c, sm.red, Add{}, 0);
  };
  auto mass_above = [&](uint32_t at) {
    int64_t c = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) c += key[e] > at ? w[e] : 0;
    return block_reduce<NT>(c, sm.red, Add{}, (int64_t)0);
  };
  // kept: key > cut, and of those with key == cut the first `ties` in index order
  uint32_t cut = 0;
  int ties = INT_MAX;
  if (k > 0) {
    if (count_from(1u) < k) return false;
    uint32_t lo = kmin, hi = kmax;  // the largest key with at least k tokens from it on
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo) / 2 + 1;
      if (count_from(mid) >= k)
        lo = mid;
      else
        hi = mid - 1;
    }
    cut = lo;
    ties = k - count_from(cut + 1);
  }
  if (use_p) {
    const double unit = (double)((int64_t)1 << p.sh), pp = tp > 0.0f ? (double)tp : 0.0;
    double z_lo, z_hi, within;
    if (k > 0) {
      z_lo = z_hi = within = (double)(mass_above(cut) + (int64_t)ties * we(value_of(cut)));
    } else {
      within = (double)block_reduce<NT>(sum, sm.red, Add{}, (int64_t)0);
      const double t = block_reduce<NT>(tail.v, sm.red, Add{}, 0.0) * unit;
      // the fp32 weights' error, and what rounding every one of them to a unit may change
      const double err = Expo32::kErr * t + (double)p.V;
      z_lo = within + t - err;
      z_hi = within + t + err;
    }
    const double want_lo = pp * z_lo, want_hi = pp * z_hi;
    if (k <= 0 && !(within >= want_hi)) return false;  // the cut lies past the list
    uint32_t lo = max(cut, kmin), hi = kmax;  // the smallest key with less than what is wanted above it
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo) / 2;
      const double s = (double)mass_above(mid);
      if (s < want_lo)
        hi = mid;
      else if (s >= want_hi)
        lo = mid + 1;
      else
        return false;
    }
    const double s = (double)mass_above(lo), wt = (double)we(value_of(lo));
    int m = INT_MAX;  // of its ties, those with less before them
    if (wt > 0.0) {
      const double a = ceil((want_lo - s) / wt), b = ceil((want_hi - s) / wt);
      if (a != b) return false;
      m = a < 1.0 ? 1 : (int)fmin(a, 2147483647.0);
    }
    ties = lo == cut ? min(ties, m) : m;
    cut = lo;
  }
  const int64_t wmin = mp > 0.0f ? __double2ll_ru((double)fminf(mp, 1.0f) * (double)((int64_t)1 << p.sh)) : 0;
  int mt = 0;
#pragma unroll
  for (int e = 0; e < kPer; ++e) mt += key[e] == cut && cut != 0u;
  int64_t seen = block_scan<NT>((int64_t)mt, sm.red) - mt;
  sum = 0;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const bool tie = key[e] == cut;
    const bool keep = key[e] > cut || (tie && seen < ties);
    seen += tie;
    if (!keep || w[e] < wmin) w[e] = 0;
    sum += w[e];
  }
  const int64_t inc = block_scan<NT>(sum, sm.red);
  if (tid == NT - 1) sm.seg[0] = inc;
  __syncthreads();
  const int64_t total = sm.seg[0];
  const double target = (u > 0.0f ? (double)u : 0.0) * (double)total;
  const bool last = target >= (double)total;  // u >= 1: the last kept token
  if (sum > 0 && (last ? inc == total : (double)inc > target && (double)(inc - sum) <= target)) {
    int64_t run = inc - sum;
    int pick = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      if (w[e] > 0 && (last || (double)run <= target)) pick = e;
      run += w[e];
    }
    const uint64_t code = mine[lane * kPer + pick];
    p.tokens[row] = (int)~(uint32_t)code - r.off;
    if (p.logprob) {
      const float l = value_of((uint32_t)(code >> 32));
      const double z = log((double)total) - (double)p.sh * 0.6931471805599453;
      p.logprob[row] = (float)((l == we.mx ? 0.0 : ((double)l - (double)we.mx) / (double)T) - z);
    }
  }
  return true;
}

// The token among the kept ones: the segment (sm.seg: every warp's kept mass) whose
// part of the running mass holds u times the total, each warp's share of that
// segment, and the position.  kept(position, logit): a token's mass.  EXACT: the
// masses are integers; else fp32 weights, and the token is only named where the
// errors leave its borders clear of the target.  The position in every lane of
// the warp that finds it, -1 in the others.  For the whole block.
template <int NT, bool EXACT, typename A, typename F>
__device__ __forceinline__ int locate(const Row& r, Smem<NT>& sm, float u, A& total, F kept,
                                      double err = Expo32::kErr) {
  constexpr int NW = NT / 32, U = EXACT ? 2 : 8;  // loads in flight
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const A sv = lane < NW ? *reinterpret_cast<const A*>(&sm.seg[lane]) : A(0), sc = warp_scan(sv);
  total = __shfl_sync(0xffffffffu, sc, 31);
  const double z = (double)total, target = (u > 0.0f ? (double)u : 0.0) * z;
  const bool last = EXACT && target >= z;  // u >= 1: the last kept token
  const uint32_t has = __ballot_sync(0xffffffffu, sv > A(0) && (last || (double)sc > target));
  if (!EXACT && !has) return -1;
  const int s = last ? 31 - __clz(has) : __ffs(has) - 1;
  const A before = __shfl_sync(0xffffffffu, sc - sv, s);
  const int sub = (r.per + NT - 1) / NT * 32;  // positions a warp
  const int s0 = s * r.per + warp * sub, s1 = min(min(s0 + sub, (s + 1) * r.per), r.end);
  float l[U];
  auto load = [&](int j) {
#pragma unroll
    for (int e = 0; e < U; ++e) {
      const int i = j + e * 32 + lane;
      l[e] = i >= r.off && i < s1 ? r.base[i] : NAN;
    }
  };
  A part = 0;
#pragma unroll 1
  for (int j = s0; j < s1; j += 32 * U) {
    load(j);
#pragma unroll
    for (int e = 0; e < U; ++e) part += kept(j + e * 32 + lane, l[e]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
  __syncthreads();
  if (lane == 0) *reinterpret_cast<A*>(&sm.seg[warp]) = part;
  __syncthreads();
  const A pv = lane < NW ? *reinterpret_cast<const A*>(&sm.seg[lane]) : A(0), pc = warp_scan(pv);
  const uint32_t at = __ballot_sync(0xffffffffu, pv > A(0) && (last || (double)(before + pc) > target));
  const int owner = at ? (last ? 31 - __clz(at) : __ffs(at) - 1) : -1;
  if (warp != owner) return -1;
  A run = before + __shfl_sync(0xffffffffu, pc - pv, warp);
  int pick = -1;
  bool found = false;
#pragma unroll 1
  for (int j = s0; j < s1 && (last || !found); j += 32 * U) {
    load(j);
#pragma unroll
    for (int e = 0; e < U; ++e) {
      const A w = kept(j + e * 32 + lane, l[e]), cum = warp_scan(w);
      const uint32_t hit = __ballot_sync(0xffffffffu, w > A(0) && (last || (double)(run + cum) > target));
      if (hit && (last || !found)) {
        const int h = last ? 31 - __clz(hit) : __ffs(hit) - 1;
        found = true;
        pick = j + e * 32 + h;
        if (!EXACT) {
          // the token's borders; the first token's lower and the last one's upper are certain
          const double up = (double)__shfl_sync(0xffffffffu, run + cum, h),
                       down = (double)__shfl_sync(0xffffffffu, run + cum - w, h);
          const double v = fmin(fmax((double)u, 0.0), 1.0);
          const double slack = sm.slack;
          if (!(up - target > Expo32::off_by(v, up, z, slack, err)) ||
              !(target - down > Expo32::off_by(v, down, z, slack, err)))
            pick = -1;
        }
      }
      run += __shfl_sync(0xffffffffu, cum, 31);
    }
  }
  return pick;
}

// The token where there is no filter: the logits are read once.  The weights are
// counted against a power of two 2^12 (kRoom) or more above the largest of the first
// tokens of every segment; should one of the rest be above that, the sums are not
// valid and the answer is -1.  0 where the fp32 errors leave the token open (a row in
// a hundred at 32768 tokens); FINE: for those, with fp64 weights.  Else 1.  For the
// whole block.
template <int NT, bool FINE>
__device__ __noinline__ int pick_plain(const Row r, float u, float T, double c, Smem<NT>& sm, const SampleParams& p,
                                        int row) {
  constexpr int NW = NT / 32, U = 4, kRoom = 12;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float4 v[U];
  const int j0 = r.seg0 + lane * 4;
  auto load = [&](int j) {
#pragma unroll
    for (int e = 0; e < U; ++e)
      v[e] = j + e * 128 < r.seg1 ? load4(r, j + e * 128) : make_float4(NAN, NAN, NAN, NAN);
  };
  load(j0);
  float mx = -INFINITY;
  auto upto = [&](const float4& x) { mx = fmaxf(mx, fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w))); };  // ignores NaN
#pragma unroll
  for (int e = 0; e < U; ++e) upto(v[e]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (lane == 0) sm.redf[0][warp] = mx;
  __syncthreads();
  mx = lane < NW ? sm.redf[0][lane] : -INFINITY;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (!(mx > -INFINITY) || !Expo32::usable(mx, T)) return -1;
  const float n0 = ceilf(mx * (float)c) + (float)kRoom;
  const Expo32 wf = Expo32::against(n0, mx, c, T);
  constexpr float kBig = 1.0f / (1 << (kRoom + 2));  // the maximum's weight is more
  auto weight = [&](float l) -> double {
    if constexpr (FINE)
      return wf.fine(l, n0, sm.tab);
    else
      return wide_weight(wf.scaled(l));
  };
  Sum sum;
#pragma unroll 1
  for (int j = j0; j - lane * 4 < r.seg1;) {
    float4 x[U];
#pragma unroll
    for (int e = 0; e < U; ++e) x[e] = v[e];
    j += 128 * U;
    if (j - lane * 4 < r.seg1) load(j);
#pragma unroll
    for (int e = 0; e < U; ++e) {
      upto(x[e]);
      if constexpr (FINE)
        sum.v += (weight(x[e].x) + weight(x[e].y)) + (weight(x[e].z) + weight(x[e].w));
      else
        sum.add(wf.scaled(x[e].x), wf.scaled(x[e].y), wf.scaled(x[e].z), wf.scaled(x[e].w), kBig);
    }
  }
  double mass = sum.v;
  const bool above = mx * (float)c > n0;  // a weight above 1 (its bits may be anything)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mass += __shfl_xor_sync(0xffffffffu, mass, o);
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  __syncthreads();
  if (lane == 0) {
    *reinterpret_cast<double*>(&sm.seg[warp]) = mass;
    sm.redf[0][warp] = mx;
  }
  if (__syncthreads_or(above)) return -1;
  double total;
  const int pick = locate<NT, false>(
      r, sm, u, total, [&](int, float l) { return l > -INFINITY ? weight(l) : 0.0; },
      FINE ? Expo32::kErrFine : Expo32::kErr);
  if (lane == 0 && pick >= 0) {
    p.tokens[row] = pick - r.off;
    if (p.logprob) {
      // the token's weight and the largest enter in full: a token that is nearly certain
      // has a logprob as exact as what is beside it
      for (int w = 0; w < NW; ++w) mx = fmaxf(mx, sm.redf[0][w]);
      const float l = r.base[pick];
      const double y = fma((double)l, c, -(double)n0), w = exp2(y);
      total += w - weight(l);
      if (l != mx) total += exp2(fma((double)mx, c, -(double)n0)) - weight(mx);
      p.logprob[row] = (float)-log(total / w);
    }
  }
  return __syncthreads_or(pick >= 0) ? 1 : 0;
}

// What the histogram found out.
struct Cut {
  bool bins, use_k, use_p;
  float mx, scale;
  int k, b1, b2, bk;  // top-k's bin; the bracket of top-p's (without it: bk twice)
  int n1, cnt_above, cnt_bk;  // tokens in the bracket, before it, before bk
  bool fits;  // the tokens of the bracket and of bk can be sorted
  double z;  // the sum of all tokens' fp32 weights (top-p alone)

  // Rounded to the nearest bin: never falls where l falls, which is all that is
  // asked of it; a float, so comparing needs no conversion.  Not clamped to the
  // last bin, kFar; NaN stays NaN.
  static constexpr float kOne = 8388608.0f;  // 2^23: the sum's last bit is 1
  static constexpr float kFar = kOne + (float)(kBins - 1);
  __device__ __forceinline__ float fbin(float l) const { return fmaf(mx - l, scale, kOne); }
};

// The row's token from its bracket: a pass that sums every segment's sure tokens
// and lists the bracket's, the cut in the list, then the segment, the warp's
// share of it and the token.  EXACT: integer weights (and, if the bracket fails,
// the bisection); else fp32 ones, false where their error leaves it open.
template <int NT, bool EXACT>
__device__ __noinline__ bool pick_from_row(const Row r, const Cut q, float tp, float mp, float u, float T,
                                           const Expo we, Smem<NT>& sm, const SampleParams& p, int row) {
  using A = typename std::conditional<EXACT, int64_t, double>::type;
  constexpr int NW = NT / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Expo32 wf(q.mx, we.c, T);
  A wmin = 0;
  if (mp > 0.0f)
    wmin = EXACT ? (A)__double2ll_ru((double)fminf(mp, 1.0f) * (double)((int64_t)1 << p.sh)) : (A)fminf(mp, 1.0f);
  const bool use_m = mp > 0.0f;
  bool open = false;  // fp32: a weight too near min-p's border
  const float near = (float)wmin * 1e-5f + two_units(p);
  auto weight = [&](float l) -> A {
    if constexpr (EXACT) {
      return we(l);
    } else {
      return wide_weight(wf(l));
    }
  };
  // a bin as a bound of fbin: with top-k the last one took in all beyond it
  auto upto = [&](int b) { return q.use_k && b >= kBins - 1 ? INFINITY : Cut::kOne + (float)b; };
  const float f1 = Cut::kOne + (float)q.b1, f2 = upto(q.b2), fk = Cut::kOne + (float)q.bk, fk2 = upto(q.bk);
  auto listed = [&](float l, float b) {
    return l > -INFINITY && ((b >= f1 && b <= f2) || (q.use_k && b >= fk && b <= fk2));
  };
  if (tid == 0) sm.ncand = 0;
  __syncthreads();
  bool good = q.fits;
  A za = 0, zt = 0, mass = 0;  // before the bracket; all that top-p's share is of; kept of the segment
  Sum as, ts, ms;
  if (good) {
    if constexpr (EXACT) {
      uint64_t sum = 0;  // modulo 2^64 until the 2^52 of every position is taken off
      if (!q.bins && !use_m) {
        walk<1>(r, [&](int, float l) { sum += (uint64_t)we.raw(l); });
        const int lane0 = r.seg0 + lane * 4;
        sum -= (uint64_t)(lane0 < r.seg1 ? (r.seg1 - lane0 + 127) / 128 * 4 : 0) * (uint64_t)Expo::kRaw0;
        mass = (A)sum;
      } else {
        const float f_rest = q.use_k ? fk : INFINITY;  // top-p's mass ends before it
        walk<1>(r, [&](int j, float l) {
          const int64_t w = we(l);
          if (!q.bins) {
            mass += w >= wmin ? w : 0;
            return;
          }
          const float b = q.fbin(l);
          if (b < f1) {
            za += w;
            if (use_m) mass += w >= wmin ? w : 0;
          } else if (listed(l, b)) {
            sm.cand[atomicAdd(&sm.ncand, 1)] = code_of(l, j);
          } else if (b < f_rest) {
            zt += w;
          }
        });
        zt += za;
        if (q.bins && !use_m) mass = za;
      }
    } else if (!q.bins) {
      walk4<1>(r, [&](int, const float4& v) {
        float w0 = wf(v.x), w1 = wf(v.y), w2 = wf(v.z), w3 = wf(v.w);
        if (use_m) {
          const float m = (float)wmin;
          open = open || fabsf(w0 - m) <= near || fabsf(w1 - m) <= near || fabsf(w2 - m) <= near ||
                 fabsf(w3 - m) <= near;
          w0 = w0 >= m ? w0 : 0.0f;
          w1 = w1 >= m ? w1 : 0.0f;
          w2 = w2 >= m ? w2 : 0.0f;
          w3 = w3 >= m ? w3 : 0.0f;
        }
        ms.add(w0, w1, w2, w3);
      });
    } else {
      // tokens past the bracket (with top-k: past its bin) need no weight: without
      // top-k, top-p's mass comes from the histogram
      const float fl = q.use_k ? fk2 : f2;
      walk4<1>(r, [&](int j, const float4& v) {
        const float l[4] = {v.x, v.y, v.z, v.w};
        const float b[4] = {q.fbin(v.x), q.fbin(v.y), q.fbin(v.z), q.fbin(v.w)};
        if (!(fminf(fminf(b[0], b[1]), fminf(b[2], b[3])) <= fl)) return;  // NaN gives way to the others
        float a[4], t[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float w = wf(l[e]);
          a[e] = b[e] < f1 ? w : 0.0f;
          t[e] = b[e] > f2 && b[e] < fk ? w : 0.0f;
          if (!(b[e] < f1) && listed(l[e], b[e])) sm.cand[atomicAdd(&sm.ncand, 1)] = code_of(l[e], j + e);
        }
        as.add(a[0], a[1], a[2], a[3]);
        if (q.use_k) ts.add(t[0], t[1], t[2], t[3]);
        if (use_m) {
          const float m = (float)wmin;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            open = open || fabsf(a[e] - m) <= near;
            a[e] = a[e] >= m ? a[e] : 0.0f;
          }
          ms.add(a[0], a[1], a[2], a[3]);
        }
      });
    }
    if constexpr (!EXACT) {
      za = as.v;
      zt = za + ts.v;
      mass = q.bins && !use_m ? za : ms.v;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, o);
  }
  uint64_t cutcode = 0;  // kept: the tokens with at least this code
  if (good && q.bins) {
    __syncthreads();
    const int nc = sm.ncand, P = pow2_from(nc);
    if (lane == 0) *reinterpret_cast<A*>(&sm.seg[warp]) = mass;
    const uint64_t code = block_sort<NT>(tid < nc ? sm.cand[tid] : 0ull, P, sm.s.buf);
    const A wc = tid < nc ? weight(value_of((uint32_t)(code >> 32))) : A(0);
    const A cum = block_scan<NT>(wc, sm.red, (P + 31) & ~31);
    A* cums = reinterpret_cast<A*>(sm.s.mass);
    cums[tid] = cum;
    sm.cand[tid] = code;
    za = block_reduce<NT>(za, sm.red, Add{}, A(0));
    zt = block_reduce<NT>(zt, sm.red, Add{}, A(0));
    // how many candidates top-k leaves, then top-p
    int cut = nc;
    if (q.use_k) cut = q.bk > q.b2 ? q.n1 + (q.k - q.cnt_bk) : q.k - q.cnt_above;
    if (q.use_p) {
      const double pp = tp > 0.0f ? (double)tp : 0.0, zk = (double)(zt + (cut > 0 ? cums[cut - 1] : A(0)));
      const double z = EXACT || q.use_k ? zk : q.z;  // (without top-k the fp32 pass stops at the bracket)
      const double want = pp * z;
      int lo = 0, hi = min(q.n1, cut);  // candidates with less than `want` before them
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if ((double)(za + (mid ? cums[mid - 1] : A(0))) < want)
          lo = mid + 1;
        else
          hi = mid;
      }
      // the bracket holds the cut
      good = (q.cnt_above == 0 || (double)za < want) &&
             (lo < q.n1 || (q.use_k && q.b2 == q.bk) ||
              (q.n1 > 0 && (double)(za + cums[q.n1 - 1]) >= want));
      if (!EXACT && good) {  // and no token's border is within the error of what is wanted
        auto before = [&](int i) { return (double)(za + (i ? cums[i - 1] : A(0))); };
        const double slack = sm.slack;
        auto err = [&](double a) { return Expo32::off_by(pp, a, z, slack); };
        if (lo == 0)
          good = q.cnt_above == 0;
        else
          good = want - before(lo - 1) > err(before(lo - 1)) || (lo == 1 && q.cnt_above == 0);
        if (lo < min(q.n1, cut) || (lo == q.n1 && !(q.use_k && q.b2 == q.bk)))
          good = good && before(lo) - want > err(before(lo));
      }
      cut = q.cnt_above == 0 ? max(lo, 1) : lo;
    }
    good = good && cut > 0;
    if (good) {
      cutcode = sm.cand[cut - 1];
      // kept candidates into their segments, in a fixed order
      A add = 0;
      for (int i = lane; i < cut; i += 32) {
        const int at = (int)~(uint32_t)sm.cand[i];
        const A w = weight(value_of((uint32_t)(sm.cand[i] >> 32)));
        if (at >= r.seg0 && at < r.seg1 && w >= wmin) add += w;
        if (!EXACT && use_m) open = open || fabs((double)w - (double)wmin) <= (double)near;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) add += __shfl_xor_sync(0xffffffffu, add, o);
      mass += add;
    }
    __syncthreads();
  }
  if (!good) {
    if constexpr (EXACT) {
      const Filter f{q.use_k ? q.k : 0, tp};
      cutcode = cut_by_bisection<NT>(r, f, we, sm);
      mass = 0;
      walk<1>(r, [&](int j, float l) {
        if (!(l > -INFINITY) || code_of(l, j) < cutcode) return;
        const int64_t w = we(l);
        mass += w >= wmin ? w : 0;
      });
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, o);
      __syncthreads();
    } else {
      return false;
    }
  }
  if (lane == 0) *reinterpret_cast<A*>(&sm.seg[warp]) = mass;
  if constexpr (!EXACT) {
    if (use_m && __syncthreads_or(open)) return false;
  }
  __syncthreads();
  auto kept = [&](int j, float l) -> A {
    if (!(l > -INFINITY) || code_of(l, j) < cutcode) return A(0);
    const A w = weight(l);
    return w >= wmin ? w : A(0);
  };
  A total;
  const int pick = locate<NT, EXACT>(r, sm, u, total, kept);
  if (lane == 0 && pick >= 0) {
    const float l = r.base[pick];
    p.tokens[row] = pick - r.off;
    if (p.logprob) {
      const double z = EXACT ? log((double)total) - (double)p.sh * 0.6931471805599453 : log((double)total);
      p.logprob[row] = (float)((l == q.mx ? 0.0 : ((double)l - (double)q.mx) / (double)T) - z);
    }
  }
  return EXACT || __syncthreads_or(pick >= 0);
}

// One CTA a row.  STAGED: the row is kept in shared memory after its first pass.
template <int NT, bool STAGED>
__global__ void __launch_bounds__(NT, NT == 256 ? 4 : 1) sample_kernel(const SampleParams p) {
  __shared__ Smem<NT> sm;
  extern __shared__ __align__(16) uint64_t list[];  // [NT / 32 * kPart], then the staged row
  float* staged = reinterpret_cast<float*>(list + NT / 32 * kPart);
  constexpr int NW = NT / 32;
  const int row = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float* x = p.logits + (int64_t)row * p.ld;
  Row r;
  r.off = (int)((reinterpret_cast<uintptr_t>(x) >> 2) & 3);
  r.base = x - r.off;
  r.end = r.off + p.V;
  r.per = ((r.end + NW - 1) / NW + 127) / 128 * 128;
  r.seg0 = min(warp * r.per, r.end);
  r.seg1 = min(r.seg0 + r.per, r.end);
  const int sh = p.sh;
  const float T = p.temperature ? p.temperature[row] : 1.0f;
  if (tid < 32) sm.tab[tid] = kExp2[tid];
  if (tid == 32) {
    sm.c = 1.4426950408889634 / (double)T;
    sm.slack = slack_of(p);
  }
  const float u = p.u[row];
  int k = p.top_k ? p.top_k[row] : 0;
  const float tp = p.top_p ? p.top_p[row] : 1.0f;
  const float mp = p.min_p ? p.min_p[row] : 0.0f;

  bool late = false;  // the copy did not arrive
  if (STAGED) {
    // each warp's segment by one asynchronous copy of its own, the row's first and
    // last few tokens (not whole 16 bytes) by plain loads
    const int a = max(r.seg0, (r.off + 3) & ~3), b = min(r.seg1, r.end & ~3);
    if (lane == 0) {
      mbar_init(smem_u32(&sm.bar[warp]), 1);
      fence_mbar_init();
      if (a < b) {
        mbar_arrive_expect_tx(smem_u32(&sm.bar[warp]), (uint32_t)(b - a) * 4);
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                         smem_u32(staged + a)),
                     "l"(r.base + a), "r"((b - a) * 4), "r"(smem_u32(&sm.bar[warp]))
                     : "memory");
      }
    }
    if (r.seg0 == 0 && lane >= r.off && lane < min(4, r.end)) staged[lane] = r.base[lane];
    if (b < r.seg1 && lane < r.seg1 - b && b + lane >= r.off) staged[b + lane] = r.base[b + lane];
    __syncwarp();
    r.base = staged;
    if (a < b) {  // a copy that comes too late is still waited for, as long again: its target must be there
      const uint64_t t0 = global_timer_ns();
      uint64_t waited = 0;
      while (waited <= 2 * kWaitLimitNs && !mbar_try_wait(smem_u32(&sm.bar[warp]), 0)) waited = global_timer_ns() - t0;
      late = waited > kWaitLimitNs;
    }
  }
  if (T > 0.0f && u < 1.0f && tp >= 1.0f && !(mp > 0.0f) && (k <= 0 || k >= p.V)) {
    if (__syncthreads_or(late)) {
      if (tid == 0) {
        p.tokens[row] = -1;
        if (p.logprob) p.logprob[row] = NAN;
      }
      return;
    }
    int done = pick_plain<NT, false>(r, u, T, sm.c, sm, p, row);
    __syncthreads();
    if (done == 0) {
      done = pick_plain<NT, true>(r, u, T, sm.c, sm, p, row);
      __syncthreads();
    }
    if (done > 0) return;
  }
  // the maximum; the smallest of the threads' maxima
  float my_max = -INFINITY;
  walk4<4>(r, [&](int j, const float4& v) {
    my_max = fmaxf(my_max, fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)));  // ignores NaN
  });
  float mx = my_max, mm = my_max > -INFINITY ? my_max : INFINITY;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    mm = fminf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
  }
  if (lane == 0) {
    sm.redf[0][warp] = mx;
    sm.redf[1][warp] = mm;
  }
  for (int i = tid; i < kTopBins; i += NT) sm.h.cnt[i] = 0u;
  if (tid == 0) sm.ncand = 0;
  if (__syncthreads_or(late)) {
    if (tid == 0) {
      p.tokens[row] = -1;
      if (p.logprob) p.logprob[row] = NAN;
    }
    return;
  }
  mx = lane < NW ? sm.redf[0][lane] : -INFINITY;
  mm = lane < NW ? sm.redf[1][lane] : INFINITY;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    mm = fminf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
  }
  if (mx == -INFINITY) {  // nothing can be sampled
    if (tid == 0) {
      p.tokens[row] = -1;
      if (p.logprob) p.logprob[row] = -INFINITY;
    }
    return;
  }
  if (!(T > 0.0f)) {  // greedy
    int at = INT_MAX;
    if (my_max == mx)
      walk<4>(r, [&](int j, float l) {
        if (l == mx) at = min(at, j);
      });
    at = block_reduce<NT>(at, sm.red, Min{}, INT_MAX);
    if (tid == 0) {
      p.tokens[row] = at - r.off;
      if (p.logprob) p.logprob[row] = 0.0f;
    }
    return;
  }
  const Expo weight(mx, sm.c, sh, sm.tab);
  int64_t wmin = 0;
  if (mp > 0.0f) wmin = __double2ll_ru((double)fminf(mp, 1.0f) * (double)((int64_t)1 << sh));
  const bool use_p = !(tp >= 1.0f);
  Cut q;
  q.mx = mx;
  q.scale = 0.0f;

  // A small top-k: the bin of the k-th largest of the threads' maxima holds, with
  // the bins above it, at least k tokens and not many more, so one more pass
  // collects them all.
  if (k > 0 && k <= NT / 2 && mx < INFINITY) {
    const float range = fminf(mx - mm, 128.0f);
    q.scale = range > 0.0f ? fminf((float)(kTopBins - 1) / range, 1e30f) : 0.0f;  // 0: all the same
    if (my_max > -INFINITY)
      atomicAdd(&sm.h.cnt[__float_as_int(fminf(q.fbin(my_max), Cut::kOne + (float)(kTopBins - 1))) - 0x4b000000], 1u);
    __syncthreads();
    // every warp finds the bin
    int c8[kTopBins / 32], sum = 0;
#pragma unroll
    for (int e = 0; e < kTopBins / 32; ++e) {
      sum += (int)sm.h.cnt[lane * (kTopBins / 32) + e];
      c8[e] = sum;
    }
    const int64_t inc = warp_scan((int64_t)sum);
    const int pre = (int)inc - sum;
    int bstar = INT_MAX;
#pragma unroll
    for (int e = kTopBins / 32 - 1; e >= 0; --e)
      if (pre + c8[e] >= k) bstar = lane * (kTopBins / 32) + e;
    bstar = __reduce_min_sync(0xffffffffu, bstar);
    if (bstar < kTopBins - 1) {  // (the last bin takes in what is far below)
      // a value at or below every one in the bins up to it (a little lower: it was
      // fp32 arithmetic that put them there)
      const float edge = mx - ((float)bstar + 0.51f) / q.scale - fabsf(mx) * 1e-6f;
      const int n = q.scale > 0.0f ? collect<NT, 2>(r, list, sm.cand, NT, &sm.ncand,
                                                    [&](float l) { return l >= edge; })
                                   : NT + 1;
      if (n <= NT) {
        pick_from_list<NT>(n, k, tp, -1, -1, wmin, u, weight, T, sm, p, row, r.off);
        return;
      }
    }
    __syncthreads();
  }

  if (k >= p.V) k = 0;
  bool far_cut = false;
  if ((use_p || k > 0 || mp > 0.0f) && T <= 4.0f && Expo32::usable(mx, T)) {
    // How far from the maximum to list: min-p's reach where that is the only filter,
    // else what about five eighths of the list hold, judged by the first 128 tokens
    // of every segment (in 64 steps of T / 4).  Where those tokens' likely ones hold
    // far less than top-p's share, the list would be made in vain (10 of 60 us at
    // 32768 tokens).
    // (a weight that rounds to min-p's units may be under it: two units less)
    float least = mx + logf(fmaxf(fminf(mp, 1.0f) - two_units(p), 0.0f)) * T * 1.00001f - 1e-5f * T - fabsf(mx) * 1e-6f;
    bool enough = true;
    if (use_p || k > 0) {
      const Expo32 wf(mx, sm.c, T);
      for (int i = tid; i < 64; i += NT) sm.h.cnt[i] = sm.h.lo[i] = 0u;
      __syncthreads();
      const int j = r.seg0 + lane * 4;
      const float4 v = j < r.seg1 ? load4(r, j) : make_float4(NAN, NAN, NAN, NAN);
      const float l[4] = {v.x, v.y, v.z, v.w};
      uint32_t far = 0u;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t m = (uint32_t)(wf(l[e]) * 1048576.0f);
        const float step = (mx - fmaxf(l[e], wf.least)) * (4.0f / T);
        if (step < 64.0f) {
          atomicAdd(&sm.h.cnt[(int)step], 1u);
          atomicAdd(&sm.h.lo[(int)step], m);
        } else {
          far += m;
        }
      }
      const int64_t rest = block_reduce<NT>((int64_t)far, sm.red, Add{}, (int64_t)0);  // (a barrier too)
      // inclusive counts and masses, two steps a lane
      const uint32_t c0 = sm.h.cnt[2 * lane], c1 = c0 + sm.h.cnt[2 * lane + 1];
      const int64_t m0 = sm.h.lo[2 * lane], m1 = m0 + sm.h.lo[2 * lane + 1];
      const int64_t cb = warp_scan((int64_t)c1) - c1, mb = warp_scan(m1) - m1, all = __shfl_sync(0xffffffffu, mb + m1, 31);
      const int64_t most = (int64_t)(NT / 32 * kPart) * 5 / 8 * min(r.per, 128) / r.per;
      const int steps = __reduce_add_sync(0xffffffffu, (cb + c0 <= most) + (cb + c1 <= most));
      const int64_t near = __reduce_max_sync(0xffffffffu, (uint32_t)(cb + c1 <= most ? mb + m1 : cb + c0 <= most ? mb + m0 : 0));
      least = mx - 0.25f * T * (float)steps;
      const double scale = (double)r.per / min(r.per, 128);
      const double z = (all + rest) * scale + 1048576.0, want = tp * z - 1048576.0;
      // (the sample knows the tail's share, of many tokens, better than the head's)
      enough = steps > 0 && (k > 0 ? k <= most * scale : near * scale + 1048576.0 > (1.25 * tp - 0.25) * z);
      far_cut = __popc(__ballot_sync(0xffffffffu, (mb + m1) * scale < want)) >= 15;  // past 7.5 T
    }
    __syncthreads();
    if (enough && pick_from_top<NT>(r, k, tp, mp, u, T, least, weight, list, sm, p, row)) return;
    __syncthreads();
  }

  q.use_p = use_p;
  q.use_k = k > 0;
  // Top-p alone: the histogram covers what weighs e^-8 and more, where the cut
  // mostly is, or else down to 2^-32.
  float spread = INFINITY;
  if (q.use_k || T > 4.0f) {
    int nf = 0;
    float mn = INFINITY;
    walk<4>(r, [&](int, float l) {
      if (l > -INFINITY) {
        ++nf;
        mn = fminf(mn, l);
      }
    });
    q.use_k = q.use_k && k < block_reduce<NT>((int64_t)nf, sm.red, Add{}, (int64_t)0);
    spread = mx - block_reduce<NT>(mn, sm.red, MinF{}, INFINITY);
  }
  q.k = q.use_k ? k : 0;
  q.bins = q.use_k || use_p;
  q.b1 = q.b2 = q.bk = kBins;
  q.z = 0.0;
  q.n1 = q.cnt_above = q.cnt_bk = 0;
  q.fits = true;
  if (q.bins && !(mx < INFINITY)) q.fits = false;
  for (int turn = far_cut ? 1 : 0; q.bins && q.fits && turn < 2; ++turn) {
    // with top-k, what is farther shares the last bin
    const float range = q.use_k ? fminf(spread, 128.0f) : fminf(spread, (turn == 0 ? 8.0f : 22.5f) * T);
    q.scale = range > 0.0f ? fminf((float)(kBins - 1) / range, 1e30f) : 0.0f;
    __syncthreads();
    for (int i = tid; i < kBins; i += NT) sm.h.cnt[i] = sm.h.lo[i] = sm.h.hi[i] = 0u;
    if (tid == 0) {
      sm.ncand = 0;
      sm.bk = sm.b1 = sm.b2 = kBins - 1;
      sm.cnt_bk = 0;
    }
    __syncthreads();
    const Expo32 wf(mx, sm.c, T);
    const float unit = (float)(1u << (2 * p.half));
    Sum all;
    walk4<1>(r, [&](int, const float4& v) {
      const float l[4] = {v.x, v.y, v.z, v.w};
      uint32_t m[4] = {0u, 0u, 0u, 0u};
      float b[4];
      if (use_p) {
        const float w[4] = {wf(v.x), wf(v.y), wf(v.z), wf(v.w)};
        if (!q.use_k) all.add(w[0], w[1], w[2], w[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) m[e] = (uint32_t)(w[e] * unit);  // 0 for -inf and NaN
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e] = q.fbin(l[e]);
      // (-inf and NaN fall out of every bin; with top-k only NaN and -inf beyond a bin's reach do)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (q.use_k ? l[e] > -INFINITY : b[e] <= Cut::kFar) {
          const int at = __float_as_int(fminf(b[e], Cut::kFar)) - 0x4b000000;
          atomicAdd(&sm.h.cnt[at], 1u);
          if (m[e]) {
            atomicAdd(&sm.h.lo[at], m[e] & ((1u << p.half) - 1u));
            if (m[e] >> p.half) atomicAdd(&sm.h.hi[at], m[e] >> p.half);
          }
        }
      }
    });
    __syncthreads();
    constexpr int BPT = kBins / NT;  // bins a thread
    int64_t cn[BPT], ms[BPT], cs = 0, mass = 0;
#pragma unroll
    for (int e = 0; e < BPT; ++e) {
      const int b = tid * BPT + e;
      cs += sm.h.cnt[b];
      mass += ((int64_t)sm.h.hi[b] << p.half) + sm.h.lo[b];
      cn[e] = cs;
      ms[e] = mass;
    }
    const int64_t c0 = block_scan<NT>(cs, sm.red) - cs;
    int64_t m0 = 0;
    if (use_p) {
      q.z = q.use_k ? 0.0 : block_reduce<NT>(all.v, sm.red, Add{}, 0.0);
      m0 = block_scan<NT>(mass, sm.red) - mass;
      if (tid == NT - 1) {
        sm.seg[0] = sm.seg[1] = q.use_k ? 0 : (int64_t)(q.z * (double)unit);
        sm.seg[2] = m0 + mass;  // the bins'
      }
    }
    // sm.seg[0, 1]: mass before and with the last bin that counts
    __syncthreads();
    if (q.use_k) {
#pragma unroll
      for (int e = 0; e < BPT; ++e) {
        const int64_t pre = c0 + (e ? cn[e - 1] : 0);
        if (pre < k && c0 + cn[e] >= k) {
          sm.bk = tid * BPT + e;
          sm.cnt_bk = (int)pre;
          sm.seg[0] = m0 + (e ? ms[e - 1] : 0);
          sm.seg[1] = m0 + ms[e];
        }
      }
      __syncthreads();
      q.bk = sm.bk;
      q.cnt_bk = sm.cnt_bk;
    }
    const int last = q.use_k ? q.bk : kBins - 1;
    if (use_p) {
      // a bin's true mass is between m and m + its tokens (truncated units), well to 1e-4
      const double pp = tp > 0.0f ? (double)tp : 0.0;
      const double w_lo = pp * (double)sm.seg[0] * 0.9998 - (double)p.V,
                   w_hi = pp * ((double)sm.seg[1] + p.V) * 1.0002 + 1.0;
      if (!q.use_k && turn == 0 && spread > 8.0f * T && (double)sm.seg[2] < w_hi) continue;  // the cut may be in the tail
#pragma unroll
      for (int e = 0; e < BPT; ++e) {
        const int b = tid * BPT + e;
        const double cum = (double)(m0 + ms[e]), pre = (double)(m0 + (e ? ms[e - 1] : 0));
        // the first bin that may, and the first that must, reach what is wanted
        if (cum + p.V >= w_lo && (b == 0 || pre + p.V < w_lo)) sm.b1 = b;
        if (cum >= w_hi && (b == 0 || pre < w_hi)) sm.b2 = b;
      }
      __syncthreads();
      q.b1 = min(sm.b1, last);
      q.b2 = min(sm.b2, last);
    } else {
      q.b1 = q.b2 = q.bk;
    }
#pragma unroll
    for (int e = 0; e < BPT; ++e) {
      const int b = tid * BPT + e;
      if (b == q.b1) sm.cnt_b1 = (int)(c0 + (e ? cn[e - 1] : 0));
      if (b == q.b2) sm.cnt_b2 = (int)(c0 + cn[e]);
    }
    __syncthreads();
    q.cnt_above = sm.cnt_b1;
    q.n1 = sm.cnt_b2 - q.cnt_above;
    const int in_bk = q.use_k ? (int)sm.h.cnt[q.bk] : 0;
    q.fits = q.n1 + (q.use_k && q.bk > q.b2 ? in_bk : 0) <= NT;
    __syncthreads();
    if (!q.use_k && q.cnt_above + q.n1 <= NT && Expo32::usable(mx, T)) {
      // A small nucleus: all its tokens fit the list, and the fp32 mass of all tokens
      // settles the cut unless it falls within its error of a token's border.
      const float edge = Cut::kOne + (float)q.b2;  // (b2 is the last bin: what is past it weighs nothing)
      collect<NT, 2>(r, list, sm.cand, NT, &sm.ncand,
                     [&](float l) { return l > -INFINITY && q.fbin(l) <= edge; });
      const double z = q.z * (double)((int64_t)1 << sh);
      const double err = z * Expo32::kErr + (double)p.V;  // and the units' rounding
      const int64_t z_lo = (int64_t)(z - err), z_hi = (int64_t)(z + err) + 1;
      if (pick_from_list<NT>(q.cnt_above + q.n1, INT_MAX, tp, z_lo, z_hi, wmin, u, weight, T, sm, p, row, r.off))
        return;
      __syncthreads();
    }
    break;
  }
  if (q.fits && u < 1.0f && Expo32::usable(mx, T)) {
    if (pick_from_row<NT, false>(r, q, tp, mp, u, T, weight, sm, p, row)) return;
    __syncthreads();
  }
  pick_from_row<NT, true>(r, q, tp, mp, u, T, weight, sm, p, row);
}

template <int NT, bool STAGED>
nc_status launch_t(const SampleParams& p, int M, size_t smem, cudaStream_t stream) {
  auto* fn = sample_kernel<NT, STAGED>;
  if (smem > 0) {
    static bool attr_done[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 64 || !attr_done[dev]) {
      if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kStageBytes) != cudaSuccess)
        return NC_ERR_CUDA;
      if (dev < 64) attr_done[dev] = true;
    }
  }
  fn<<<M, NT, smem, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? NC_OK : NC_ERR_CUDA;
}

}  // namespace

nc_status sample_launch(const float* logits, int64_t ld, const float* u, const float* temperature,
                        const int32_t* top_k, const float* top_p, const float* min_p, int32_t* tokens,
                        float* logprob, int M, int V, cudaStream_t stream) {
  if (M == 0) return NC_OK;
  int bits = 0;  // V <= 2^bits
  while (((int64_t)1 << bits) < V) ++bits;
  const int sh = 62 - bits < 51 ? 62 - bits : 51;
  const int half = 31 - bits < 15 ? 31 - bits : 15;  // V tokens in one bin do not overflow a sum
  const SampleParams p{logits, ld, u, temperature, top_k, top_p, min_p, tokens, logprob, V, sh, half};
  // Rows for every SM and more: some on each SM, they load and compute in turn (from
  // L2 after a row's first pass).  Fewer: a row's later passes from shared memory.
  // Measured, us, staged / four an SM, 32768 logits, top-k 50 with top-p 0.95: 148 rows 16.4 / 22.0,
  // 149 rows 25.6 / 21.5, 592 rows 54 / 32.  Top-p alone: 148 rows 64 / 104, 296 rows 112 / 151, 592
  // rows 184 / 148; without a filter 149 rows 32 / 40, 400 rows 48 / 42: those two would turn over
  // at some 400 rows, but what a row asks for is not known here.
  if (M > device_sm_count()) return launch_t<256, false>(p, M, 8 * kPart * 8, stream);
  const size_t smem = 16 * kPart * 8 + ((size_t)V + 7) / 4 * 16;
  if (smem <= kStageBytes) return launch_t<512, true>(p, M, smem, stream);
  return launch_t<512, false>(p, M, 16 * kPart * 8, stream);
}

}  // namespace nc
