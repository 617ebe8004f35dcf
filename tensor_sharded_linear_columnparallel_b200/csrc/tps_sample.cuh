// tps_sample.cuh -- sampling one token per row of logits from given uniform numbers:
// temperature, then top-k, then top-p over what is left, then min-p, then the inverse
// of the cumulative weights in vocabulary order.
//
// w_i = exp((l_i - max) / T). The filters keep a top part of the order (logit
// descending, index ascending), so the kept set is {key > t} plus the first r tokens
// with key == t, and no sort is needed: t and r are found from counts (top-k) and from
// sums of weights (top-p). Weights are held as integers in units of 2^-44, so sums are
// exact, do not depend on the order of the additions, and agree with 64-bit floating
// point to 2^-45 per token: a float sum would let the rounding of a 128256-token sum
// decide which token a uniform number falls on.
#pragma once

#include <cstdint>

namespace tps {

constexpr int kSampleThreads = 1024;

__device__ __forceinline__ float sample_load(const void* p, int f32, long long i) {
  const float x = f32 ? static_cast<const float*>(p)[i]
                      : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return x == x ? x : -INFINITY;   // a NaN logit is never drawn
}

// Unsigned key with the order of the floats; -0 counts as +0.
__device__ __forceinline__ uint32_t sample_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// exp(-(mx - x) / T) in units of 2^-44.
__device__ __forceinline__ unsigned long long sample_weight(float x, float mx, double inv_t) {
  if (!(x > -INFINITY)) return 0ull;
  if (x == mx) return 1ull << 44;
  if (mx == INFINITY) return 0ull;
  const double y = (static_cast<double>(x) - static_cast<double>(mx)) * inv_t;
  return y < -32.0 ? 0ull : __double2ull_rn(exp(y) * 17592186044416.0);
}

template <class T, class Op>
__device__ __forceinline__ T sample_block_reduce(T v, T* red, Op op) {
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
  for (int i = 1; i < kSampleThreads / 32; ++i) v = op(v, red[i]);
  return v;
}

// Plain form: one CTA per row, every threshold found bit by bit from passes over the row.
__global__ void __launch_bounds__(kSampleThreads) tps_sample_plain_kernel(const SampleArgs a) {
  typedef unsigned long long u64;
  __shared__ u64 red[32];
  __shared__ float redf[32];
  __shared__ int pick;
  griddep_wait();
  auto add = [](u64 x, u64 y) { return x + y; };
  for (int row = blockIdx.x; row < a.m; row += gridDim.x) {
    const long long base = static_cast<long long>(row) * a.V;
    auto at = [&](int i) { return sample_load(a.logits, a.f32, base + i); };
    float mx = -INFINITY;
    for (int i = threadIdx.x; i < a.V; i += kSampleThreads) mx = fmaxf(mx, at(i));
    mx = sample_block_reduce(mx, redf, [](float x, float y) { return fmaxf(x, y); });
    const float T = a.temperature ? a.temperature[row] : 1.0f;
    const bool greedy = !(T > 0.0f);
    const double inv_t = greedy ? 0.0 : 1.0 / static_cast<double>(T);
    const long long k = a.top_k ? a.top_k[row] : 0;
    const double p = a.top_p ? static_cast<double>(a.top_p[row]) : 1.0;
    const double q = a.min_p ? static_cast<double>(a.min_p[row]) * 17592186044416.0 : 0.0;
    uint32_t t = 0;                              // kept: key > t, and the first r with key == t
    long long r = a.V;
    if (greedy) {
      t = sample_key(mx);
      r = 1;
    } else {
      if (k > 0 && k < a.V) {
        u64 above = 0;
        for (int bit = 31; bit >= 0; --bit) {
          const uint32_t c = t | (1u << bit);
          u64 n = 0;
          for (int i = threadIdx.x; i < a.V; i += kSampleThreads) n += sample_key(at(i)) >= c;
          n = sample_block_reduce(n, red, add);
          if (n >= static_cast<u64>(k)) t = c;
          else above = n;
        }
        r = k - static_cast<long long>(above);
      }
      if (p < 1.0) {
        const uint32_t tk = t;
        const long long rk = r;
        const u64 wk = tk ? sample_weight(__uint_as_float((tk & 0x80000000u) ? (tk ^ 0x80000000u) : ~tk), mx, inv_t) : 0;
        auto mass = [&](uint32_t c) {            // weight of the kept tokens with key >= c
          u64 s = 0;
          for (int i = threadIdx.x; i < a.V; i += kSampleThreads) {
            const float x = at(i);
            const uint32_t key = sample_key(x);
            if (key >= c && (key > tk || tk == 0)) s += sample_weight(x, mx, inv_t);
          }
          s = sample_block_reduce(s, red, add);
          return (tk && c <= tk) ? s + wk * static_cast<u64>(rk) : s;
        };
        const double target = p * static_cast<double>(mass(0));
        u64 above = 0;
        t = 0;
        for (int bit = 31; bit >= 0; --bit) {
          const uint32_t c = t | (1u << bit);
          const u64 s = mass(c);
          if (s > 0 && static_cast<double>(s) >= target) t = c;
          else above = s;
        }
        const u64 wt = sample_weight(__uint_as_float((t & 0x80000000u) ? (t ^ 0x80000000u) : ~t), mx, inv_t);
        r = 0;                                   // tie i is kept iff above + i * wt < target, the first always
        do ++r;
        while (static_cast<double>(above + static_cast<u64>(r) * wt) < target && r < a.V);
        if (t == tk && r > rk) r = rk;
      }
    }
    // the draw: each thread takes a contiguous part of the row
    const int per = (a.V + kSampleThreads - 1) / kSampleThreads;
    const int i0 = min(a.V, static_cast<int>(threadIdx.x) * per), i1 = min(a.V, i0 + per);
    u64 ties = 0;
    for (int i = i0; i < i1; ++i) ties += sample_key(at(i)) == t;
    auto exclusive = [&](u64 v, u64& total) {
      u64 s = v;
      for (int o = 1; o < 32; o <<= 1) {
        const u64 n = __shfl_up_sync(0xffffffffu, s, o);
        if ((threadIdx.x & 31) >= o) s += n;
      }
      __syncthreads();
      if ((threadIdx.x & 31) == 31) red[threadIdx.x >> 5] = s;
      __syncthreads();
      u64 before = 0;
      total = 0;
      for (int w = 0; w < kSampleThreads / 32; ++w) {
        if (w < static_cast<int>(threadIdx.x >> 5)) before += red[w];
        total += red[w];
      }
      return before + s - v;
    };
    u64 unused;
    const u64 tie0 = exclusive(ties, unused);
    auto weight = [&](int i, u64& tie) -> u64 {
      const float x = at(i);
      const uint32_t key = sample_key(x);
      if (key < t) return 0;
      if (key == t && tie++ >= static_cast<u64>(r)) return 0;
      const u64 w = sample_weight(x, mx, inv_t);
      return (x == mx || static_cast<double>(w) >= q) ? w : 0;
    };
    u64 mine = 0, tie = tie0, total;
    for (int i = i0; i < i1; ++i) mine += weight(i, tie);
    const u64 before = exclusive(mine, total);
    const double uu = a.u[row];
    u64 target = uu > 0.0 ? static_cast<u64>(uu * static_cast<double>(total)) : 0;
    if (target >= total && total > 0) target = total - 1;
    if (threadIdx.x == 0) pick = -1;
    __syncthreads();
    if (before <= target && target < before + mine) {
      u64 c = before;
      tie = tie0;
      for (int i = i0; i < i1; ++i) {
        const u64 w = weight(i, tie);
        c += w;
        if (c > target) {
          pick = i;
          a.out_idx[row] = i;
          if (a.out_logp) a.out_logp[row] = static_cast<float>(log(static_cast<double>(w) / static_cast<double>(total)));
          break;
        }
      }
    }
    __syncthreads();
    if (threadIdx.x == 0 && pick < 0) {          // no finite or infinite-positive logit in the row
      a.out_idx[row] = -1;
      if (a.out_logp) a.out_logp[row] = -INFINITY;
    }
    __syncthreads();
  }
}

}  // namespace tps
