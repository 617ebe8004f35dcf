// tps_sample.cuh -- sampling one token per row of logits from given uniform numbers:
// temperature, then top-k, then top-p over what is left, then min-p, then the inverse
// of the running sum of the kept weights in vocabulary order.
//
// w_i = exp((l_i - max) / T) as an integer in units of 2^-44. Sums of integers are exact
// and do not depend on the order of the additions, and they agree with 64-bit floating
// point to half a unit per token; a float sum would let the rounding of a sum over
// 128256 tokens decide which token a uniform number falls on.
//
// Every filter keeps a top part of the order (logit descending, index ascending), which is
// the order of the 64-bit number rank = (sortable logit bits << 32 | ~index). So a row's
// filters are one threshold C, kept = rank >= C, and no sort of the row is needed. One
// thread-block cluster holds a row in the shared memory of its CTAs (fp32, read once from
// HBM) and finds C from a histogram of 1024 equal bins over the logits within 32 T of the
// maximum (what lies below has no weight): counts, and weights in units of 2^-15 with the
// error that truncation and the bin's borders allow, so the bins that can hold the cut are
// known for certain. Their few tokens go to the first CTA, which sorts them and takes the
// cut from exact sums. Where they are more than the list holds (equal logits, one far
// outlier that stretches the bins), C is found bit by bit from passes over shared memory.
//
// Bound by latency for few rows (a dozen cluster barriers of about a microsecond) and by
// the 64-bit exponentials for many.
#pragma once

#include <cstdint>

namespace tps {

typedef unsigned long long u64;

constexpr int kSampleThreads = 512;
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int kSampleBins = 1024;
constexpr int kSampleList = 1024;              // entries of the candidate list, which overlays the histogram
constexpr u64 kSampleOne = 1ull << 44;         // weight of the largest logit
constexpr int kSampleMassShift = 29;           // histogram weights in units of 2^-15: 49152 of them fit 32 bits

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ u64 ld_cluster_u64(uint32_t addr) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// Unsigned key with the order of the floats (NaN and -0 do not occur: sample_clean).
__device__ __forceinline__ uint32_t sample_key(float x) {
  const uint32_t u = __float_as_uint(x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float sample_unkey(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}
__device__ __forceinline__ u64 sample_rank(float x, int i) {
  return static_cast<u64>(sample_key(x)) << 32 | (0xffffffffu - static_cast<uint32_t>(i));
}
// A NaN logit is never drawn; -0 equals +0.
__device__ __forceinline__ float sample_clean(float x) { return x == x ? x + 0.0f : -INFINITY; }

// 2^-y for y >= 0 in units of 2^-44, rounded: y = n + f with f in [-1/2, 1/2], 2^-f as its
// Taylor sum to (f ln 2)^11 / 11! (the rest is below 2^-47), the power of two put into the
// exponent field, and the integer read from the low bits after adding 2^52.
__device__ __forceinline__ u64 sample_exp2(double y) {
  if (!(y < 46.0)) return 0ull;
  const double t = y + 6755399441055744.0;                  // 1.5 * 2^52: y rounded to an integer, in the low bits
  const int n = static_cast<int>(__double2loint(t));
  const double f = (t - 6755399441055744.0) - y;
  double p = 4.4455382718708115e-10;                        // ln(2)^k / k!, k = 11 ... 0
  p = fma(p, f, 7.0549116208011233e-09);
  p = fma(p, f, 1.0178086009239699e-07);
  p = fma(p, f, 1.3215486790144310e-06);
  p = fma(p, f, 1.5252733804059840e-05);
  p = fma(p, f, 1.5403530393381609e-04);
  p = fma(p, f, 1.3333558146428443e-03);
  p = fma(p, f, 9.6181291076284772e-03);
  p = fma(p, f, 5.5504108664821580e-02);
  p = fma(p, f, 2.4022650695910072e-01);
  p = fma(p, f, 6.9314718055994531e-01);
  p = fma(p, f, 1.0);
  const double v = __hiloint2double(__double2hiint(p) + ((44 - n) << 20), __double2loint(p));   // p * 2^(44 - n)
  return static_cast<u64>(__double_as_longlong(v + 4503599627370496.0)) & ((1ull << 52) - 1);
}

struct SampleRow {             // one row's parameters, the same in every CTA of its cluster
  float mx, mn;                // largest logit, smallest one above -inf
  double c;                    // log2(e) / T
  float bin_scale;             // bins per logit
  double q;                    // min_p in units of 2^-44
};

__device__ __forceinline__ u64 sample_weight(float x, const SampleRow& r) {
  if (!(x > -INFINITY)) return 0ull;
  if (x == r.mx) return kSampleOne;
  return sample_exp2((static_cast<double>(r.mx) - static_cast<double>(x)) * r.c);   // mx = inf: 0
}

// Bin of a logit: 0 holds the largest, the last one everything from 32 T below it on.
__device__ __forceinline__ int sample_bin(float x, const SampleRow& r) {
  return x == r.mx ? 0 : static_cast<int>(fminf((r.mx - x) * r.bin_scale, static_cast<float>(kSampleBins - 1)));
}

// What the first CTA tells the others about the next step (one copy per CTA).
struct SampleCmd {
  int lo, hi;                  // bins whose tokens are listed
  int n;                       // their number; -1: too many (bit by bit); -2: no cut
  int unused;
  u64 C;                       // threshold so far
  u64 total;                   // weight of the tokens at or above it
};

struct SampleSmem {
  u64 red[kSampleWarps];
  u64 part[2][8];              // values that the CTAs of the cluster exchange, two in turn
  SampleCmd cmd;
  int count;                   // list entries of this CTA so far
  int unused;
  float fred[2 * kSampleWarps];
  int ired[kSampleWarps];
  int pad[2];
};

constexpr int sample_smem_bytes(int slice) {
  return static_cast<int>(sizeof(SampleSmem)) + kSampleBins * 8 + slice * 4;
}

template <class T, class Op>
__device__ __forceinline__ T sample_warp_reduce(T v, Op op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ u64 sample_block_sum(u64 v, SampleSmem& s) {
  v = sample_warp_reduce(v, [](u64 x, u64 y) { return x + y; });
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s.red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int i = 0; i < kSampleWarps; ++i) v += s.red[i];
  return v;
}
// Exclusive sum over the block, and the total.
__device__ __forceinline__ u64 sample_block_scan(u64 v, u64& total, SampleSmem& s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 n = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += n;
  }
  __syncthreads();
  if (lane == 31) s.red[warp] = incl;
  __syncthreads();
  u64 before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < kSampleWarps; ++i) {
    if (i < warp) before += s.red[i];
    total += s.red[i];
  }
  return before + incl - v;
}

__global__ void __launch_bounds__(kSampleThreads) tps_sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SampleSmem& s = *reinterpret_cast<SampleSmem*>(smem_raw);
  uint32_t* cnt = reinterpret_cast<uint32_t*>(smem_raw + sizeof(SampleSmem));
  uint32_t* mass = cnt + kSampleBins;
  u64* list = reinterpret_cast<u64*>(cnt);
  float* xs = reinterpret_cast<float*>(cnt + 2 * kSampleBins);
  static_assert(sizeof(SampleSmem) % 16 == 0 && kSampleList * 8 <= kSampleBins * 8, "shared memory layout");

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cs = static_cast<int>(cluster_nctarank()), cr = static_cast<int>(cluster_ctarank());
  const int row = static_cast<int>(blockIdx.x) / cs;
  const int i0 = min(a.V, cr * a.slice), n = min(a.V, i0 + a.slice) - i0;   // this CTA's tokens [i0, i0 + n)
  // address of a member of SampleSmem (or of what follows it) in CTA r
  auto remote = [&](const void* p, int r) { return mapa_shared(smem_u32(p), static_cast<uint32_t>(r)); };
  int turn = 0;
  // sum of one value per CTA, in every CTA (v the same in all threads of a CTA)
  auto cluster_all = [&](u64 v) {
    if (tid < cs) st_cluster_u64(remote(&s.part[turn][cr], tid), v);
    cluster_sync_all();
    u64 t = 0;
    for (int r = 0; r < cs; ++r) t += s.part[turn][r];
    turn ^= 1;
    return t;
  };
  griddep_wait();

  // ------------------------------------------------ the row into shared memory, its largest and smallest logit
  float mx = -INFINITY, mn = INFINITY;
  int arg = 0x7fffffff;
  auto take = [&](float x, int i) {
    if (x > mx || (x == mx && i < arg)) mx = x, arg = i;
    if (x > -INFINITY) mn = fminf(mn, x);
  };
  if (a.f32) {
    const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) +
                                                        static_cast<long long>(row) * a.V + i0);
#pragma unroll 4
    for (int v = tid; v < n / 4; v += kSampleThreads) {
      float4 x = __ldcs(src + v);
      x = make_float4(sample_clean(x.x), sample_clean(x.y), sample_clean(x.z), sample_clean(x.w));
      reinterpret_cast<float4*>(xs)[v] = x;
      take(x.x, i0 + 4 * v), take(x.y, i0 + 4 * v + 1), take(x.z, i0 + 4 * v + 2), take(x.w, i0 + 4 * v + 3);
    }
  } else {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.logits) +
                                                      static_cast<long long>(row) * a.V + i0);
#pragma unroll 2
    for (int v = tid; v < n / 8; v += kSampleThreads) {
      const uint4 b = __ldcs(src + v);
      const uint32_t w[4] = {b.x, b.y, b.z, b.w};
      float x[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[2 * j] = sample_clean(__uint_as_float(w[j] << 16));
        x[2 * j + 1] = sample_clean(__uint_as_float(w[j] & 0xffff0000u));
      }
      reinterpret_cast<float4*>(xs)[2 * v] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4*>(xs)[2 * v + 1] = make_float4(x[4], x[5], x[6], x[7]);
#pragma unroll
      for (int j = 0; j < 8; ++j) take(x[j], i0 + 8 * v + j);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, mx, o);
    const int i = __shfl_xor_sync(0xffffffffu, arg, o);
    if (y > mx || (y == mx && i < arg)) mx = y, arg = i;
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
  }
  if (lane == 0) s.fred[warp] = mx, s.fred[kSampleWarps + warp] = mn, s.ired[warp] = arg;
  __syncthreads();
  for (int w = 0; w < kSampleWarps; ++w) {
    if (s.fred[w] > mx || (s.fred[w] == mx && s.ired[w] < arg)) mx = s.fred[w], arg = s.ired[w];
    mn = fminf(mn, s.fred[kSampleWarps + w]);
  }
  if (tid < cs) {
    st_cluster_u64(remote(&s.part[0][cr], tid), sample_rank(mx, arg));
    st_cluster_u64(remote(&s.part[1][cr], tid), __float_as_uint(mn));
  }
  cluster_sync_all();
  u64 top = 0;
  for (int r = 0; r < cs; ++r) {
    top = max(top, s.part[0][r]);
    mn = fminf(mn, __uint_as_float(static_cast<uint32_t>(s.part[1][r])));
  }
  mx = sample_unkey(static_cast<uint32_t>(top >> 32));
  cluster_sync_all();                          // part[] is free again

  const float T = a.temperature ? a.temperature[row] : 1.0f;
  const float pf = a.top_p ? a.top_p[row] : 1.0f;
  const int k = a.top_k ? a.top_k[row] : 0;
  const bool greedy = !(T > 0.0f);
  if (greedy || mx == -INFINITY) {             // the same in the whole cluster
    if (cr == 0 && tid == 0) {
      const bool none = mx == -INFINITY;
      a.out_idx[row] = none ? -1 : static_cast<int>(0xffffffffu - static_cast<uint32_t>(top));
      if (a.out_logp) a.out_logp[row] = none ? -INFINITY : 0.0f;
    }
    return;
  }
  SampleRow r;
  r.mx = mx;
  r.mn = mn;
  r.c = 1.4426950408889634 / static_cast<double>(T);
  r.q = a.min_p ? static_cast<double>(a.min_p[row]) * static_cast<double>(kSampleOne) : 0.0;
  const float range = fminf(mx - mn, 32.0f * T);
  r.bin_scale = range > 0.0f ? static_cast<float>(kSampleBins - 1) / range : 0.0f;
  const double p = static_cast<double>(pf);
  u64 C = 0;                                   // kept: rank >= C (and min_p)
  auto each = [&](auto f) {                    // every token of this CTA at or above C with a finite or +inf logit
    for (int j = tid; j < n; j += kSampleThreads) {
      const float x = xs[j];
      if (x > -INFINITY && sample_rank(x, i0 + j) >= C) f(x, i0 + j);
    }
  };

  // Largest threshold >= C that keeps at least `want` tokens (weight: at least `target`), bit by bit.
  auto bisect = [&](bool by_weight, u64 want, double target) {
    u64 t = 0;
    for (int bit = 63; bit >= 0; --bit) {
      const u64 c = t | (1ull << bit);
      u64 v = 0;
      each([&](float x, int i) {
        if (sample_rank(x, i) >= c) v += by_weight ? sample_weight(x, r) : 1ull;
      });
      v = cluster_all(sample_block_sum(v, s));
      if (by_weight ? (v > 0 && static_cast<double>(v) >= target) : v >= want) t = c;
    }
    if (t > C) C = t;
  };

  // One cut of the tokens at or above C: the k first of them, and / or those that reach share
  // p of their weight. Returns whether the share of p has been taken too.
  auto cut = [&](int k, bool by_p) -> bool {
    for (int j = tid; j < 2 * kSampleBins; j += kSampleThreads) cnt[j] = 0;
    __syncthreads();
    u64 sum = 0;
    each([&](float x, int) {
      const int b = sample_bin(x, r);
      atomicAdd(cnt + b, 1u);
      if (k == 0) {
        const u64 w = sample_weight(x, r);
        sum += w;
        const uint32_t m = static_cast<uint32_t>(w >> kSampleMassShift);
        if (m) atomicAdd(mass + b, m);
      }
    });
    const u64 total = cluster_all(sample_block_sum(sum, s));
    if (cr == 0) {
      // bins 2 tid and 2 tid + 1 over the cluster
      u64 c2[2] = {0, 0}, m2[2] = {0, 0};
      for (int q = 0; q < cs; ++q) {
        const u64 c = ld_cluster_u64(remote(cnt + 2 * tid, q));
        const u64 m = ld_cluster_u64(remote(mass + 2 * tid, q));
        c2[0] += c & 0xffffffffu, c2[1] += c >> 32;
        m2[0] += m & 0xffffffffu, m2[1] += m >> 32;
      }
      u64 all;
      const u64 cb = sample_block_scan(c2[0] + c2[1], all, s);   // tokens in the bins before
      const u64 cum[3] = {cb, cb + c2[0], cb + c2[0] + c2[1]};
      if (tid == 0) s.cmd.lo = s.cmd.hi = kSampleBins - 1, s.cmd.n = 0;
      __syncthreads();
      if (k > 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (cum[j] < static_cast<u64>(k) && static_cast<u64>(k) <= cum[j + 1]) {
            const bool from0 = cum[j + 1] <= kSampleList;       // every kept token fits the list: p in the same step
            s.cmd.lo = from0 ? 0 : 2 * tid + j;
            s.cmd.hi = 2 * tid + j;
            s.cmd.n = static_cast<int>(cum[j + 1] - (from0 ? 0 : cum[j]));
            s.cmd.total = from0 ? 0 : cum[j];                   // tokens before the list
          }
        __syncthreads();
        if (tid == 0 && static_cast<u64>(k) >= all) s.cmd.n = -2;
      } else {
        // bounds of each bin's weight: truncation, and the weights at its borders (a hundredth
        // of a bin wider, for the rounding of sample_bin)
        const double target = p * static_cast<double>(total);
        const double step = r.bin_scale > 0.0f ? r.c / static_cast<double>(r.bin_scale) : 0.0;   // log2 per bin
        u64 lw[2], hw[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int b = 2 * tid + j;
          const u64 wh = b == 0 ? kSampleOne : sample_exp2((b - 0.01) * step) + 1;
          const u64 e = sample_exp2((b + 1.01) * step);
          const u64 wl = b == kSampleBins - 1 || e == 0 ? 0 : e - 1;
          lw[j] = max(m2[j] << kSampleMassShift, c2[j] * wl);
          hw[j] = min((m2[j] + c2[j]) << kSampleMassShift, c2[j] * wh);
        }
        u64 t1, t2;
        const u64 lb = sample_block_scan(lw[0] + lw[1], t1, s), hb = sample_block_scan(hw[0] + hw[1], t2, s);
        const u64 lc[3] = {lb, lb + lw[0], lb + lw[0] + lw[1]}, hc[3] = {hb, hb + hw[0], hb + hw[0] + hw[1]};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          // the first bin that may reach the target, and the first that must
          if ((static_cast<double>(hc[j]) < target || 2 * tid + j == 0) && static_cast<double>(hc[j + 1]) >= target) s.cmd.lo = 2 * tid + j;
          if ((static_cast<double>(lc[j]) < target || 2 * tid + j == 0) && static_cast<double>(lc[j + 1]) >= target) s.cmd.hi = 2 * tid + j;
        }
        __syncthreads();
        const int lo = s.cmd.lo, hi = s.cmd.hi;
        int c = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (2 * tid + j >= lo && 2 * tid + j <= hi) c += static_cast<int>(c2[j]);
        const u64 nl = sample_block_sum(static_cast<u64>(c), s);
        if (tid == 0) s.cmd.n = static_cast<int>(nl), s.cmd.total = total;
      }
      __syncthreads();
      if (tid == 0 && s.cmd.n > kSampleList) s.cmd.n = -1;
      __syncthreads();
      // the command to the other CTAs
      if (tid < static_cast<int>(sizeof(SampleCmd) / 8))
        for (int q = 1; q < cs; ++q)
          st_cluster_u64(remote(reinterpret_cast<u64*>(&s.cmd) + tid, q), reinterpret_cast<const u64*>(&s.cmd)[tid]);
    }
    cluster_sync_all();
    const SampleCmd cmd = s.cmd;
    if (cmd.n == -2) return false;             // top_k keeps everything
    if (cmd.n == -1) {
      if (k > 0) bisect(false, static_cast<u64>(k), 0.0);
      else bisect(true, 0, p * static_cast<double>(cmd.total));
      return k == 0;
    }
    // this CTA's listed tokens: their number from its own histogram, then their place in the list
    u64 c = 0;
    for (int b = cmd.lo + tid; b <= cmd.hi; b += kSampleThreads) c += cnt[b];
    c = sample_block_sum(c, s);
    if (tid < cs) st_cluster_u64(remote(&s.part[turn][cr], tid), c);
    if (tid == 0) s.count = 0;
    cluster_sync_all();                        // also: every histogram has been read, the list may overwrite it
    int at = 0;
    for (int q = 0; q < cr; ++q) at += static_cast<int>(s.part[turn][q]);
    turn ^= 1;
    u64 above = 0;                             // weight of the tokens above the list
    each([&](float x, int i) {
      const int b = sample_bin(x, r);
      if (b >= cmd.lo && b <= cmd.hi)
        st_cluster_u64(remote(list + at + atomicAdd(&s.count, 1), 0), sample_rank(x, i));
      else if (k == 0 && b < cmd.lo)
        above += sample_weight(x, r);
    });
    above = cluster_all(sample_block_sum(above, s));
    const bool both = k > 0 && by_p && cmd.lo == 0;   // the list begins at the top
    if (cr == 0) {
      int m = 32;                              // bitonic sort, descending, padded with zeros
      while (m < cmd.n) m <<= 1;
      for (int j = cmd.n + tid; j < m; j += kSampleThreads) list[j] = 0;
      __syncthreads();
      for (int size = 2; size <= m; size <<= 1)
        for (int d = size >> 1; d > 0; d >>= 1) {
          for (int j = tid; j < m / 2; j += kSampleThreads) {
            const int lo = 2 * j - (j & (d - 1)), hi = lo + d;
            const u64 x = list[lo], y = list[hi];
            if ((x < y) == ((lo & size) == 0)) list[lo] = y, list[hi] = x;
          }
          __syncthreads();
        }
      int last;                                // index of the last kept entry
      const int kk = k > 0 ? k - static_cast<int>(cmd.total) : cmd.n;
      if (k > 0 && !both) {
        last = kk - 1;
      } else {
        // entries 2 tid, 2 tid + 1: weight before each
        u64 w[2], tot;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          w[j] = 2 * tid + j < kk ? sample_weight(sample_unkey(static_cast<uint32_t>(list[2 * tid + j] >> 32)), r) : 0;
        const u64 before = sample_block_scan(w[0] + w[1], tot, s) + above;
        const double target = p * static_cast<double>(both ? tot : cmd.total);
        u64 kept = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          kept += 2 * tid + j < kk && static_cast<double>(before + (j ? w[0] : 0)) < target;
        last = max(static_cast<int>(sample_block_sum(kept, s)), 1) - 1;
      }
      if (tid < cs) st_cluster_u64(remote(&s.cmd.C, tid), list[last]);
    }
    cluster_sync_all();
    C = s.cmd.C;
    return k == 0 || both;
  };
  bool p_taken = !(p < 1.0);
  if (k > 0 && k < a.V) p_taken = cut(k, !p_taken) || p_taken;
  if (!p_taken) cut(0, true);

  // ------------------------------------------------ the draw, in vocabulary order: a warp has a contiguous part
  const int per = (((n + kSampleWarps - 1) / kSampleWarps) + 31) & ~31;
  const int j0 = min(n, warp * per), j1 = min(n, j0 + per);
  auto kept = [&](int j) -> u64 {
    const float x = j < j1 ? xs[j] : -INFINITY;
    if (!(x > -INFINITY) || sample_rank(x, i0 + j) < C) return 0ull;
    const u64 w = sample_weight(x, r);
    return x == r.mx || static_cast<double>(w) >= r.q ? w : 0ull;
  };
  u64 mine = 0;
  for (int j = j0 + lane; j < j1; j += 32) mine += kept(j);
  mine = sample_warp_reduce(mine, [](u64 x, u64 y) { return x + y; });
  __syncthreads();
  if (lane == 0) s.red[warp] = mine;
  __syncthreads();
  u64 before = 0, block = 0;
  for (int w = 0; w < kSampleWarps; ++w) {
    if (w < warp) before += s.red[w];
    block += s.red[w];
  }
  if (tid < cs) st_cluster_u64(remote(&s.part[turn][cr], tid), block);
  cluster_sync_all();                          // the last access to another CTA's memory
  u64 total = 0;
  for (int q = 0; q < cs; ++q) {
    if (q < cr) before += s.part[turn][q];
    total += s.part[turn][q];
  }
  const double u = static_cast<double>(a.u[row]);
  u64 target = u > 0.0 ? static_cast<u64>(fmin(u, 1.0) * static_cast<double>(total)) : 0ull;
  if (target >= total) target = total - 1;
  if (before <= target && target < before + mine) {
    for (int jb = j0; jb < j1; jb += 32) {
      const int j = jb + lane;
      const u64 w = kept(j);
      u64 incl = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, before + incl > target);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
          a.out_idx[row] = i0 + j;
          if (a.out_logp)
            a.out_logp[row] = static_cast<float>(log(static_cast<double>(w) / static_cast<double>(total)));
        }
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
}

}  // namespace tps
