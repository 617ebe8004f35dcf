// tps_sample.cuh -- sampling one token per row of logits from given uniform numbers:
// temperature, then top-k, then top-p over what is left, then min-p, then the inverse
// of the running sum of the kept weights in vocabulary order.
//
// w_i = exp((l_i - max) / T) as an integer in units of 2^-44. Sums of integers are exact
// and do not depend on the order of the additions, and they agree with 64-bit floating
// point to half a unit per token; a float sum would let the rounding of a sum over
// 128256 tokens decide which token a uniform number falls on.
//
// Every filter keeps a top part of the order (logit descending, index ascending), so a
// row's filters are one threshold, the last kept token, and no sort of the row is needed.
// One thread-block cluster holds a row in the shared memory of its CTAs (fp32, read once
// from HBM) and finds the threshold from a histogram of 1024 equal bins over the logits
// within 32 T of the maximum (what lies below has no weight): counts for top-k, exact
// weights for top-p, so the bin that holds the cut is known. The tokens of that bin go to
// the first CTA. When the k largest fit its list of 1024 it takes both cuts there, and with
// up to 256 of them it draws there too: each token finds its own place by comparing itself
// with the others, which needs no sort and no further step of the cluster. Where the bin
// holds more than the list (equal logits, one far outlier that stretches the bins), the
// threshold is found bit by bit from passes over shared memory.
//
// Bound by latency for few rows (six cluster barriers of about a microsecond) and by the
// 64-bit exponentials and the passes over shared memory for many.
#pragma once

#include <cstdint>

namespace tps {

typedef unsigned long long u64;

constexpr int kSampleThreads = 512;
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int kSampleBins = 1024;
constexpr int kSampleList = 1024;              // entries of the candidate list, which overlays the histogram's weights
constexpr u64 kSampleOne = 1ull << 44;         // weight of the largest logit
constexpr int kSampleSmall = 256;              // kept tokens that the first CTA draws from by itself

__device__ __forceinline__ uint32_t atomic_add_cluster_u32(uint32_t addr, uint32_t x) {
  uint32_t v;
  asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(v) : "r"(addr), "r"(x) : "memory");
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
  float mx;                    // largest logit
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
  int drawn;                   // the row is finished
  u64 C;                       // the last kept token's rank
  u64 total;                   // top-k: tokens above the list; top-p: the weight of all
};

struct SampleSmem {
  u64 red[kSampleWarps];
  u64 part[2][8];              // values that the CTAs of the cluster exchange, two in turn
  u64 top[8];
  SampleCmd cmd;
  int listed;                  // first CTA: list entries handed out to the CTAs
  int place;                   // next free entry of this CTA's
  float fred[2 * kSampleWarps];
};

constexpr int kSampleHead = (static_cast<int>(sizeof(SampleSmem)) + 15) / 16 * 16;
constexpr int sample_smem_bytes(int slice) { return kSampleHead + kSampleBins * 12 + slice * 4; }

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
  u64* mass = reinterpret_cast<u64*>(smem_raw + kSampleHead);
  u64* list = mass;
  uint32_t* cnt = reinterpret_cast<uint32_t*>(mass + kSampleBins);
  float* xs = reinterpret_cast<float*>(cnt + kSampleBins);
  static_assert(kSampleList <= kSampleBins && kSampleBins == 2 * kSampleThreads, "shared memory layout");

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cs = static_cast<int>(cluster_nctarank()), cr = static_cast<int>(cluster_ctarank());
  const int row = static_cast<int>(blockIdx.x) / cs;
  const int i0 = min(a.V, cr * a.slice), n = min(a.V, i0 + a.slice) - i0;   // this CTA's tokens [i0, i0 + n)
  // address of the same place in CTA r of the cluster
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
  auto take = [&](float x) {
    mx = fmaxf(mx, x);
    mn = fminf(mn, x > -INFINITY ? x : INFINITY);
  };
  if (a.f32) {
    const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) +
                                                        static_cast<long long>(row) * a.V + i0);
#pragma unroll 8
    for (int v = tid; v < n / 4; v += kSampleThreads) {
      float4 x = __ldcs(src + v);
      x = make_float4(sample_clean(x.x), sample_clean(x.y), sample_clean(x.z), sample_clean(x.w));
      reinterpret_cast<float4*>(xs)[v] = x;
      take(x.x), take(x.y), take(x.z), take(x.w);
    }
  } else {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.logits) +
                                                      static_cast<long long>(row) * a.V + i0);
#pragma unroll 4
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
      for (int j = 0; j < 8; ++j) take(x[j]);
    }
  }
  for (int j = tid; j < kSampleBins; j += kSampleThreads) cnt[j] = 0, mass[j] = 0;
  if (tid == 0) s.listed = s.cmd.drawn = 0;
  mx = sample_warp_reduce(mx, [](float x, float y) { return fmaxf(x, y); });
  mn = sample_warp_reduce(mn, [](float x, float y) { return fminf(x, y); });
  if (lane == 0) s.fred[warp] = mx, s.fred[kSampleWarps + warp] = mn;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSampleWarps; ++w) {
    mx = fmaxf(mx, s.fred[w]);
    mn = fminf(mn, s.fred[kSampleWarps + w]);
  }
  if (tid < cs)
    st_cluster_u64(remote(&s.top[cr], tid), static_cast<u64>(__float_as_uint(mx)) << 32 | __float_as_uint(mn));
  cluster_sync_all();
  for (int r = 0; r < cs; ++r) {
    mx = fmaxf(mx, __uint_as_float(static_cast<uint32_t>(s.top[r] >> 32)));
    mn = fminf(mn, __uint_as_float(static_cast<uint32_t>(s.top[r])));
  }

  const float T = a.temperature ? a.temperature[row] : 1.0f;
  const float pf = a.top_p ? a.top_p[row] : 1.0f;
  const int top_k = a.top_k ? a.top_k[row] : 0;
  const double u = fmin(fmax(static_cast<double>(a.u[row]), 0.0), 1.0);    // NaN: 0
  const bool greedy = !(T > 0.0f);
  float cx = -INFINITY;                        // kept: x > cx, or x == cx and index <= ci (and min_p)
  int ci = -1;
  auto each = [&](auto f) {                    // every kept token of this CTA (never a logit of -inf)
    for (int v = tid; v < n / 4; v += kSampleThreads) {
      const float4 q = reinterpret_cast<const float4*>(xs)[v];
      const float x[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (x[j] > cx || (x[j] == cx && i0 + 4 * v + j <= ci)) f(x[j], i0 + 4 * v + j);
    }
  };
  if (greedy || mx == -INFINITY) {             // the same in the whole cluster
    int arg = 0x7fffffff;
    if (mx > -INFINITY)
      each([&](float x, int i) {
        if (x == mx) arg = min(arg, i);
      });
    arg = sample_warp_reduce(arg, [](int x, int y) { return min(x, y); });
    __syncthreads();
    if (lane == 0) s.red[warp] = static_cast<u64>(arg);
    __syncthreads();
    for (int w = 0; w < kSampleWarps; ++w) arg = min(arg, static_cast<int>(s.red[w]));
    if (tid == 0) st_cluster_u64(remote(&s.part[0][cr], 0), static_cast<u64>(arg));
    cluster_sync_all();
    if (cr == 0 && tid == 0) {
      for (int r = 0; r < cs; ++r) arg = min(arg, static_cast<int>(s.part[0][r]));
      a.out_idx[row] = mx > -INFINITY ? arg : -1;
      if (a.out_logp) a.out_logp[row] = mx > -INFINITY ? 0.0f : -INFINITY;
    }
    return;
  }
  SampleRow r;
  r.mx = mx;
  r.c = 1.4426950408889634 / static_cast<double>(T);
  r.q = a.min_p ? static_cast<double>(a.min_p[row]) * static_cast<double>(kSampleOne) : 0.0;
  const float range = fminf(mx - mn, 32.0f * T);
  r.bin_scale = range > 0.0f ? static_cast<float>(kSampleBins - 1) / range : 0.0f;
  const double p = static_cast<double>(pf);
  auto survives = [&](u64 w) { return w == kSampleOne || static_cast<double>(w) >= r.q; };   // min_p
  auto goal = [&](u64 total) {                 // the draw falls on the token whose running sum exceeds this
    const u64 t = static_cast<u64>(u * static_cast<double>(total));
    return t < total ? t : total - 1;
  };
  auto draw = [&](int i, u64 w, u64 total) {
    a.out_idx[row] = i;
    if (a.out_logp) a.out_logp[row] = static_cast<float>(log(static_cast<double>(w) / static_cast<double>(total)));
  };

  // Largest threshold at which `want` tokens (or, by weight, `target`) are kept, bit by bit.
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
    return t;
  };
  auto set_threshold = [&](u64 rank) {
    const float x = sample_unkey(static_cast<uint32_t>(rank >> 32));
    const int i = static_cast<int>(0xffffffffu - static_cast<uint32_t>(rank));
    if (x > cx || (x == cx && i < ci)) cx = x, ci = i;
  };

  // One cut of the kept tokens: the k first of them (k > 0), or those that reach the share p
  // of their weight. With by_p the cut to k may take p, or the draw, in the same step:
  // returns what is left to do.
  enum { NOTHING, DRAW, CUT_P };
  auto cut = [&](int k, bool by_p) -> int {
    u64 sum = 0;
    each([&](float x, int) {
      const int b = sample_bin(x, r);
      atomicAdd(cnt + b, 1u);
      if (k == 0) {
        const u64 w = sample_weight(x, r);
        sum += w;
        if (w) atomicAdd(mass + b, w);
      }
    });
    if (k == 0) sum = sample_block_sum(sum, s);
    else __syncthreads();
    const u64 total = cluster_all(sum);
    if (cr == 0) {
      // bins 2 tid and 2 tid + 1 over the cluster: what lies before each, in tokens or weight
      u64 c2[2] = {0, 0}, v2[2] = {0, 0}, all;
#pragma unroll 4
      for (int q = 0; q < cs; ++q) {
        const u64 c = ld_cluster_u64(remote(cnt + 2 * tid, q));
        c2[0] += c & 0xffffffffu, c2[1] += c >> 32;
        if (k == 0) {
          v2[0] += ld_cluster_u64(remote(mass + 2 * tid, q));
          v2[1] += ld_cluster_u64(remote(mass + 2 * tid + 1, q));
        }
      }
      if (k > 0) v2[0] = c2[0], v2[1] = c2[1];
      const u64 before = sample_block_scan(v2[0] + v2[1], all, s);
      const u64 cum[3] = {before, before + v2[0], before + v2[0] + v2[1]};
      if (tid == 0) s.cmd.n = -2;              // k >= the number of tokens
      __syncthreads();
      const double target = k > 0 ? static_cast<double>(k) : p * static_cast<double>(total);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        // the bin in which the running value reaches the target (the first that has any for a target of 0)
        const bool reaches = v2[j] > 0 && static_cast<double>(cum[j + 1]) >= target &&
                             (cum[j] == 0 || static_cast<double>(cum[j]) < target);
        if (reaches && (k == 0 || static_cast<u64>(k) < all)) {
          const bool from0 = k > 0 && cum[j + 1] <= kSampleList;   // every kept token fits the list
          s.cmd.lo = from0 ? 0 : 2 * tid + j;
          s.cmd.hi = 2 * tid + j;
          const u64 len = from0 ? cum[j + 1] : c2[j];
          s.cmd.n = len > kSampleList ? -1 : static_cast<int>(len);
          s.cmd.total = k == 0 ? total : from0 ? 0 : cum[j];
          s.cmd.C = k == 0 ? cum[j] : 0;       // weight above the list
        }
      }
      __syncthreads();
      // the command to the other CTAs
      if (tid < static_cast<int>(sizeof(SampleCmd) / 8))
        for (int q = 1; q < cs; ++q)
          st_cluster_u64(remote(reinterpret_cast<u64*>(&s.cmd) + tid, q), reinterpret_cast<const u64*>(&s.cmd)[tid]);
    }
    cluster_sync_all();                        // also: the histograms' weights have been read, the list may overwrite them
    const SampleCmd cmd = s.cmd;
    const int after = by_p && k > 0 ? CUT_P : DRAW;
    if (cmd.n < 0) {
      if (cmd.n == -1)
        set_threshold(k > 0 ? bisect(false, static_cast<u64>(k), 0.0)
                            : bisect(true, 0, p * static_cast<double>(cmd.total)));
      for (int j = tid; j < kSampleBins; j += kSampleThreads) cnt[j] = 0, mass[j] = 0;
      __syncthreads();
      return after;
    }
    // this CTA's place in the list: as many entries as its own histogram says
    u64 c = 0;
    for (int b = cmd.lo + tid; b <= cmd.hi; b += kSampleThreads) c += cnt[b];
    c = sample_block_sum(c, s);
    if (tid == 0) s.place = c ? static_cast<int>(atomic_add_cluster_u32(remote(&s.listed, 0), static_cast<uint32_t>(c))) : 0;
    __syncthreads();
    if (c)
      each([&](float x, int i) {
        const int b = sample_bin(x, r);
        if (b >= cmd.lo && b <= cmd.hi) st_cluster_u64(remote(list + atomicAdd(&s.place, 1), 0), sample_rank(x, i));
      });
    for (int j = tid; j < kSampleBins; j += kSampleThreads) {   // for a second cut
      cnt[j] = 0;
      if (cr > 0) mass[j] = 0;
    }
    cluster_sync_all();
    const bool whole = k > 0 && cmd.lo == 0;   // the list begins at the top
    if (cr == 0) {
      const int len = cmd.n;
      if (whole && len <= kSampleSmall) {
        // Two threads per token e: how many tokens come before it and their weight, then the
        // weight of the kept tokens up to it in vocabulary order.
        const int e = tid >> 1, half = tid & 1;
        const u64 re = e < len ? list[e] : 0;
        const u64 we = e < len ? sample_weight(sample_unkey(static_cast<uint32_t>(re >> 32)), r) : 0;
        u64* w = list + kSampleSmall;          // weights, by list entry (each pair writes its own)
        if (half == 0) w[e] = we;
        __syncthreads();
        int place = 0;
        u64 above = 0;
        for (int j = half; j < len; j += 2)
          if (list[j] > re) ++place, above += w[j];
        place += __shfl_xor_sync(0xffffffffu, place, 1);
        above += __shfl_xor_sync(0xffffffffu, above, 1);
        bool in = e < len && place < k;
        if (by_p) {
          const u64 wk = sample_block_sum(in && half == 0 ? we : 0, s);
          in = in && (place == 0 || static_cast<double>(above) < p * static_cast<double>(wk));
        }
        in = in && survives(we);
        __syncthreads();
        if (half == 0) w[e] = in ? we : 0;
        const u64 tot = sample_block_sum(in && half == 0 ? we : 0, s);
        const uint32_t ie = static_cast<uint32_t>(re);           // ~index: larger is earlier
        u64 upto = 0;
        for (int j = half; j < len; j += 2)
          if (static_cast<uint32_t>(list[j]) >= ie) upto += w[j];
        upto += __shfl_xor_sync(0xffffffffu, upto, 1);
        const u64 t = goal(tot);
        if (in && half == 0 && upto > t && upto - we <= t) draw(static_cast<int>(0xffffffffu - ie), we, tot);
        if (tid < cs) {
          SampleCmd done = cmd;
          done.drawn = 1;
          st_cluster_u64(remote(&s.cmd.n, tid), reinterpret_cast<const u64*>(&done)[1]);
        }
      } else {
        int m = 32;                            // bitonic sort, descending, padded with zeros
        while (m < len) m <<= 1;
        for (int j = len + tid; j < m; j += kSampleThreads) list[j] = 0;
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
        const int kk = k > 0 ? k - static_cast<int>(cmd.total) : len;   // entries that may stay
        int last = kk - 1;                     // the last kept one
        if (k == 0 || (whole && by_p)) {
          u64 w[2], tot;                       // entries 2 tid and 2 tid + 1: the weight before each
#pragma unroll
          for (int j = 0; j < 2; ++j)
            w[j] = 2 * tid + j < kk ? sample_weight(sample_unkey(static_cast<uint32_t>(list[2 * tid + j] >> 32)), r) : 0;
          const u64 before = sample_block_scan(w[0] + w[1], tot, s) + (k == 0 ? cmd.C : 0);
          const double target = p * static_cast<double>(k == 0 ? cmd.total : tot);
          u64 kept = 0;
#pragma unroll
          for (int j = 0; j < 2; ++j)
            kept += 2 * tid + j < kk && static_cast<double>(before + (j ? w[0] : 0)) < target;
          last = max(static_cast<int>(sample_block_sum(kept, s)), 1) - 1;
        }
        const u64 C = list[last];
        __syncthreads();
        if (tid < cs) st_cluster_u64(remote(&s.cmd.C, tid), C);
        for (int j = tid; j < kSampleBins; j += kSampleThreads) mass[j] = 0;
        if (tid == 0) s.listed = 0;
      }
    }
    cluster_sync_all();
    if (s.cmd.drawn) return NOTHING;
    set_threshold(s.cmd.C);
    return whole ? DRAW : after;
  };
  const bool by_p = p < 1.0;
  int left = by_p ? CUT_P : DRAW;
  if (top_k > 0 && top_k < a.V) left = cut(top_k, by_p);
  if (left == CUT_P) left = cut(0, true);
  if (left == NOTHING) return;

  // ------------------------------------------------ the draw, in vocabulary order: a warp has a contiguous part
  const int per = (((n + kSampleWarps - 1) / kSampleWarps) + 31) & ~31;
  const int j0 = min(n, warp * per), j1 = min(n, j0 + per);
  auto kept = [&](int j) -> u64 {
    const float x = j < j1 ? xs[j] : -INFINITY;
    if (!(x > cx || (x == cx && i0 + j <= ci))) return 0ull;
    const u64 w = sample_weight(x, r);
    return survives(w) ? w : 0ull;
  };
  u64 mine = 0;
#pragma unroll 4
  for (int j = j0 + lane; j < j1; j += 32) mine += kept(j);
  mine = sample_warp_reduce(mine, [](u64 x, u64 y) { return x + y; });
  __syncthreads();
  if (lane == 0) s.red[warp] = mine;
  __syncthreads();
  u64 before = 0, block = 0;
#pragma unroll
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
  const u64 target = goal(total);
  if (before <= target && target < before + mine) {
    for (int jb = j0; jb < j1; jb += 32) {
      const u64 w = kept(jb + lane);
      u64 incl = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, before + incl > target);
      if (hit) {
        if (lane == __ffs(hit) - 1) draw(i0 + jb + lane, w, total);
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
}

}  // namespace tps
