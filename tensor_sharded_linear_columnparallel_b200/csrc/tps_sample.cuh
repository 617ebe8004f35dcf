// tps_sample.cuh -- sampling one token per row of logits from given uniform numbers:
// temperature, then top-k, then top-p over what is left, then min-p, then the inverse
// of the running sum of the kept weights in vocabulary order.
//
// w_i = exp((l_i - max) / T) as an integer in units of 2^-44, within 2^-36 of itself and half
// a unit. Sums of integers are exact and do not depend on the order of the additions; a float
// sum would let the rounding of a sum over 128256 tokens decide which token a uniform number
// falls on.
//
// Every filter keeps a top part of the order (logit descending, index ascending), so a
// row's filters are one threshold, the last kept token, and no sort of the row is needed.
// One thread-block cluster holds a row in the shared memory of its CTAs (in its own type,
// read once from HBM) and finds the threshold in steps that end in a short list:
//  - top-k: each thread has kept the largest logit of its part of the row. The k-th largest
//    of those is a lower bound of the k-th largest logit, so their histogram (an entry per
//    thread, not per token) gives a bin down to which all k lie, with few others.
//  - top-p: a histogram of fast approximate weights, as 16-bit numbers with a shift per
//    octave of bins, so that a bin's 32-bit sum keeps its relative precision. It tells the
//    bin of the cut but for roundings; the one pass that computes the exact weights, of all
//    tokens and of those above the bin, tells whether it is that bin or the one beside it.
// The tokens of those bins go to a list, each CTA's part first in its own memory, then all in
// the first CTA, which takes the cut from exact sums (sample_select), for top-k that of top-p
// too. With a list of up to 256 tokens from the top it draws there: each token finds its own place
// by comparing itself with the others, without a sort. After a cut to p it sends the weights
// of the list's kept tokens to the warps whose tokens they are, so that the draw needs no pass
// over the row. Bins are equal parts of the logits within 32 T of the maximum (what lies below
// has no weight). Where the cut's bin holds more than the list of 1024, the threshold is found
// bit by bit from 64 passes over shared memory: with many equal logits, an outlier that stretches
// the bins (masks do not, see there), and in large vocabularies, whose bins hold more. Normal
// logits cut to p: never at 151936, some rows at 202048, most from 262144 on, where 8 rows then
// take 980 us instead of 34.
//
// Bound by latency for few rows: of the 46,000 cycles of one of 8 rows of 128256 bf16 logits cut
// to p (512 threads, eight CTAs), 4,000 load it, 7,600 fill the histogram, 3,700 find the bin,
// 10,000 sum the exact weights, 8,000 cut the list, and six cluster barriers take about 1,100
// each. For many rows by the instructions of the two passes: an approximate and a 64-bit
// exponential and a shared-memory atomic per token. With all filters and 64 rows 43 us, where
// reading the logits takes 2.5.
#pragma once

#include <cstddef>
#include <cstdint>

namespace tps {

typedef unsigned long long u64;

constexpr int kSampleMaxWarps = 16;
constexpr int kSampleBins = 1024;
constexpr int kSampleList = 1024;              // entries of the candidate list, whose second half overlays the histogram
constexpr u64 kSampleOne = 1ull << 44;         // weight of the largest logit
constexpr int kSampleFew = 64;                 // entries that sample_select compares with one another
constexpr int kSampleSmall = 256;              // kept tokens that the first CTA draws from by itself
constexpr float kSampleSpan = 46.2f;           // 32 log2(e): logits this many factors of 2 below the largest have no weight

__device__ __forceinline__ void atomic_add_cluster_u64(uint32_t addr, u64 x) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u64 [%0], %1;" ::"r"(addr), "l"(x) : "memory");
}
// N consecutive words of another CTA's shared memory (N = 2 or 4).
template <int N>
__device__ __forceinline__ void ld_cluster(uint32_t addr, uint32_t (&v)[N]) {
  if constexpr (N == 4)
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(addr)
                 : "memory");
  else
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(addr) : "memory");
}
__device__ __forceinline__ u64 ld_cluster_u64(uint32_t addr) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// Unsigned key with the order of the floats, -0 as +0 (never called with a NaN).
__device__ __forceinline__ uint32_t sample_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float sample_unkey(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}
__device__ __forceinline__ u64 sample_rank(float x, int i) {
  return static_cast<u64>(sample_key(x)) << 32 | (0xffffffffu - static_cast<uint32_t>(i));
}

// Four consecutive logits of a row part in shared memory, held in the type that they came in.
__device__ __forceinline__ void sample_get4(const float* xs, int v, float (&x)[4]) {
  const float4 q = reinterpret_cast<const float4*>(xs)[v];
  x[0] = q.x, x[1] = q.y, x[2] = q.z, x[3] = q.w;
}
__device__ __forceinline__ void sample_get4(const __nv_bfloat16* xs, int v, float (&x)[4]) {
  const uint2 q = reinterpret_cast<const uint2*>(xs)[v];
  x[0] = __uint_as_float(q.x << 16), x[1] = __uint_as_float(q.x & 0xffff0000u);
  x[2] = __uint_as_float(q.y << 16), x[3] = __uint_as_float(q.y & 0xffff0000u);
}
__device__ __forceinline__ void sample_put4(float* xs, int v, const float (&x)[4]) {
  reinterpret_cast<float4*>(xs)[v] = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void sample_put4(__nv_bfloat16* xs, int v, const float (&x)[4]) {   // bf16 values: exact
  reinterpret_cast<uint2*>(xs)[v] =
      make_uint2(__float_as_uint(x[0]) >> 16 | __float_as_uint(x[1]), __float_as_uint(x[2]) >> 16 | __float_as_uint(x[3]));
}

struct SampleRow {             // one row's parameters, the same in every CTA of its cluster
  double mx, c;                // largest logit; log2(e) / T
  float mxf;                   // largest logit
  float bin_scale;             // bins per logit: 2^octave of them per factor of 2 in the weight
  int octave;                  // (31 for more: all bins are within one factor)
  u64 q;                       // min_p in units of 2^-44
};

// exp((x - mx) / T) in units of 2^-44, without a branch: 2^-y with y = (mx - x) log2(e) / T =
// n + f, f in [-1/2, 1/2], 2^-f as its Taylor sum to (f ln 2)^9 / 9! (the rest is below
// 2^-37), the power of two put into the exponent field, and the integer read from the low
// bits after adding 2^52. The largest logit gives exactly 2^44; a y above 46 (or a NaN)
// counts as 46, whose weight rounds to 0: the weight of -inf and of NaN.
__device__ __forceinline__ u64 sample_weight(float x, const SampleRow& r) {
  const double y = fmin((r.mx - static_cast<double>(x)) * r.c, 46.0);
  const double t = y + 6755399441055744.0;                  // 1.5 * 2^52: y rounded to an integer, in the low bits
  const double f = (t - 6755399441055744.0) - y;
  double p = 1.0178086009239700e-07;                        // ln(2)^k / k!, k = 9 ... 0
  p = fma(p, f, 1.3215486790144310e-06);
  p = fma(p, f, 1.5252733804059841e-05);
  p = fma(p, f, 1.5403530393381610e-04);
  p = fma(p, f, 1.3333558146428443e-03);
  p = fma(p, f, 9.6181291076284770e-03);
  p = fma(p, f, 5.5504108664821580e-02);
  p = fma(p, f, 2.4022650695910072e-01);
  p = fma(p, f, 6.9314718055994530e-01);
  p = fma(p, f, 1.0);
  const double v = __hiloint2double(__double2hiint(p) + ((44 - __double2loint(t)) << 20), __double2loint(p));
  const double m = v + 4503599627370496.0;                  // 2^52
  return static_cast<u64>(static_cast<uint32_t>(__double2hiint(m)) & 0xfffffu) << 32 |
         static_cast<uint32_t>(__double2loint(m));
}

// A float in [0, 2^23) rounded to an integer, and an integer as a float, by an addition of 2^23:
// the conversions go through the unit of the exponential, which bounds the pass over the row.
__device__ __forceinline__ uint32_t sample_round(float x) { return __float_as_uint(x + 8388608.0f) - 0x4b000000u; }
__device__ __forceinline__ float sample_float(uint32_t i) { return __uint_as_float(i + 0x4b000000u) - 8388608.0f; }

// Bin of a logit: 0 holds the largest, the last one everything beyond.
__device__ __forceinline__ int sample_bin(float x, const SampleRow& r) {
  return static_cast<int>(sample_round(fminf((r.mxf - x) * r.bin_scale, static_cast<float>(kSampleBins - 1))));
}
// Weights of bin b are below 2^(15.1 + shift): the bins of an octave, and half a bin (at most
// 1/32 octave) of the one before.
__device__ __forceinline__ int sample_shift(int b, const SampleRow& r) { return max(0, 29 - (b >> r.octave)); }

enum { SAMPLE_CUT, SAMPLE_DRAWN, SAMPLE_SHORT, SAMPLE_DOWN, SAMPLE_UP };   // threshold C; row finished; list too
                                                                           // short; the cut is in a bin before / behind
// What the first CTA tells the others about the next step (one copy per CTA).
struct SampleCmd {
  int lo, hi;                  // bins whose tokens are listed
  int skip;                    // nothing to list: 1 the cut keeps everything
  int result;                  // after the list: one of SAMPLE_*
  u64 C;                       // the last kept token's rank
  u64 total;                   // top-k: tokens above the list
};

struct SampleSmem {
  u64 red[kSampleMaxWarps];
  u64 part[2][8];              // values that the CTAs of the cluster exchange, two in turn
  u64 part2[2][8];
  u64 top[8], have[8];
  u64 wsum[kSampleMaxWarps];   // after a cut to p: weight of the warps' drawable tokens of the list
  SampleCmd cmd;
  int listed;                  // entries of this CTA's part of the list
  int members;                 // first CTA, sample_select: what is left of the list
  u64 pivot[32], few[kSampleFew], found;
  uint32_t bucket[2][33];
  float fred[2 * kSampleMaxWarps];
};

constexpr int kSampleHead = (static_cast<int>(sizeof(SampleSmem)) + 15) / 16 * 16;
constexpr int sample_smem_bytes(int slice, int f32) { return kSampleHead + kSampleBins * 8 + slice * (f32 ? 4 : 2); }

template <bool B>
struct SampleFlag {
  static constexpr bool value = B;
};

template <class T, class Op>
__device__ __forceinline__ T sample_warp_reduce(T v, Op op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
// Sum over the block, in every thread.
template <int THREADS>
__device__ __forceinline__ u64 sample_block_sum(u64 v, SampleSmem& s) {
  v = sample_warp_reduce(v, [](u64 x, u64 y) { return x + y; });
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s.red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < THREADS / 32 ? s.red[threadIdx.x & 31] : 0;
  return sample_warp_reduce(v, [](u64 x, u64 y) { return x + y; });
}
// Exclusive sum over the block, and the total.
template <int THREADS>
__device__ __forceinline__ u64 sample_block_scan(u64 v, u64& total, SampleSmem& s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto scan = [&](u64 x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 n = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += n;
    }
    return x;
  };
  const u64 incl = scan(v);
  __syncthreads();
  if (lane == 31) s.red[warp] = incl;
  __syncthreads();
  const u64 w = lane < THREADS / 32 ? s.red[lane] : 0;
  const u64 ws = scan(w);
  total = __shfl_sync(0xffffffffu, ws, 31);
  return __shfl_sync(0xffffffffu, ws - w, warp) + incl - v;
}

// The entry v of a list (BPT per thread, those with a weight w) with which the running sum of
// the weights, from the largest entry down and beginning at S, reaches target: S < target <=
// S + all weights. 32 entries cut the list into 33 buckets; the one that has the entry (a 33rd of
// the list, give or take) is what is left, until few enough are left to compare each with all.
// Sums are exact, as two halves of 22 bits of up to 993 weights in a bucket. Sorting the
// list instead took 55 steps of 330 cycles for 1024 entries, 9 us; this takes 3 to 5.
template <int THREADS, int BPT>
__device__ __forceinline__ u64 sample_select(const u64 (&v)[BPT], const u64 (&w)[BPT], u64 S, double target, u64* list,
                                             SampleSmem& s) {
  const int tid = threadIdx.x, lane = tid & 31;
  bool in[BPT];
#pragma unroll
  for (int j = 0; j < BPT; ++j) in[j] = w[j] > 0;
  for (;;) {
    __syncthreads();
    if (tid == 0) s.members = 0;
    if (tid < 66) s.bucket[tid >= 33][tid >= 33 ? tid - 33 : tid] = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < BPT; ++j) {
      const uint32_t m = __ballot_sync(0xffffffffu, in[j]);
      int at = 0;
      if (lane == 0 && m) at = atomicAdd(&s.members, __popc(m));
      at = __shfl_sync(0xffffffffu, at, 0) + __popc(m & ((1u << lane) - 1u));
      if (in[j]) {
        list[at] = v[j];
        if (at < kSampleFew) s.few[at] = w[j];
      }
    }
    __syncthreads();
    const int n = s.members;
    if (n <= kSampleFew) break;
    if (tid < 32) {
      const u64 mine = list[lane * n >> 5];
      int place = 0;
#pragma unroll 8
      for (int i = 0; i < 32; ++i) place += list[i * n >> 5] > mine;
      s.pivot[place] = mine;
    }
    __syncthreads();
    int b[BPT];
#pragma unroll
    for (int j = 0; j < BPT; ++j) {
      b[j] = 0;                                // pivots above the entry
      if (in[j]) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          if (s.pivot[b[j] + o - 1] > v[j]) b[j] += o;
        if (s.pivot[b[j]] > v[j]) ++b[j];
        atomicAdd(&s.bucket[0][b[j]], static_cast<uint32_t>(w[j]) & 0x3fffffu);
        atomicAdd(&s.bucket[1][b[j]], static_cast<uint32_t>(w[j] >> 22));
      }
    }
    __syncthreads();
    const u64 mine = s.bucket[0][lane] + (static_cast<u64>(s.bucket[1][lane]) << 22);
    u64 incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, static_cast<double>(S + incl) >= target);
    const int sel = hit ? __ffs(hit) - 1 : 32;
    S += __shfl_sync(0xffffffffu, hit ? incl - mine : incl, hit ? sel : 31);
#pragma unroll
    for (int j = 0; j < BPT; ++j) in[j] = in[j] && b[j] == sel;
  }
  if (tid < s.members) {
    const u64 mine = list[tid];
    u64 before = S;
#pragma unroll 4
    for (int i = 0; i < s.members; ++i) before += list[i] > mine ? s.few[i] : 0;
    if (static_cast<double>(before) < target && static_cast<double>(before + s.few[tid]) >= target) s.found = mine;
  }
  __syncthreads();
  return s.found;
}

template <class E, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) tps_sample_kernel(const SampleArgs a) {
  constexpr int WARPS = THREADS / 32;
  constexpr int BPT = kSampleBins / THREADS;     // bins (and list entries) per thread
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SampleSmem& s = *reinterpret_cast<SampleSmem*>(smem_raw);
  u64* list = reinterpret_cast<u64*>(smem_raw + kSampleHead);
  uint32_t* hist = reinterpret_cast<uint32_t*>(list + kSampleList / 2);
  E* xs = reinterpret_cast<E*>(hist + kSampleBins);
  static_assert(kSampleList * 8 == kSampleBins * 8 && kSampleSmall <= THREADS && (BPT == 2 || BPT == 4),
                "shared memory layout");

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cs = static_cast<int>(cluster_nctarank()), cr = static_cast<int>(cluster_ctarank());
  const int row = static_cast<int>(blockIdx.x) / cs;
  const int i0 = min(a.V, cr * a.slice), n = min(a.V, i0 + a.slice) - i0;   // this CTA's tokens [i0, i0 + n)
  // address of the same place in CTA r of the cluster
  auto remote = [&](const void* p, int r) { return mapa_shared(smem_u32(p), static_cast<uint32_t>(r)); };
  int turn = 0;
  // sums of two values per CTA, in every CTA (the same in all threads of a CTA)
  auto cluster_all2 = [&](u64 v, u64& v2) {
    if (tid < cs) {
      st_cluster_u64(remote(&s.part[turn][cr], tid), v);
      st_cluster_u64(remote(&s.part2[turn][cr], tid), v2);
    }
    cluster_sync_all();
    u64 t = 0;
    v2 = 0;
    for (int r = 0; r < cs; ++r) t += s.part[turn][r], v2 += s.part2[turn][r];
    turn ^= 1;
    return t;
  };
  auto cluster_all = [&](u64 v) {
    u64 none = 0;
    return cluster_all2(v, none);
  };
  cluster_arrive();                            // waited for before the first access to another CTA's memory
  griddep_wait();
  const float T = a.temperature ? a.temperature[row] : 1.0f;
  const float pf = a.top_p ? a.top_p[row] : 1.0f;
  const float qf = a.min_p ? a.min_p[row] : 0.0f;
  const int top_k = a.top_k ? a.top_k[row] : 0;
  const double u = fmin(fmax(static_cast<double>(a.u[row]), 0.0), 1.0);    // NaN: 0
  const bool greedy = !(T >= 7.888609e-31f);   // 2^-100: the bins' scale stays finite
  // what needs 64-bit arithmetic and not the row: ahead of the loads that it can wait for
  SampleRow r;
  r.c = 1.4426950408889634 / static_cast<double>(T);
  r.q = qf > 0.0f ? static_cast<u64>(ceil(fmin(static_cast<double>(qf), 1.0) * static_cast<double>(kSampleOne))) : 0;
  const float cf = static_cast<float>(r.c);

  // ------------------------------------------------ the row into shared memory, its largest and smallest logit
  float mx = -INFINITY, mn = INFINITY;         // neither takes a NaN
  const E* src = static_cast<const E*>(a.logits) + static_cast<long long>(row) * a.V + i0;
  constexpr int EPV = 16 / sizeof(E);
  for (int v0 = tid; v0 < n / EPV; v0 += 8 * THREADS) {
    uint4 in[8];                               // 8 loads in flight, in the last round too
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (v0 + c * THREADS < n / EPV) in[c] = __ldcs(reinterpret_cast<const uint4*>(src) + v0 + c * THREADS);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (v0 + c * THREADS >= n / EPV) break;
      reinterpret_cast<uint4*>(xs)[v0 + c * THREADS] = in[c];
      const uint32_t w[4] = {in[c].x, in[c].y, in[c].z, in[c].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x = __uint_as_float(EPV == 4 ? w[j] : w[j] & 0xffff0000u);
        const float y = EPV == 4 ? x : __uint_as_float(w[j] << 16);
        mx = fmaxf(fmaxf(mx, x), y);
        mn = fminf(fminf(mn, x), y);
      }
    }
  }
  float most = mx;                             // this thread's largest
  for (int j = tid; j < kSampleBins; j += THREADS) hist[j] = 0;
  if (tid == 0) s.listed = 0;
  if (tid < WARPS) s.wsum[tid] = 0;
  mx = sample_warp_reduce(mx, [](float x, float y) { return fmaxf(x, y); });
  mn = sample_warp_reduce(mn, [](float x, float y) { return fminf(x, y); });
  if (lane == 0) s.fred[warp] = mx, s.fred[WARPS + warp] = mn;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    mx = fmaxf(mx, s.fred[w]);
    mn = fminf(mn, s.fred[WARPS + w]);
  }
  // The bins divide the range of the logits that have a weight. Masks (-inf, the type's lowest
  // value, -1e4) and outliers of that size become -inf and leave it: stretched by them, a cut's bin
  // outgrows the list (8 rows of 128256, top_p 0.9, the last 20000 masked: 527 us, so 26; top_k 50,
  // all but 30 masked by the lowest value: 264 and 16). No logits of a model's own lie 1024 below its largest.
  auto weightless = [&](float top, float x) { return (top - x) * cf > kSampleSpan; };
  auto masked = [&](float top, float low) {
    return __builtin_expect(top - low > 1024.0f && weightless(top, low), false);
  };
  const float own = mx;                        // this CTA's largest
  if (!greedy && mx > -INFINITY && mx < INFINITY && masked(mx, mn)) {
    mn = INFINITY;
    for (int v = tid; v < n / 4; v += THREADS) {
      float x[4];
      sample_get4(xs, v, x);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (weightless(own, x[j])) x[j] = -INFINITY;
        else mn = fminf(mn, x[j]);
      }
      sample_put4(xs, v, x);
    }
    if (weightless(own, most)) most = -INFINITY;
    mn = sample_warp_reduce(mn, [](float x, float y) { return fminf(x, y); });
    __syncthreads();
    if (lane == 0) s.fred[warp] = mn;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WARPS; ++w) mn = fminf(mn, s.fred[w]);
  }
  // also: how many threads have a logit above -inf
  const int finite = __syncthreads_count(most > -INFINITY);
  cluster_wait();                              // every CTA of the cluster runs
  if (tid < cs) {
    st_cluster_u64(remote(&s.top[cr], tid), static_cast<u64>(__float_as_uint(mx)) << 32 | __float_as_uint(mn));
    st_cluster_u64(remote(&s.have[cr], tid), static_cast<u64>(finite));
  }
  cluster_sync_all();
  u64 have = 0;
  auto top_of = [&](int r) { return __uint_as_float(static_cast<uint32_t>(s.top[r] >> 32)); };
  auto low_of = [&](int r) { return __uint_as_float(static_cast<uint32_t>(s.top[r])); };
  for (int r = 0; r < cs; ++r) {
    have += s.have[r];
    mx = fmaxf(mx, top_of(r));
    mn = fminf(mn, low_of(r));
  }
  bool hidden = false;                         // none of this CTA's tokens has a weight
  if (masked(mx, mn)) {                        // leaves out such CTAs
    have = 0;
    mn = INFINITY;
    for (int r = 0; r < cs; ++r)
      if (!weightless(mx, top_of(r))) {
        have += s.have[r];
        mn = fminf(mn, low_of(r));
      }
    hidden = weightless(mx, own);
  }

  float cx = -INFINITY;                        // kept: x > cx, or x == cx and index <= ci (and min_p)
  int ci = -1;
  auto keeps = [&](float x, int i) { return x > cx || (x == cx && i <= ci); };
  auto each = [&](auto f) {                    // every token of this CTA
    for (int v = tid; v < n / 4; v += THREADS) {
      float x[4];
      sample_get4(xs, v, x);
#pragma unroll
      for (int j = 0; j < 4; ++j) f(x[j], i0 + 4 * v + j);
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
    for (int w = 0; w < WARPS; ++w) arg = min(arg, static_cast<int>(s.red[w]));
    if (tid == 0) st_cluster_u64(remote(&s.part[0][cr], 0), static_cast<u64>(arg));
    cluster_sync_all();
    if (cr == 0 && tid == 0) {
      for (int r = 0; r < cs; ++r) arg = min(arg, static_cast<int>(s.part[0][r]));
      a.out_idx[row] = mx > -INFINITY ? arg : -1;
      if (a.out_logp) a.out_logp[row] = mx > -INFINITY ? 0.0f : -INFINITY;
    }
    return;
  }
  if (mx == INFINITY) {                        // +inf logits share the weight: as 0 among -inf
    for (int v = tid; v < n / 4; v += THREADS) {
      float x[4];
      sample_get4(xs, v, x);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = x[j] == INFINITY ? 0.0f : -INFINITY;
      sample_put4(xs, v, x);
    }
    mx = mn = 0.0f;
    most = -INFINITY;
    have = 0;                                  // top_k counts tokens
    __syncthreads();
  } else if (__builtin_expect(hidden, false)) {
    for (int v = tid; v < n / 4; v += THREADS) sample_put4(xs, v, {-INFINITY, -INFINITY, -INFINITY, -INFINITY});
    most = -INFINITY;
    __syncthreads();
  }
  r.mxf = mx;
  r.mx = static_cast<double>(mx);
  // 2^octave bins per factor of 2 in the weight: as many as keep the range within the bins
  const float span = fminf((mx - mn) * cf, kSampleSpan);   // in factors of 2
  const int octave = span > 0.0f ? min(100, ilogbf(static_cast<float>(kSampleBins - 1) / span)) : 0;   // at least 4
  r.bin_scale = scalbnf(cf, octave);
  r.octave = min(octave, 31);
  const double p = static_cast<double>(pf);
  auto survives = [&](u64 w) { return w >= r.q; };         // min_p
  auto goal = [&](u64 total) {                 // the draw falls on the token whose running sum exceeds this
    const u64 t = static_cast<u64>(u * static_cast<double>(total));
    return t < total ? t : total - 1;
  };
  auto draw = [&](int i, u64 w, u64 total) {
    a.out_idx[row] = i;
    if (a.out_logp) a.out_logp[row] = logf(static_cast<float>(static_cast<double>(w) / static_cast<double>(total)));
  };

  // Largest threshold at which `want` tokens (or, by weight, the given share) are kept, bit by bit.
  auto bisect = [&](bool by_weight, u64 want, double share) {
    u64 t = 0;
    double target = 0.0;
    if (by_weight) {
      u64 v = 0;
      each([&](float x, int i) {
        if (keeps(x, i)) v += sample_weight(x, r);
      });
      target = share * static_cast<double>(cluster_all(sample_block_sum<THREADS>(v, s)));
    }
    for (int bit = 63; bit >= 0; --bit) {
      const u64 c = t | (1ull << bit);
      u64 v = 0;
      each([&](float x, int i) {
        if (keeps(x, i) && sample_rank(x, i) >= c) v += by_weight ? sample_weight(x, r) : 1ull;
      });
      v = cluster_all(sample_block_sum<THREADS>(v, s));
      if (by_weight ? (v > 0 && static_cast<double>(v) >= target) : v >= want) t = c;
    }
    return t;
  };
  // A warp has a contiguous part [j0, j1) of the CTA's tokens.
  auto warp_part = [](int n) { return (((n + WARPS - 1) / WARPS) + 127) & ~127; };
  const int per = warp_part(n);
  const int j0 = min(n, warp * per), j1 = min(n, j0 + per);
  // After a cut to p: weight of the warp's drawable tokens, those before the list and those of the list.
  u64 base = 0;
  bool summed = false;
  auto set_threshold = [&](u64 rank) {
    cx = sample_unkey(static_cast<uint32_t>(rank >> 32));    // always within the tokens kept so far
    ci = static_cast<int>(0xffffffffu - static_cast<uint32_t>(rank));
  };

  // One cut of the kept tokens: the k first of them (k > 0), or those that reach the share p
  // of their weight. With by_p the cut to k may take p, or the draw, in the same step.
  // by_thread: k from the threads' largest logits, of which the row has more than k. Returns
  // what is left to do.
  enum { NOTHING, DRAW, CUT_P, RETRY };
  auto cut = [&](int k, bool by_p, bool by_thread) -> int {
    if (k > 0 && by_thread) {
      if (most > -INFINITY) atomicAdd(hist + sample_bin(most, r), 1u);
      __syncthreads();
    } else if (k > 0) {
      each([&](float x, int i) {
        if (keeps(x, i)) atomicAdd(hist + sample_bin(x, r), 1u);
      });
      __syncthreads();
    } else {
      each([&](float x, int i) {
        const int b = sample_bin(x, r);
        // 2^(44 - y - shift), at most 2^15 but for a rounding: 49152 of them fit 32 bits
        const uint32_t m = sample_round(ex2_approx(sample_float(44 - sample_shift(b, r)) - (r.mxf - x) * cf));
        if (keeps(x, i) && m) atomicAdd(hist + b, m);
      });
      __syncthreads();
    }
    cluster_sync_all();
    if (cr == 0) {
      // BPT bins per thread over the cluster: what lies before each, in tokens or in weight
      u64 v[BPT], sum = 0, all;
      uint32_t h[8][BPT];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < cs) ld_cluster<BPT>(remote(hist + tid * BPT, q), h[q]);
#pragma unroll
      for (int j = 0; j < BPT; ++j) {
        v[j] = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q < cs) v[j] += h[q][j];
        if (k == 0) v[j] <<= sample_shift(tid * BPT + j, r);
        sum += v[j];
      }
      u64 before = sample_block_scan<THREADS>(sum, all, s);
      if (tid == 0) {
        s.cmd.lo = s.cmd.hi = k > 0 ? kSampleBins - 1 : 0;
        s.cmd.skip = k > 0 && !by_thread && static_cast<u64>(k) >= all;
        s.cmd.total = 0;
      }
      __syncthreads();
      // the bin in which the running value reaches the target (rounded weights: of their own total)
      const double target = k > 0 ? static_cast<double>(k) : p * static_cast<double>(all);
#pragma unroll
      for (int j = 0; j < BPT; ++j) {
        if (static_cast<double>(before) < target && static_cast<double>(before + v[j]) >= target) {
          const bool from0 = k > 0 && (by_thread || before + v[j] <= kSampleList);   // the k largest may fit the list
          s.cmd.lo = from0 ? 0 : tid * BPT + j;
          s.cmd.hi = tid * BPT + j;
          if (k > 0) s.cmd.total = from0 ? 0 : before;
        }
        before += v[j];
      }
      __syncthreads();
      // the command to the other CTAs
      if (tid < static_cast<int>(sizeof(SampleCmd) / 8))
        for (int q = 1; q < cs; ++q)
          st_cluster_u64(remote(reinterpret_cast<u64*>(&s.cmd) + tid, q), reinterpret_cast<const u64*>(&s.cmd)[tid]);
    }
    cluster_sync_all();                        // also: the histograms have been read, the list may overwrite the first one
    SampleCmd cmd = s.cmd;
    const int after = by_p && k > 0 ? CUT_P : DRAW;
    const bool whole = k > 0 && cmd.lo == 0;   // the list begins at the top
    auto tell = [&](int result) {              // first CTA: what comes of the list
      if (tid < cs) st_cluster_u64(remote(&s.cmd.skip, tid), static_cast<u64>(result) << 32);
    };
    static_assert(offsetof(SampleCmd, skip) % 8 == 0 && offsetof(SampleCmd, result) == offsetof(SampleCmd, skip) + 4,
                  "one 64-bit store");
    int result = SAMPLE_CUT;
    do {
      u64 above = 0, all = 0;                    // weight above the list, and of all tokens
      auto enlist = [&](float x, int i) {
        const int at = atomicAdd(&s.listed, 1);
        if (at < kSampleList) list[at] = sample_rank(x, i);
      };
      if (k > 0 && !cmd.skip) {
        each([&](float x, int i) {
          if (!keeps(x, i)) return;
          const int b = sample_bin(x, r);
          if (b >= cmd.lo && b <= cmd.hi) enlist(x, i);
        });
      } else if (k == 0) {
        base = 0;
        auto pass = [&](auto plain) {            // plain: no other filter
          for (int j = j0 + 4 * lane; j < j1; j += 128) {
            float x[4];
            u64 w[4];
            bool in[4];
            sample_get4(xs, j >> 2, x);
#pragma unroll
            for (int q = 0; q < 4; ++q) {        // four exponentials side by side: no branch among them
              const int b = sample_bin(x[q], r);
              w[q] = sample_weight(x[q], r);
              if (!plain.value) w[q] = keeps(x[q], i0 + j + q) ? w[q] : 0;
              const u64 wa = b < cmd.lo ? w[q] : 0;
              all += w[q];
              above += wa;
              if (!plain.value) base += survives(wa) ? wa : 0;
              in[q] = b == cmd.lo && w[q];
            }
            if (in[0] | in[1] | in[2] | in[3])
#pragma unroll
              for (int q = 0; q < 4; ++q)
                if (in[q]) enlist(x[q], i0 + j + q);
          }
          if (plain.value) base = above;
        };
        if (r.q == 0 && cx == -INFINITY) pass(SampleFlag<true>{});
        else pass(SampleFlag<false>{});
        base = sample_warp_reduce(base, [](u64 x, u64 y) { return x + y; });
        above = sample_block_sum<THREADS>(above, s);
        all = sample_block_sum<THREADS>(all, s);
      }
      __syncthreads();
      if (tid == 0) st_cluster_u64(remote(&s.have[cr], 0), static_cast<u64>(s.listed));
      all = cluster_all2(all, above);
      if (cmd.skip) {
        for (int j = tid; j < kSampleBins; j += THREADS) hist[j] = 0;
        __syncthreads();
        return after;
      }
      if (cr == 0) {
        // the other CTAs' parts of the list behind this one's
        int end[8], len = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          if (q < cs) len += static_cast<int>(s.have[q]);
          end[q] = len;
        }
        if (len <= kSampleList)
          for (int e = end[0] + tid; e < len; e += THREADS) {
            int q = 0, from = 0;
#pragma unroll
            for (int o = 0; o < 7; ++o)
              if (e >= end[o]) q = o + 1, from = end[o];
            list[e] = ld_cluster_u64(remote(list + (e - from), q));
          }
        __syncthreads();
        if (len > kSampleList) {
          tell(SAMPLE_SHORT);
        } else if (whole && len <= kSampleSmall) {
          // THREADS / 256 threads per token e: how many tokens come before it and their weight, then the
          // weight of the kept tokens up to it in vocabulary order.
          constexpr int TPE = THREADS / kSampleSmall;
          const int e = tid / TPE, half = tid % TPE;
          const u64 re = e < len ? list[e] : 0;
          const u64 we = e < len ? sample_weight(sample_unkey(static_cast<uint32_t>(re >> 32)), r) : 0;
          u64* w = list + kSampleSmall;          // weights, by list entry (each pair writes its own)
          if (half == 0) w[e] = we;
          __syncthreads();
          int place = 0;
          u64 larger = 0;
#pragma unroll 4
          for (int j = half; j < len; j += TPE) {
            const bool before = list[j] > re;
            place += before;
            larger += before ? w[j] : 0;
          }
#pragma unroll
          for (int o = 1; o < TPE; o <<= 1) {
            place += __shfl_xor_sync(0xffffffffu, place, o);
            larger += __shfl_xor_sync(0xffffffffu, larger, o);
          }
          bool in = e < len && place < k;
          if (by_p) {
            const u64 wk = sample_block_sum<THREADS>(in && half == 0 ? we : 0, s);
            in = in && (place == 0 || static_cast<double>(larger) < p * static_cast<double>(wk));
          }
          in = in && survives(we);
          __syncthreads();
          if (half == 0) w[e] = in ? we : 0;
          const u64 tot = sample_block_sum<THREADS>(in && half == 0 ? we : 0, s);
          const uint32_t ie = static_cast<uint32_t>(re);           // ~index: larger is earlier
          u64 upto = 0;
#pragma unroll 4
          for (int j = half; j < len; j += TPE) upto += static_cast<uint32_t>(list[j]) >= ie ? w[j] : 0;
#pragma unroll
          for (int o = 1; o < TPE; o <<= 1) upto += __shfl_xor_sync(0xffffffffu, upto, o);
          const u64 t = goal(tot);
          if (in && half == 0 && upto > t && upto - we <= t) draw(static_cast<int>(0xffffffffu - ie), we, tot);
          tell(SAMPLE_DRAWN);
        } else {
          u64 v[BPT], w[BPT], C = 0;
#pragma unroll
          for (int j = 0; j < BPT; ++j) v[j] = tid * BPT + j < len ? list[tid * BPT + j] : 0;
          int found = SAMPLE_CUT;
          for (bool count = k > 0;; count = false) {
            u64 sum = 0;                         // to k: entries as they are; to p: those the cut to k left
#pragma unroll
            for (int j = 0; j < BPT; ++j) {
              const bool in = tid * BPT + j < len && v[j] >= C;
              w[j] = !in ? 0 : count ? 1 : sample_weight(sample_unkey(static_cast<uint32_t>(v[j] >> 32)), r);
              sum += w[j];
            }
            double target = static_cast<double>(k) - static_cast<double>(cmd.total);
            if (!count) {
              const u64 tot = above + sample_block_sum<THREADS>(sum, s);
              target = p * static_cast<double>(k == 0 ? all : tot);
              if (k == 0 && cmd.lo > 0 && static_cast<double>(above) >= target) found = SAMPLE_DOWN;
              else if (k == 0 && cmd.hi < kSampleBins - 1 && static_cast<double>(tot) < target) found = SAMPLE_UP;
              if (found != SAMPLE_CUT) break;
              target = fmin(fmax(target, static_cast<double>(above) + 0.5), static_cast<double>(tot));   // the first always
            }
            C = sample_select<THREADS, BPT>(v, w, above, target, list, s);
            if (!count || !whole || !by_p) break;
          }
          if (tid < cs) st_cluster_u64(remote(&s.cmd.C, tid), C);
          if (k == 0 && found == SAMPLE_CUT)
#pragma unroll
            for (int j = 0; j < BPT; ++j)
              if (w[j] && v[j] >= C && survives(w[j])) {
                const int i = static_cast<int>(0xffffffffu - static_cast<uint32_t>(v[j])), q = i / a.slice;
                const int nq = min(a.V, (q + 1) * a.slice) - q * a.slice;
                atomic_add_cluster_u64(remote(&s.wsum[(i - q * a.slice) / warp_part(nq)], q), w[j]);
              }
          tell(found);
        }
      }
      cluster_sync_all();
      result = s.cmd.result;
      for (int j = tid; j < kSampleBins; j += THREADS) hist[j] = 0;   // the list has been read
      if (tid == 0) s.listed = 0;
      __syncthreads();
      const int move = result == SAMPLE_UP ? 1 : result == SAMPLE_DOWN ? -1 : 0;
      cmd.lo += move;
      cmd.hi += move;
    } while (result >= SAMPLE_DOWN);           // ends: the exact sums order the bins
    if (result == SAMPLE_DRAWN) return NOTHING;
    if (result == SAMPLE_SHORT) {
      if (k > 0 && by_thread) return RETRY;
      set_threshold(bisect(k == 0, static_cast<u64>(k), p));
      return after;
    }
    set_threshold(s.cmd.C);
    if (k == 0) {
      base += s.wsum[warp];
      summed = true;
    }
    return whole ? DRAW : after;
  };
  const bool by_p = p < 1.0;
  int left = DRAW, k = top_k > 0 && top_k < a.V ? top_k : 0;
  bool by_thread = k > 0 && have > static_cast<u64>(k);
  for (bool more = k > 0 || by_p; more;) {     // one call: the cut stays inline, its state in registers
    left = cut(k, by_p, by_thread);
    more = left == RETRY || left == CUT_P;
    if (left == CUT_P) k = 0;
    by_thread = false;
  }
  if (left == NOTHING) return;

  // ------------------------------------------------ the draw, in vocabulary order
  auto kept = [&](float x, int j) -> u64 {
    const u64 w = sample_weight(x, r);
    return keeps(x, i0 + j) && survives(w) ? w : 0ull;
  };
  u64 mine = 0;
  auto part = [&](auto f) {
    for (int j = j0 + 4 * lane; j < j1; j += 128) {
      float x[4];
      sample_get4(xs, j >> 2, x);
      if (fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) >= cx)
        mine += (f(x[0], j) + f(x[1], j + 1)) + (f(x[2], j + 2) + f(x[3], j + 3));
    }
  };
  if (!summed) {
    if (r.q > 0 || cx > -INFINITY) part(kept);
    else part([&](float x, int) { return sample_weight(x, r); });
    mine = sample_warp_reduce(mine, [](u64 x, u64 y) { return x + y; });
  } else {
    mine = base;
  }
  // the sums of the warps before: of this CTA, then of the cluster
  auto warps = [&](u64 v, u64& block) {
    __syncthreads();
    if (lane == 0) s.red[warp] = v;
    __syncthreads();
    u64 before = 0;
    block = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) before += s.red[w];
      block += s.red[w];
    }
    return before;
  };
  u64 block, before = warps(mine, block);
  if (tid < cs) st_cluster_u64(remote(&s.part[turn][cr], tid), block);
  cluster_sync_all();                          // the last access to another CTA's memory
  u64 total = 0, first = 0;
  for (int q = 0; q < cs; ++q) {
    if (q < cr) first += s.part[turn][q];
    total += s.part[turn][q];
  }
  const u64 target = goal(total);
  if (target < first || target >= first + block) return;   // in another CTA's part
  before += first;
  if (before <= target && target < before + mine && lane == 0) s.listed = j0, s.red[0] = before;
  __syncthreads();
  // the part of the warp that has it, once more by all warps, then by the one that has it
  const int g0 = s.listed, sub = per / WARPS < 32 ? 32 : (per / WARPS + 31) & ~31;
  const u64 start = s.red[0];
  const int k0 = min(n, g0 + warp * sub), k1 = min(min(n, g0 + per), k0 + sub);
  u64 v = 0;
  for (int j = k0 + lane; j < k1; j += 32) v += kept(static_cast<float>(xs[j]), j);
  v = sample_warp_reduce(v, [](u64 x, u64 y) { return x + y; });
  before = start + warps(v, block);
  if (before <= target && target < before + v) {
    for (int jb = k0; jb < k1; jb += 32) {
      const u64 w = jb + lane < k1 ? kept(static_cast<float>(xs[jb + lane]), jb + lane) : 0;
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
