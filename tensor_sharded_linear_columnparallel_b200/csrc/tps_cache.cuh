// tps_cache.cuh -- the shards' KV caches: appending the K and V of a QKV output and
// the attention of one new token per sequence against them (a sliding window with
// sinks, or a prefix shared by the batch).
//
// A cache is [nseq][nkv][cap][128] bf16 with nkv = tp * kvs: KV head slot g = r * kvs + j
// is KV head j of shard r (a replicated head has a copy in every shard that holds it).
// The first nsink positions keep slots 0..nsink-1; the positions behind them share the
// other cap - nsink slots as a ring, slot(t) = nsink + (t - nsink) mod (cap - nsink).
// Without positions in the keys the order of the slots does not matter to a softmax, so
// a ring is read in slot order.
#pragma once

#include "tps_attn.cuh"

namespace tps {

// ---------------------------------------------------------------- append
// Token i of sequence b (position pos[b] + i, i < count[b]) writes its K and V rows to its
// slot, unless a newer token of the same call would overwrite it: with R ring slots that
// leaves the tokens [0, sinks) and [n - R, n), each slot with one writer. Pure copies, bound
// by HBM or, for one token per sequence, by the launch. A block takes 8 of a sequence's
// remaining tokens, a thread the same 16 bytes of each: what depends on the head is computed
// once and 8 loads are in flight (a thread per 16 bytes with its own divisions: 4 prompts of
// 2048 tokens into rings of 1028, 8 KB per token and copy, in 13.3 us; so in 8.3).
constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 8;

__global__ void __launch_bounds__(kAppendThreads) tps_kv_append_kernel(const KvAppendArgs a, int groups) {
  griddep_wait();
  const int b = static_cast<int>(blockIdx.x) / groups;
  const int l0 = (static_cast<int>(blockIdx.x) - b * groups) * kAppendTokens;
  const int p = a.pos ? a.pos[b] : 0;
  if (p < 0) return;
  const uint32_t first = static_cast<uint32_t>(p), R = static_cast<uint32_t>(a.cap - a.nsink);
  const int n = a.count ? min(max(a.count[b], 0), a.S) : a.S;
  const int tail = max(0, n - static_cast<int>(R));              // the ring keeps the tokens from here on
  const int sinks = min(max(0, a.nsink - p), tail);              // and the slots of the sinks those before here
  const int live = sinks + n - tail;
  if (l0 >= live) return;
  long long row[kAppendTokens];                                  // slot of each token
  int tok[kAppendTokens];
#pragma unroll
  for (int j = 0; j < kAppendTokens; ++j) {
    const int l = l0 + j;
    tok[j] = l < sinks ? l : tail + l - sinks;
    const uint32_t t = first + static_cast<uint32_t>(tok[j]);    // below 2^32
    row[j] = t < static_cast<uint32_t>(a.nsink) ? t : a.nsink + (t - a.nsink) % R;
  }
  const int units = a.tp * 2 * a.kvs * 16;                       // 16-byte units of a token: per shard its K, then its V heads
  for (int u = threadIdx.x; u < units; u += kAppendThreads) {
    const int hr = u >> 4, r = hr / (2 * a.kvs), h = hr - r * 2 * a.kvs;
    const int is_v = h >= a.kvs, g = r * a.kvs + h - is_v * a.kvs;
    const uint4* src = reinterpret_cast<const uint4*>(a.qkv + static_cast<long long>(b) * a.S * a.ld +
                                                      static_cast<long long>(r) * a.shard_cols + (a.qs + h) * kAttnD) +
                       (u & 15);
    uint4* dst = reinterpret_cast<uint4*>((is_v ? a.v : a.k) +
                                          (static_cast<long long>(b) * a.tp * a.kvs + g) * a.cap * kAttnD) + (u & 15);
    uint4 x[kAppendTokens];
#pragma unroll
    for (int j = 0; j < kAppendTokens; ++j)
      if (l0 + j < live) x[j] = __ldg(src + tok[j] * (a.ld / 8));
#pragma unroll
    for (int j = 0; j < kAppendTokens; ++j)
      if (l0 + j < live) dst[row[j] * (kAttnD / 8)] = x[j];
  }
}

// ---------------------------------------------------------------- decode
// One new token per sequence, G = qs / kvs query heads per KV head slot. The work is the
// stream of the visible keys (512 bytes each), so it is cut by bytes: the 128-slot blocks
// of all (sequence, KV head slot, chunk of 16 heads) items stand in one line, each item
// with some blocks' room ahead of it for what it costs besides its stream, and every CTA
// (one per SM) takes an equal part of the line, wherever that begins and ends. An item
// cut by a border leaves its parts (running max, sum, unnormalised output, fp32) in the
// workspace, and the CTA that finishes last merges them. A CTA's part ends in at most one
// item that goes on behind it, so the item's counter is that of the CTA which has its first
// block: a place in the workspace that no size moves. It returns to zero.
// Behind a shared prefix every item leaves a part, to be merged with the prefix kernel's.
// Merging waits until the CTA's stream has ended and then uses all its warps, one output
// row each: done where an item ends, it held the stream up (64 sequences behind a prefix of
// 16384 took 118 us with it). Now 32 sequences with windows of 4096 take 92 us (483 MB, 0.80 of
// the copy rate), one with a window of 2048 12.5 (start 1.3, its block 4, the part 1.5, counting
// 0.6, the merge of 17 parts 3.5: latencies), 64 behind a prefix 75 in all.
//
// Blocks of 128 slots, with the roles of the two products exchanged so that the few heads
// are the small side: S^T = K Q^T has M = 128 slots, N = 16 heads, K = 128 dimensions;
// O^T += V^T P^T has M = 128 dimensions, N = 16 heads, K = 128 slots. Tensor memory holds
// S^T twice and O^T twice (64 columns). Warp 0 loads K and V (three stages of 64 KB), warp
// 1 issues the products, warps 2-5 hold one slot per thread for the softmax, warp 6 loads
// the next item's queries and its new K and V rows ahead.
//  - The new token's rows come from the QKV row itself: warp 6 writes them to the cache, and
//    warp 1 puts them into the loaded block, so nothing waits for the write. Rows of V that
//    the token does not see are zeroed there too: a slot never written may hold a NaN.
//  - The reference max behind P moves only when a score exceeds it by more than 8 (base 2):
//    one vote per block, and a reduction over the block only then (always at an item's
//    first block). The weights are rounded to bf16 for the product, as in the prefill (the
//    reason and the price stand there); the sum keeps them in fp32, a partial sum per thread
//    until the item ends.
constexpr int kDecWarps = 12;                                     // warps 7-11 only merge; more would leave each 128 registers
constexpr int kDecThreads = kDecWarps * 32;
constexpr int kDecStages = 3;
constexpr int kDecHeads = 16;                                     // heads per item
constexpr int kDecStageBytes = 2 * kAttnTileBytes;                // K and V of one block
constexpr int kDecOpBytes = kDecHeads * 256;                      // Q, or P: 16 rows of 128 bf16
constexpr int kDecOffQ = kDecStages * kDecStageBytes;             // [2]
constexpr int kDecOffP = kDecOffQ + 2 * kDecOpBytes;              // [2]
constexpr int kDecOffNew = kDecOffP + 2 * kDecOpBytes;            // [2][K row, V row]
constexpr int kDecOffRed = kDecOffNew + 2 * 512;                  // [4 warps][16] max, [4][16] sum, flags
constexpr int kDecOffBar = kDecOffRed + 1024;
constexpr int kDecSmemBytes = kDecOffBar + 256 + 1024;
constexpr uint32_t kDecIdescS = idesc_bf16_f32(128, kDecHeads);
constexpr uint32_t kDecIdescO = idesc_bf16_f32(128, kDecHeads) | (1u << 15);   // A (= V^T) MN-major
static_assert(kDecSmemBytes <= 232448, "shared memory budget");

// What the token at position t of a sequence sees, in slots: the sinks up to t, and the
// `ring` newest positions behind them, whose newest has ring offset e. As blocks: [0, na)
// and [nb0, nb1), no block in both.
struct DecView {
  int t, ring, e;
  int slot;                    // the new token's own
  int na, nb0, nb1;
  __device__ __forceinline__ int blocks() const { return na + nb1 - nb0; }
  __device__ __forceinline__ int block(int i) const { return i < na ? i : nb0 + i - na; }
};

__device__ __forceinline__ DecView dec_view(const DecodeArgs& a, int t) {
  DecView v;
  v.t = t;
  v.slot = t;
  v.ring = v.e = v.na = v.nb0 = v.nb1 = 0;
  if (t < 0 || (a.linear && t >= a.cap)) return v;
  if (t < a.nsink) {
    v.na = (t >> 7) + 1;
    return v;
  }
  const int R = a.cap - a.nsink;
  v.ring = min(t - a.nsink, a.window - 1) + 1;             // no t + 1: pos may be 2^31 - 1
  v.e = (t - a.nsink) % R;
  v.slot = a.nsink + v.e;
  const int first = v.e - (v.ring - 1);                    // ring offset of the oldest, negative when wrapped
  const int a_end = first >= 0 ? a.nsink : a.nsink + v.e + 1;
  const int b_beg = first >= 0 ? a.nsink + first : a.nsink + first + R;
  const int b_end = first >= 0 ? a.nsink + v.e + 1 : a.cap;
  v.na = (a_end + 127) >> 7;
  v.nb0 = max(b_beg >> 7, v.na);
  v.nb1 = max((b_end + 127) >> 7, v.nb0);
  return v;
}

__device__ __forceinline__ bool dec_sees(const DecodeArgs& a, const DecView& v, int slot) {
  if (slot < a.nsink) return slot <= v.t;
  int age = v.e - (slot - a.nsink);
  if (age < 0) age += a.cap - a.nsink;
  return slot < a.cap && age < v.ring;
}

// The line of all items (sequence, then KV head slot, then chunk): an item of nb blocks
// has a.room + nb places, block i at place room + i of them. This CTA works on the places
// [w0, w1): the first `rem` CTAs take share + 1, the others share. The line has fewer than
// 2^31 places (the host checks).
// The room is what an item costs besides its stream, in blocks (1.4 us): with none, 64
// sequences of 1 to 512 tokens behind a prefix left CTAs with nine items of one block each
// that took 27 us for their part of the line, those with three of three blocks 19.
struct DecWork {
  int ctas, share, rem;        // CTAs with work (at most the grid, at most one per place)
  int w0, w1;
  int b, t;                    // the sequence that w0 lies in, its token's position
  int base;                    // place where that sequence's first item begins
};

__device__ __forceinline__ int dec_border(const DecWork& w, int cta) { return cta * w.share + min(cta, w.rem); }
// The CTA that works on place x of the line.
__device__ __forceinline__ int dec_owner(const DecWork& w, int x) {
  const int head = w.rem * (w.share + 1);
  return x < head ? x / (w.share + 1) : w.rem + (x - head) / w.share;
}
__device__ __forceinline__ int dec_places(const DecodeArgs& a, const DecView& v) {   // of one item
  const int nb = v.blocks();
  return nb ? a.room + nb : 0;
}

// One item as a CTA meets it: blocks [i0, i1) of its nb are this CTA's.
struct DecItem {
  int b, g, ch;                // sequence, KV head slot, chunk of 16 heads
  int nb, i0, i1;
  int s;                       // place of its first block
  DecView v;
  __device__ __forceinline__ bool whole() const { return i0 == 0 && i1 == nb; }
};

// Walks the items of a CTA's part in order; every role walks them by itself.
struct DecWalk {
  int b, k, tnext;             // next item: its sequence, its number there; position of sequence b + 1
  int at;                      // where it begins
  DecView v;
  __device__ __forceinline__ DecWalk(const DecodeArgs& a, const DecWork& w) : b(w.b), k(0) {
    v = dec_view(a, w.t);
    tnext = b + 1 < a.nseq ? __ldcg(a.pos + b + 1) : -1;
    if (w.w0 < w.w1) k = (w.w0 - w.base) / dec_places(a, v);
    at = w.base + k * dec_places(a, v);
  }
  __device__ __forceinline__ bool next(const DecodeArgs& a, const DecWork& w, DecItem& it) {
    do {
      if (at >= w.w1 || w.w0 == w.w1) return false;
      while (k == a.nkv * a.nch || v.blocks() == 0) {           // the next sequence with blocks
        if (++b >= a.nseq) return false;                        // never, unless the positions change meanwhile
        v = dec_view(a, tnext);
        tnext = b + 1 < a.nseq ? __ldcg(a.pos + b + 1) : -1;
        k = 0;
      }
      it.b = b;
      it.g = a.nch == 1 ? k : k / a.nch;
      it.ch = k - it.g * a.nch;
      it.nb = v.blocks();
      it.s = at + a.room;
      it.i0 = max(0, w.w0 - it.s);
      it.i1 = min(it.nb, w.w1 - it.s);
      it.v = v;
      at = it.s + it.nb;
      ++k;
    } while (it.i0 >= it.i1);                                   // only its room is this CTA's
    return true;
  }
};

// Where CTA cta leaves its part of an item: per item where it has the whole of it (behind a
// prefix), else per CTA, which cuts at most the item that it begins in and the one it ends in.
__device__ __forceinline__ float* dec_part(const DecodeArgs& a, const DecWork& w, const DecItem& it, int cta) {
  if (it.whole()) return a.item_parts + (static_cast<long long>(it.b * a.nkv + it.g) * a.nch + it.ch) * kDecPartFloats;
  return a.parts + (static_cast<long long>(cta) * 2 + (it.s <= dec_border(w, cta) ? 0 : 1)) * kDecPartFloats;
}

// Max (or sum) over the 32 lanes of 16 values per lane: lane l ends with the result of
// value l >> 1 (both lanes of a pair the same): 8 + 4 + 2 + 1 exchanges, then one.
template <bool MAX>
__device__ __forceinline__ float warp_reduce16(const float (&x)[16], int lane) {
  float v[8];
  auto op = [](float p, float q) { return MAX ? fmaxf(p, q) : p + q; };
  const bool h4 = lane & 16, h3 = lane & 8, h2 = lane & 4, h1 = lane & 2;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float keep = h4 ? x[8 + i] : x[i], give = h4 ? x[i] : x[8 + i];
    v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, 16));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float keep = h3 ? v[4 + i] : v[i], give = h3 ? v[i] : v[4 + i];
    v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, 8));
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float keep = h2 ? v[2 + i] : v[i], give = h2 ? v[i] : v[2 + i];
    v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, 4));
  }
  const float keep = h1 ? v[1] : v[0], give = h1 ? v[0] : v[1];
  v[0] = op(keep, __shfl_xor_sync(0xffffffffu, give, 2));
  return op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}

__device__ __forceinline__ void dec_bar_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// Barrier over the four softmax warps that returns whether any thread passed true.
__device__ __forceinline__ bool dec_bar_or(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x))
      : "memory");
  return r != 0;
}

// Byte offset of 16-byte chunk c (0..15) of row r of a [rows][128] bf16 tile held as two
// boxes of [rows][64] with the 128-byte swizzle, `box` bytes apart.
__device__ __forceinline__ uint32_t sw128_chunk(int r, int c, uint32_t box) {
  return (c >> 3) * box + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

__device__ __forceinline__ void fence_proxy_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Merges the n parts of one output row with one warp, a lane holding four dimensions.
// part(c): the address of part c's outputs, with its max and sum in m and l; the lane's
// float4 is `lane` of the first `rows` parts (a row of 128 numbers) and `image` of the others.
// The loads of 18 parts are in flight before the first is used.
template <class Part>
__device__ __forceinline__ void dec_merge(int n, int rows, int lane, int image, Part part, __nv_bfloat16* dst) {
  float M = -INFINITY, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kIn = 18;
  for (int c0 = 0; c0 < n; c0 += kIn) {
    const int k = min(kIn, n - c0);
    const float* o = nullptr;
    float m = -INFINITY, l = 0.f;
    if (lane < k) o = part(c0 + lane, m, l);
    float4 v[kIn];
#pragma unroll
    for (int i = 0; i < kIn; ++i) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<uintptr_t>(
          __shfl_sync(0xffffffffu, static_cast<unsigned long long>(reinterpret_cast<uintptr_t>(o)), i)));
      v[i] = i < k ? __ldcg(p + (c0 + i < rows ? lane : image)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float mx = m;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
    const float Mn = fmaxf(M, mx);
    const float sc = M == -INFINITY ? 0.f : ex2_approx(M - Mn);
    const float f = m == -INFINITY ? 0.f : ex2_approx(m - Mn);
    float fl = f * l;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) fl += __shfl_xor_sync(0xffffffffu, fl, x);
    L = L * sc + fl;
    M = Mn;
    acc.x *= sc, acc.y *= sc, acc.z *= sc, acc.w *= sc;
#pragma unroll
    for (int i = 0; i < kIn; ++i) {
      const float fi = __shfl_sync(0xffffffffu, f, i);
      acc.x = fmaf(fi, v[i].x, acc.x);
      acc.y = fmaf(fi, v[i].y, acc.y);
      acc.z = fmaf(fi, v[i].z, acc.z);
      acc.w = fmaf(fi, v[i].w, acc.w);
    }
  }
  const float inv = 1.0f / L;
  reinterpret_cast<uint2*>(dst)[lane] = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
}

__global__ void __launch_bounds__(kDecThreads, 1)
    tps_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const DecodeArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t sBar = base + kDecOffBar;
  auto kv_full = [&](int i) { return sBar + 8u * i; };            // [3] K and V of a block have landed
  auto kv_empty = [&](int i) { return sBar + 24u + 8u * i; };     // [3]
  auto s_full = [&](int i) { return sBar + 48u + 8u * i; };       // [2]
  auto p_full = [&](int i) { return sBar + 64u + 8u * i; };       // [2]
  auto q_full = [&](int i) { return sBar + 80u + 8u * i; };       // [2] by item
  auto q_empty = [&](int i) { return sBar + 96u + 8u * i; };      // [2]
  auto o_free = [&](int i) { return sBar + 112u + 8u * i; };      // [2] O^T of the item has been read
  // Product n with V completes a phase of barrier n & 1. A wait for product k is exact: k + 2
  // cannot complete before the waiting warps have gone on, and k - 2 has completed before.
  auto pv_done = [&](int i) { return sBar + 128u + 8u * i; };     // [2]
  const uint32_t done_bar = sBar + 144u, epi_done_bar = sBar + 152u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + kDecOffBar + 160);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + kDecOffBar + 164);
  volatile int* never_flag = reinterpret_cast<volatile int*>(gbase + kDecOffBar + 168);
  int* last_flag = reinterpret_cast<int*>(gbase + kDecOffBar + 172);    // [4]: cut items' counters, their other CTAs
  DecWork* sWork = reinterpret_cast<DecWork*>(gbase + kDecOffBar + 192);
  static_assert(192 + sizeof(DecWork) <= 256, "barrier block");
  int* scan = reinterpret_cast<int*>(gbase + kDecOffRed);   // [kDecWarps] before the roles start

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kDecStages; ++i) {
      mbar_init(kv_full(i), 1);
      mbar_init(kv_empty(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i), 4);
      mbar_init(q_full(i), 1);
      mbar_init(q_empty(i), 1);
      mbar_init(o_free(i), 4);
      mbar_init(pv_done(i), 1);
    }
    mbar_init(done_bar, 1);
    mbar_init(epi_done_bar, 4);
    *abort_flag = 0;
    *never_flag = 0;
    last_flag[0] = last_flag[1] = -1;
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 64);
    tmem_relinquish();
  }
  griddep_launch_dependents();
  // Behind the prefix kernel this grid runs at the same time as that one, whose CTAs let it
  // start only after they have waited for everything before them; what it reads before its
  // own wait (the positions, the QKV rows, the caches) is older than both.
  if (!a.prefix_parts) griddep_wait();
  // the line of blocks: its length, then the sequence that this CTA's part begins in
  {
    const int per = a.nkv * a.nch;
    const int t0 = threadIdx.x < a.nseq ? __ldcg(a.pos + threadIdx.x) : -1;
    const int n0 = per * dec_places(a, dec_view(a, t0));
    int sum = n0;
    for (int b = threadIdx.x + kDecThreads; b < a.nseq; b += kDecThreads)
      sum += per * dec_places(a, dec_view(a, __ldcg(a.pos + b)));
    int incl = sum;                         // with one sequence per thread, also the scan below
    for (int x = 1; x < 32; x <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, x);
      if (lane >= x) incl += y;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int total = 0, excl = incl - sum;
    for (int i = 0; i < kDecWarps; ++i) {
      if (i < warp) excl += scan[i];
      total += scan[i];
    }
    DecWork w;
    w.ctas = min(total, static_cast<int>(gridDim.x));
    w.share = w.ctas ? total / w.ctas : 0;
    w.rem = total - w.share * w.ctas;
    const int cta = static_cast<int>(blockIdx.x);
    w.w0 = w.w1 = w.b = w.t = w.base = 0;
    if (cta < w.ctas) {
      w.w0 = dec_border(w, cta);
      w.w1 = dec_border(w, cta + 1);
    }
    if (threadIdx.x == 0) *sWork = w;
    __syncthreads();                        // also: scan[] has been read
    int before = 0;
    for (int b0 = 0; w.w0 < w.w1 && b0 < a.nseq; b0 += kDecThreads) {
      const int b = b0 + threadIdx.x;
      int t = t0, n = n0;
      if (a.nseq > kDecThreads) {
        if (b0 > 0) {
          t = b < a.nseq ? __ldcg(a.pos + b) : -1;
          n = per * dec_places(a, dec_view(a, t));
        }
        incl = n;
        for (int x = 1; x < 32; x <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, x);
          if (lane >= x) incl += y;
        }
        if (lane == 31) scan[warp] = incl;
        __syncthreads();
        excl = before + incl - n;
        for (int i = 0; i < kDecWarps; ++i) {
          if (i < warp) excl += scan[i];
          before += scan[i];
        }
      }
      if (excl <= w.w0 && w.w0 < excl + n) {
        sWork->b = b;
        sWork->t = t;
        sWork->base = excl;
      }
      if (a.nseq <= kDecThreads) break;
      __syncthreads();
      if (before > w.w0) break;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const DecWork w = *sWork;
  const uint32_t tmem_base = *tmem_slot;
  const uint64_t tmo = a.timeout_ns;
  const int G = a.qs / a.kvs;

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------ K and V of every block
      long long n = 0;
      bool ok = true;
      // read once in a call: the parts, which are read back, stay in L2 instead
      const uint64_t policy = l2_policy_evict_first();
      DecWalk walk(a, w);
      DecItem it;
      while (ok && walk.next(a, w, it)) {
        const int row = it.b * a.nkv + it.g;
        for (int i = it.i0; i < it.i1; ++i, ++n) {
          const int st = static_cast<int>(n % kDecStages);
          if (!mbar_wait(kv_empty(st), static_cast<uint32_t>((n / kDecStages) & 1) ^ 1u, abort_flag, tmo, a.status)) {
            ok = false;
            break;
          }
          const uint32_t dst = base + st * kDecStageBytes;
          const int slot0 = it.v.block(i) * kAttnBlk;
          mbar_arrive_expect_tx(kv_full(st), kDecStageBytes);
          tma_load_3d_hint(dst, &tmK, kv_full(st), 0, slot0, row, policy);
          tma_load_3d_hint(dst + kAttnHalf, &tmK, kv_full(st), 64, slot0, row, policy);
          tma_load_3d_hint(dst + kAttnTileBytes, &tmV, kv_full(st), 0, slot0, row, policy);
          tma_load_3d_hint(dst + kAttnTileBytes + kAttnHalf, &tmV, kv_full(st), 64, slot0, row, policy);
        }
      }
      // wait (bounded) for the copies still in flight before the CTA may exit
      for (long long i = n > kDecStages ? n - kDecStages : 0; i < n; ++i)
        mbar_wait(kv_full(static_cast<int>(i % kDecStages)), static_cast<uint32_t>((i / kDecStages) & 1), never_flag,
                  200000000ull, a.status);
    }
  } else if (warp == 6) {
    // -------------------------------------------------- queries and new rows, one item ahead
    int q = 0;
    DecWalk walk(a, w);
    DecItem it;
    for (; walk.next(a, w, it); ++q) {
      const int buf = q & 1;
      const int r = it.g / a.kvs, lk = it.g - r * a.kvs;
      const __nv_bfloat16* row =
          a.qkv + static_cast<long long>(it.b) * a.ld + static_cast<long long>(r) * a.shard_cols;
      const int h0 = it.ch * kDecHeads, gc = min(kDecHeads, G - h0);
      uint4 x[8], kv;
#pragma unroll
      for (int i = 0; i < 8; ++i) {                    // 16 heads x 16 chunks over 32 lanes
        const int h = 2 * i + (lane >> 4);
        x[i] = h < gc ? __ldcg(reinterpret_cast<const uint4*>(row + (lk * G + h0 + h) * kAttnD) + (lane & 15))
                      : make_uint4(0, 0, 0, 0);
      }
      const int is_v = lane >> 4;                      // lanes 0-15: the new K row, 16-31: the new V row
      kv = __ldcg(reinterpret_cast<const uint4*>(row + (a.qs + is_v * a.kvs + lk) * kAttnD) + (lane & 15));
      if (!__all_sync(0xffffffffu, mbar_wait(q_empty(buf), static_cast<uint32_t>((q >> 1) & 1) ^ 1u, abort_flag, tmo,
                                             a.status)))
        break;
      const uint32_t sq = base + kDecOffQ + buf * kDecOpBytes;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        st_shared_v4(sq + sw128_chunk(2 * i + (lane >> 4), lane & 15, kDecOpBytes / 2), x[i].x, x[i].y, x[i].z, x[i].w);
      st_shared_v4(base + kDecOffNew + buf * 512 + lane * 16, kv.x, kv.y, kv.z, kv.w);
      const int slot = it.v.slot, sb = slot >> 7;
      const int at_i = sb < it.v.na ? sb : sb - it.v.nb0 + it.v.na;   // the new slot's block, as one of the item's
      if (at_i >= it.i0 && at_i < it.i1 && it.ch == 0) {
        __nv_bfloat16* cache = is_v ? a.v : a.k;
        const long long at = (static_cast<long long>(it.b) * a.nkv + it.g) * a.cap + slot;
        reinterpret_cast<uint4*>(cache + at * kAttnD)[lane & 15] = kv;
      }
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(buf));
    }
  } else if (warp == 1) {
    // -------------------------------------------------- products
    long long n = 0;                                   // blocks of earlier items
    int q = 0;
    bool ok = true, any = false;
    DecWalk walk(a, w);
    DecItem it;
    // the block is loaded: the new K row in and S^T = K Q^T issued, then, while that runs, the
    // new V row in and the unseen V rows out
    auto issue_s = [&](int i, long long nn) -> bool {
      const int st = static_cast<int>(nn % kDecStages);
      if (!__all_sync(0xffffffffu, mbar_wait(kv_full(st), static_cast<uint32_t>((nn / kDecStages) & 1), abort_flag,
                                             tmo, a.status)))
        return false;
      const uint32_t kb = base + st * kDecStageBytes, vb = kb + kAttnTileBytes;
      const int slot0 = it.v.block(i) * kAttnBlk;
      const int nr = it.v.slot - slot0;
      const bool fresh = nr >= 0 && nr < kAttnBlk;
      const uint4 x = ld_shared_v4(base + kDecOffNew + (q & 1) * 512 + lane * 16);
      if (fresh) {
        if (lane < 16) st_shared_v4(kb + sw128_chunk(nr, lane, kAttnHalf), x.x, x.y, x.z, x.w);
        fence_proxy_async_shared();
      }
      __syncwarp();
      if (lane == 0) {
        tc_fence_after();
        const uint32_t sq = base + kDecOffQ + (q & 1) * kDecOpBytes;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint64_t off = static_cast<uint64_t>((kk & 3) * 2);   // 16 dimensions = 32 B along K
          umma_bf16(tmem_base + static_cast<uint32_t>(nn & 1) * kDecHeads,
                    smem_desc_sw128(kb + (kk < 4 ? 0 : kAttnHalf)) + off,
                    smem_desc_sw128(sq + (kk < 4 ? 0 : kDecOpBytes / 2)) + off, kDecIdescS, kk > 0 ? 1u : 0u);
        }
        umma_commit(s_full(static_cast<int>(nn & 1)));
      }
      __syncwarp();
      bool touched = fresh;
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        const int row = 32 * k + lane;
        const bool see = dec_sees(a, it.v, slot0 + row);
        if (!see) {
#pragma unroll
          for (int c = 0; c < 8; ++c) {                // any order of a row's chunks: all become zero
            st_shared_v4(vb + row * 128 + (((c + lane) & 7) << 4), 0, 0, 0, 0);
            st_shared_v4(vb + kAttnHalf + row * 128 + (((c + lane) & 7) << 4), 0, 0, 0, 0);
          }
        }
        touched |= __any_sync(0xffffffffu, !see);
      }
      if (fresh && lane >= 16) st_shared_v4(vb + sw128_chunk(nr, lane & 15, kAttnHalf), x.x, x.y, x.z, x.w);
      if (touched) fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0 && i == it.i1 - 1) umma_commit(q_empty(q & 1));
      __syncwarp();
      return true;
    };
    for (; ok && walk.next(a, w, it); ++q) {
      if (!__all_sync(0xffffffffu, mbar_wait(q_full(q & 1), static_cast<uint32_t>((q >> 1) & 1), abort_flag, tmo, a.status)) ||
          !issue_s(it.i0, n)) {
        ok = false;
        break;
      }
      any = true;
      for (int i = it.i0; i < it.i1; ++i, ++n) {
        if (i + 1 < it.i1 && !issue_s(i + 1, n + 1)) { ok = false; break; }
        const int st = static_cast<int>(n % kDecStages);
        const int pb = static_cast<int>(n & 1);
        // the first product of an item overwrites O^T of the item before the last
        if (i == it.i0 && !__all_sync(0xffffffffu, mbar_wait(o_free(q & 1), static_cast<uint32_t>((q >> 1) & 1) ^ 1u,
                                                             abort_flag, tmo, a.status))) {
          ok = false;
          break;
        }
        if (!__all_sync(0xffffffffu, mbar_wait(p_full(pb), static_cast<uint32_t>((n >> 1) & 1), abort_flag, tmo, a.status))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          tc_fence_after();
          const uint32_t vb = base + st * kDecStageBytes + kAttnTileBytes;
          const uint32_t sp = base + kDecOffP + pb * kDecOpBytes;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)               // 16 slots per product: 2048 B of V, 32 B of P
            umma_bf16(tmem_base + 32u + static_cast<uint32_t>(q & 1) * kDecHeads,
                      smem_desc_sw128_mn(vb + kk * 2048, kAttnHalf),
                      smem_desc_sw128(sp + (kk < 4 ? 0 : kDecOpBytes / 2)) + static_cast<uint64_t>((kk & 3) * 2),
                      kDecIdescO, (i > it.i0 || kk > 0) ? 1u : 0u);
          umma_commit(kv_empty(st));
          umma_commit(pv_done(pb));
        }
        __syncwarp();
      }
    }
    if (lane == 0) {
      // every issued product must be complete, and the softmax warps done, before tensor memory goes
      if (any) {
        umma_commit(done_bar);
        mbar_wait(done_bar, 0, never_flag, 200000000ull, a.status);
      }
      mbar_wait(epi_done_bar, 0, never_flag, tmo, a.status);
    }
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, 64);
  } else if (warp < 6) {
    // -------------------------------------------------- softmax and output (warps 2-5)
    // The four warps meet in named barriers, which cannot time out: a warp whose bounded
    // wait failed keeps coming to them and reports there, and all four leave together.
    const int q4 = warp & 3;                           // tensor-memory lane quarter
    const int row = q4 * 32 + lane;                    // slot of a block; dimension of the output
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    float* red = reinterpret_cast<float*>(gbase + kDecOffRed);      // [4][16]
    float* redl = red + 64;                                         // [4][16]
    volatile int* flg = reinterpret_cast<volatile int*>(red + 128); // [4]
    long long n = 0;
    int q = 0;
    bool ok = true;
    DecWalk walk(a, w);
    DecItem it;
    for (; ok && walk.next(a, w, it); ++q) {
      float mref[kDecHeads], lsum[kDecHeads];
#pragma unroll
      for (int h = 0; h < kDecHeads; ++h) {
        mref[h] = -INFINITY;
        lsum[h] = 0.f;
      }
      const uint32_t to = tmem_base + lane_off + 32u + static_cast<uint32_t>(q & 1) * kDecHeads;
      for (int i = it.i0; i < it.i1; ++i, ++n) {
        const int pb = static_cast<int>(n & 1);
        if (ok)
          ok = __all_sync(0xffffffffu, mbar_wait(s_full(pb), static_cast<uint32_t>((n >> 1) & 1), abort_flag, tmo, a.status));
        float s[kDecHeads] = {};
        bool move = !ok || i == it.i0;
        if (ok) {
          tc_fence_after();
          tmem_ld16(tmem_base + lane_off + static_cast<uint32_t>(pb) * kDecHeads, s);
          const bool see = dec_sees(a, it.v, it.v.block(i) * kAttnBlk + row);
#pragma unroll
          for (int h = 0; h < kDecHeads; ++h) {
            s[h] = see ? s[h] * a.scale_log2 : -INFINITY;
            move |= s[h] > mref[h] + 8.0f;
          }
        }
        if (dec_bar_or(move)) {
          const float mx = warp_reduce16<true>(s, lane);
          if ((lane & 1) == 0) red[q4 * 16 + (lane >> 1)] = mx;
          if (lane == 0) flg[q4] = ok ? 0 : 1;
          dec_bar_sync();
          if (flg[0] | flg[1] | flg[2] | flg[3]) {
            ok = false;
            break;
          }
          float al[kDecHeads];
#pragma unroll
          for (int h = 0; h < kDecHeads; ++h) {
            const float mn = fmaxf(fmaxf(mref[h], fmaxf(red[h], red[16 + h])), fmaxf(red[32 + h], red[48 + h]));
            al[h] = mn == -INFINITY ? 1.f : ex2_approx(mref[h] - mn);
            mref[h] = mn;
            lsum[h] *= al[h];
          }
          if (i > it.i0) {
            // O^T must hold the products of every earlier block before it is scaled: all but the last
            // are complete (S^T of this block was issued after them)
            ok = __all_sync(0xffffffffu, mbar_wait(pv_done(pb ^ 1), static_cast<uint32_t>(((n - 1) >> 1) & 1), abort_flag,
                                                        tmo, a.status));
            if (ok) {
              tc_fence_after();
              float o[16];
              tmem_ld16(to, o);
#pragma unroll
              for (int h = 0; h < kDecHeads; ++h) o[h] *= al[h];
              tmem_st16_wait(to, o);
            }
          }
          dec_bar_sync();                              // red[] is free again
        }
        if (ok) {
          // P^T: this slot's column of the 16 x 128 tile
          const uint32_t sp = base + kDecOffP + pb * kDecOpBytes + (row >> 6) * (kDecOpBytes / 2) + (row & 7) * 2;
#pragma unroll
          for (int h = 0; h < kDecHeads; ++h) {
            const float p = ex2_approx(s[h] - (mref[h] == -INFINITY ? 0.f : mref[h]));
            lsum[h] += p;
            const __nv_bfloat16 pbf = __float2bfloat16_rn(p);
            asm volatile("st.shared.b16 [%0], %1;" ::"r"(sp + h * 128 + ((((row & 63) >> 3) ^ (h & 7)) << 4)),
                         "h"(*reinterpret_cast<const uint16_t*>(&pbf))
                         : "memory");
          }
          fence_proxy_async_shared();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full(pb));
        }
      }
      if (ok)                                          // the item's last product
        ok = __all_sync(0xffffffffu, mbar_wait(pv_done(static_cast<int>((n - 1) & 1)),
                                               static_cast<uint32_t>(((n - 1) >> 1) & 1), abort_flag, tmo, a.status));
      const float lw = warp_reduce16<false>(lsum, lane);
      if ((lane & 1) == 0) redl[q4 * 16 + (lane >> 1)] = lw;
      if (lane == 0) flg[q4] = ok ? 0 : 1;
      dec_bar_sync();
      if (flg[0] | flg[1] | flg[2] | flg[3]) {
        ok = false;
        break;
      }
      tc_fence_after();
      float o[16];
      tmem_ld16(to, o);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free(q & 1));
      const int r = it.g / a.kvs, lk = it.g - r * a.kvs;
      const int h0 = it.ch * kDecHeads, gc = min(kDecHeads, G - h0);
      const int hl = lk * G + h0;                      // first head of the item within its shard
      __nv_bfloat16* dst = a.out + static_cast<long long>(it.b) * a.ldo + static_cast<long long>(r * a.qs + hl) * kAttnD;
      if (it.whole() && !a.prefix_parts) {
#pragma unroll
        for (int h = 0; h < kDecHeads; ++h)
          if (h < gc) {
            const float l = (redl[h] + redl[16 + h]) + (redl[32 + h] + redl[48 + h]);
            dst[h * kAttnD + row] = __float2bfloat16_rn(o[h] / l);
          }
      } else {
        float* slot = dec_part(a, w, it, static_cast<int>(blockIdx.x));
        if (!it.whole() && warp == 2 && lane == 0) {   // counted below, when the part is written
          const int k = it.s <= w.w0 ? 0 : 1;
          last_flag[k] = dec_owner(w, it.s);
          last_flag[2 + k] = dec_owner(w, it.s + it.nb - 1) - last_flag[k];
        }
#pragma unroll
        for (int h = 0; h < kDecHeads; ++h)
          if (h < gc) {
            __stcg(slot + h * kAttnD + row, o[h]);
            if (row == h) {
              __stcg(slot + kDecHeads * kAttnD + h, mref[h]);
              __stcg(slot + kDecHeads * kAttnD + kDecHeads + h,
                     (redl[h] + redl[16 + h]) + (redl[32 + h] + redl[48 + h]));
            }
          }
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(epi_done_bar);
  }

  // ---------------------------------------------------- merging and unused rows, all warps
  __threadfence();
  __syncthreads();                                     // every role is done, this CTA's parts are written
  // also: this grid must not complete before the prefix kernel, whichever items it had
  if (a.prefix_parts) griddep_wait();
  const int cta = static_cast<int>(blockIdx.x);
  if (!*abort_flag && w.w0 < w.w1) {
    // the cut items are this CTA's first and last: two threads count them, and put 1 where
    // the last of an item's CTAs is this one
    if (lane == 0 && warp < 2) {
      const int first = last_flag[warp];
      bool last = false;
      if (first >= 0) {
        last = atomicAdd(a.counters + first, 1) == last_flag[2 + warp];
        if (last) a.counters[first] = 0;               // left zero for the next call
      }
      __threadfence();
      last_flag[warp] = last;
    }
    __syncthreads();
    int job = 0;
    DecWalk walk(a, w);
    DecItem it;
    while (walk.next(a, w, it)) {
      const bool whole = it.whole();
      if (whole ? !a.prefix_parts : !last_flag[it.s <= w.w0 ? 0 : 1]) continue;
      const int r = it.g / a.kvs, lk = it.g - r * a.kvs;
      const int h0 = it.ch * kDecHeads, gc = min(kDecHeads, G - h0);
      const int c0 = whole ? cta : dec_owner(w, it.s);
      const int nw = whole ? 1 : dec_owner(w, it.s + it.nb - 1) - c0 + 1;
      for (int h = 0; h < gc; ++h, ++job) {
        if (job % kDecWarps != warp) continue;
        auto part = [&](int c, float& m, float& l) -> const float* {
          if (c < nw) {
            const float* sl = dec_part(a, w, it, c0 + c);
            m = __ldcg(sl + kDecHeads * kAttnD + h);
            l = __ldcg(sl + kDecHeads * kAttnD + kDecHeads + h);
            return sl + h * kAttnD;
          }
          const int per = 128 / G;                     // sequences per tile of the prefix kernel
          const long long pt =
              (static_cast<long long>(it.g) * a.prefix_tiles + it.b / per) * a.prefix_splits + (c - nw);
          const int pr = (it.b % per) * G + h0 + h;
          m = __ldcg(a.prefix_ml + pt * 256 + pr);
          l = __ldcg(a.prefix_ml + pt * 256 + 128 + pr);
          return a.prefix_parts + pt * 128 * kAttnD;
        };
        const int pr = a.prefix_parts ? (it.b % (128 / G)) * G + h0 + h : 0;
        dec_merge(nw + (a.prefix_parts ? a.prefix_splits : 0), nw, lane, attn_part_index(pr, lane), part,
                  a.out + static_cast<long long>(it.b) * a.ldo +
                      static_cast<long long>(r * a.qs + lk * G + h0 + h) * kAttnD);
      }
    }
  }
  for (int b = cta; b < a.nseq; b += gridDim.x)
    if (dec_view(a, __ldcg(a.pos + b)).blocks() == 0)
      for (int i = threadIdx.x; i < a.ldo / 8; i += kDecThreads)
        reinterpret_cast<uint4*>(a.out + static_cast<long long>(b) * a.ldo)[i] = make_uint4(0, 0, 0, 0);
}

}  // namespace tps
