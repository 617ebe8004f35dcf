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

__device__ __forceinline__ long long cache_slot(long long t, int nsink, int cap) {
  return t < nsink ? t : nsink + (t - nsink) % (cap - nsink);
}

// ---------------------------------------------------------------- append
// Token i of sequence b (position pos[b] + i, i < count[b]) writes its K and V rows to
// its slot; a token that a newer one of the same call would overwrite is skipped, so
// every slot has at most one writer. Pure copies, bound by HBM (or, for one token per
// sequence, by the launch): one thread per 16 bytes, 16 lanes per 256-byte row.
constexpr int kAppendThreads = 256;

__global__ void __launch_bounds__(kAppendThreads) tps_kv_append_kernel(const KvAppendArgs a) {
  griddep_wait();
  const long long unit = static_cast<long long>(blockIdx.x) * kAppendThreads + threadIdx.x;
  const int chunk = static_cast<int>(unit & 15);
  long long rest = unit >> 4;
  const int per = a.tp * 2 * a.kvs;                  // rows of one token: per shard kvs K heads, then kvs V heads
  const long long token = rest / per;
  if (token >= static_cast<long long>(a.nseq) * a.S) return;
  int hr = static_cast<int>(rest - token * per);
  const int b = static_cast<int>(token / a.S);
  const int i = static_cast<int>(token - static_cast<long long>(b) * a.S);
  const long long first = a.pos ? a.pos[b] : 0;
  const long long n = a.count ? min(max(a.count[b], 0), a.S) : a.S;
  if (first < 0 || i >= n) return;
  const long long t = first + i;
  if (t >= a.nsink && t + (a.cap - a.nsink) < first + n) return;   // a newer token of this call takes the slot
  const int r = hr / (2 * a.kvs);
  hr -= r * 2 * a.kvs;
  const int is_v = hr >= a.kvs;
  const int g = r * a.kvs + (hr - is_v * a.kvs);
  const uint4* src = reinterpret_cast<const uint4*>(a.qkv + token * a.ld + static_cast<long long>(r) * a.shard_cols +
                                                    static_cast<long long>(a.qs + hr) * kAttnD) + chunk;
  __nv_bfloat16* cache = is_v ? a.v : a.k;
  const long long row = (static_cast<long long>(b) * a.tp * a.kvs + g) * a.cap + cache_slot(t, a.nsink, a.cap);
  reinterpret_cast<uint4*>(cache + row * kAttnD)[chunk] = *src;
}

// ---------------------------------------------------------------- decode, plain form
// One CTA per (sequence, KV head slot): it appends the token, then for each of the slot's
// query heads its four warps walk the visible keys (a key per warp and step, a lane
// holds four dimensions) with a running max and sum and meet in shared memory.
constexpr int kDecThreads = 128;

__global__ void __launch_bounds__(kDecThreads) tps_decode_plain_kernel(const DecodeArgs a) {
  __shared__ float sm[4], sl[4], so[4][kAttnD];
  griddep_wait();
  const int g = static_cast<int>(blockIdx.x) % a.nkv;
  const int b = static_cast<int>(blockIdx.x) / a.nkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = g / a.kvs, lk = g - r * a.kvs;
  const long long t = a.pos[b];
  const bool live = t >= 0 && (a.linear == 0 || t < a.cap);
  const __nv_bfloat16* row = a.qkv + static_cast<long long>(b) * a.ld + static_cast<long long>(r) * a.shard_cols;
  __nv_bfloat16* kc = a.k + (static_cast<long long>(b) * a.nkv + g) * a.cap * kAttnD;
  __nv_bfloat16* vc = a.v + (static_cast<long long>(b) * a.nkv + g) * a.cap * kAttnD;
  if (live && threadIdx.x < 32) {
    const int is_v = threadIdx.x >> 4, ch = threadIdx.x & 15;
    const long long s = cache_slot(t, a.nsink, a.cap);
    reinterpret_cast<uint4*>((is_v ? vc : kc) + s * kAttnD)[ch] =
        reinterpret_cast<const uint4*>(row + (a.qs + is_v * a.kvs + lk) * kAttnD)[ch];
  }
  __syncthreads();
  const int R = a.cap - a.nsink;
  const int G = a.qs / a.kvs;
  const long long age0 = t >= a.nsink ? (t - a.nsink) % R : 0;   // ring offset of the newest token
  for (int h = 0; h < G; ++h) {
    const int hl = lk * G + h;
    __nv_bfloat16* dst = a.out + static_cast<long long>(b) * a.ldo + (r * a.qs + hl) * kAttnD;
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f}, q[4];
    for (int i = 0; i < 4; ++i) q[i] = __bfloat162float(row[hl * kAttnD + lane * 4 + i]);
    const int P = a.prefix_len;
    for (long long j = warp; live && j < static_cast<long long>(P) + a.cap; j += 4) {
      const __nv_bfloat16 *kr, *vr;
      if (j < P) {
        kr = a.pk + (static_cast<long long>(g) * P + j) * kAttnD;
        vr = a.pv + (static_cast<long long>(g) * P + j) * kAttnD;
      } else {
        const long long s = j - P;
        bool see;
        if (s < a.nsink) {
          see = s <= t;
        } else {
          const long long age = (age0 - (s - a.nsink) + R) % R;
          see = t >= a.nsink && age < a.window && t - age >= a.nsink;
        }
        if (!see) continue;
        kr = kc + s * kAttnD;
        vr = vc + s * kAttnD;
      }
      float s = 0.f;
      for (int i = 0; i < 4; ++i) s = fmaf(q[i], __bfloat162float(kr[lane * 4 + i]), s);
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      s *= a.scale_log2;
      const float mn = fmaxf(m, s), al = exp2f(m - mn), p = exp2f(s - mn);
      m = mn;
      l = l * al + p;
      for (int i = 0; i < 4; ++i) o[i] = o[i] * al + p * __bfloat162float(vr[lane * 4 + i]);
    }
    if (lane == 0) {
      sm[warp] = m;
      sl[warp] = l;
    }
    for (int i = 0; i < 4; ++i) so[warp][lane * 4 + i] = o[i];
    __syncthreads();
    const float mx = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    float L = 0.f, O = 0.f;
    for (int w = 0; w < 4; ++w) {
      const float f = sm[w] == -INFINITY ? 0.f : exp2f(sm[w] - mx);
      L += f * sl[w];
      O += f * so[w][threadIdx.x];
    }
    dst[threadIdx.x] = __float2bfloat16_rn(live ? O / L : 0.f);
    __syncthreads();
  }
}

}  // namespace tps
