// The 8-bit KV cache: E4M3 codes of K and V [B, Hkv, capacity, d] with one
// fp32 scale per (sequence, kv head, block of blk tokens), its append, the
// attention of one query token per sequence over it, and the eviction of its
// least attended tokens.
//
// A block's scale is a power of two, the smallest 2^e (e >= -120) with
// max|x| <= 448 * 2^e over the block's finite values: E4M3 has 4 significant
// bits at any exponent, so a power of two costs no accuracy against
// max|x| / 448, and a code moves exactly to another scale unless it drops
// below E4M3's normal range there.  A growing block can therefore be
// rescaled, and an evicted cache re-blocked, without a 16-bit copy.
#pragma once
#include "select.cuh"
#include "tc.cuh"

namespace thrift {

// ------------------------------------------------------------ conversions --

// Smallest 2^e, e >= -120, with a <= 448 * 2^e = 1.75 * 2^(e + 8); a >= 0
// finite.  The carry out of the mantissa is the step to the next e.
__device__ __forceinline__ float kv8_scale(float a) {
  const int e = (int)((__float_as_uint(a) + 0x1FFFFFu) >> 23) - 135;
  return __uint_as_float((uint32_t)(max(e, -120) + 127) << 23);
}

// 1 / s for a power of two s in [2^-120, 2^120] (exact).
__device__ __forceinline__ float kv8_inv(float s) {
  return __uint_as_float((254u << 23) - __float_as_uint(s));
}

// Two fp32 values -> two E4M3 codes (lo in the low byte), round to nearest
// even, saturating; NaN -> 0x7F.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t out;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(out) : "f"(lo), "f"(hi));
  return out;
}

// Two E4M3 codes -> two fp32 values (exact).
__device__ __forceinline__ float2 e4m3x2_decode(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ bool finite_f(float x) { return fabsf(x) < INFINITY; }

// Eight values -> eight codes under 1 / scale; what is not finite becomes NaN.
__device__ __forceinline__ uint2 kv8_encode8(const float (&x)[8], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = finite_f(x[2 * i]) ? x[2 * i] * inv : NAN;
    const float b = finite_f(x[2 * i + 1]) ? x[2 * i + 1] * inv : NAN;
    w[i] = e4m3x2(a, b);
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

__device__ __forceinline__ void kv8_decode8(uint2 c, float (&x)[8]) {
  const uint32_t w[4] = {c.x & 0xFFFFu, c.x >> 16, c.y & 0xFFFFu, c.y >> 16};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = e4m3x2_decode(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <int DT>
__device__ __forceinline__ void unpack8(uint4 r, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = h2f<DT>((uint16_t)(w[i] & 0xFFFFu));
    x[2 * i + 1] = h2f<DT>((uint16_t)(w[i] >> 16));
  }
}

// ----------------------------------------------------------------- layout --

// Codes of one cache tensor: byte (b, h, t, c) at b sb + h sh + t st + c.
struct Kv8Geom {
  int B, Hkv, capacity, blk, nblk;  // nblk = ceil(capacity / blk)
  int64_t sb, sh, st;
  __device__ __forceinline__ int64_t row(int b, int h, int t) const {
    return b * sb + h * sh + t * st;
  }
  __device__ __forceinline__ int64_t scale(int b, int h, int j) const {
    return ((int64_t)b * Hkv + h) * nblk + j;
  }
  __device__ __forceinline__ int len(const int32_t* lens, int b) const {
    return min(capacity, max(0, __ldg(lens + b)));
  }
};

// Maximum over the CTA (every thread gets it); red holds one float per warp.
__device__ __forceinline__ float block_max(float a, float* red) {
  a = fmaxf(a, 0.0f);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  __syncthreads();  // red may still be read from the previous call
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
  __syncthreads();
  a = red[0];
  for (int w = 1; w < (int)(blockDim.x >> 5); ++w) a = fmaxf(a, red[w]);
  return a;
}

// ----------------------------------------------------------------- append --

constexpr int kKv8Threads = 256;

// One CTA per (block that new tokens fall into, kv head, sequence): the
// block's new rows stay in registers between the maximum and the encoding,
// so the 16-bit values are read once; rows already there are re-encoded only
// when the new maximum raises the scale.
template <int DT, int D>
__global__ void __launch_bounds__(kKv8Threads) kv8_append_kernel(
    const uint16_t* __restrict__ kn, const uint16_t* __restrict__ vn, Kv8Geom g, int max_new,
    const int32_t* __restrict__ cache_len, const int32_t* __restrict__ n_new, uint8_t* k,
    uint8_t* v, float* ks, float* vs, float* __restrict__ weight) {
  constexpr int TPR = D / 8;                  // threads a row (8 values each)
  constexpr int RPP = kKv8Threads / TPR;      // rows a pass
  constexpr int PASSES = 128 / RPP;           // blk <= 128
  __shared__ float red[kKv8Threads / 32];
  const int h = blockIdx.y, b = blockIdx.z;
  const int len = g.len(cache_len, b);
  const int n = n_new ? min(max_new, max(0, __ldg(n_new + b))) : max_new;
  const int end = (int)min((int64_t)g.capacity, (int64_t)len + n);
  const int j = len / g.blk + (int)blockIdx.x;
  const int t0 = j * g.blk;
  const int first = max(t0, len), last = min(end, t0 + g.blk);  // new rows [first, last)
  if (first >= last) return;
  const int row = threadIdx.x / TPR, c = 8 * (threadIdx.x % TPR);
  if (weight)
    for (int t = first + threadIdx.x; t < last; t += kKv8Threads)
      weight[((int64_t)b * g.Hkv + h) * g.capacity + t] = 0.0f;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const uint16_t* src = (kv ? vn : kn) + ((int64_t)b * max_new * g.Hkv + h) * D + c;
    uint8_t* codes = (kv ? v : k) + c;
    float* scales = (kv ? vs : ks) + g.scale(b, h, j);
    uint4 raw[PASSES];
    float a = 0.0f;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int t = t0 + p * RPP + row;
      raw[p] = make_uint4(0, 0, 0, 0);
      if (t >= first && t < last)
        raw[p] = __ldg(reinterpret_cast<const uint4*>(src + (int64_t)(t - len) * g.Hkv * D));
    }
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      float x[8];
      unpack8<DT>(raw[p], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) a = fmaxf(a, finite_f(x[i]) ? fabsf(x[i]) : 0.0f);
    }
    const float was = first > t0 ? *scales : 0.0f;
    const float s = fmaxf(was, kv8_scale(block_max(a, red)));  // every thread has read was
    const float inv = 1.0f / s;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int t = t0 + p * RPP + row;
      if (t < first || t >= last) continue;
      float x[8];
      unpack8<DT>(raw[p], x);
      *reinterpret_cast<uint2*>(codes + g.row(b, h, t)) = kv8_encode8(x, inv);
    }
    if (first > t0 && s != was) {
      const float ratio = was / s;
      for (int t = t0 + row; t < first; t += RPP) {
        uint2* at = reinterpret_cast<uint2*>(codes + g.row(b, h, t));
        float x[8];
        kv8_decode8(*at, x);
        *at = kv8_encode8(x, ratio);
      }
    }
    if (threadIdx.x == 0) *scales = s;
  }
}

// new_len[b] = min(capacity, len + n).  new_len may be cache_len itself.
__global__ void kv8_advance_kernel(Kv8Geom g, int max_new, const int32_t* cache_len,
                                   const int32_t* __restrict__ n_new, int32_t* new_len) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= g.B) return;
  const int n = n_new ? min(max_new, max(0, __ldg(n_new + b))) : max_new;
  const int len = min(g.capacity, max(0, cache_len[b]));
  new_len[b] = (int)min((int64_t)g.capacity, (int64_t)len + n);
}

// ----------------------------------------------------------------- decode --

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Scores of one key (d codes at kp, 16-byte aligned) with a query row in
// shared memory.
template <int D>
__device__ __forceinline__ float kv8_dot(const uint8_t* kp, const float* qs) {
  float acc = 0.0f;
#pragma unroll
  for (int c = 0; c < D; c += 16) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(kp + c));
    float x[8];
    kv8_decode8(make_uint2(w.x, w.y), x);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc = fmaf(x[i], qs[c + i], acc);
    kv8_decode8(make_uint2(w.z, w.w), x);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc = fmaf(x[i], qs[c + 8 + i], acc);
  }
  return acc;
}

// One CTA per (query head, sequence): 128 keys at a time, one per thread,
// one running maximum and sum; then one channel per thread.
template <int DT, int D>
__global__ void __launch_bounds__(128) kv8_decode_kernel(
    const uint16_t* __restrict__ q, Kv8Geom g, int H, const uint8_t* __restrict__ k,
    const uint8_t* __restrict__ v, const float* __restrict__ ks, const float* __restrict__ vs,
    const int32_t* __restrict__ seq_len, float scale, uint16_t* __restrict__ out,
    float* __restrict__ lse) {
  __shared__ float qs[D], ps[128], red[4];
  const int hq = blockIdx.x, b = blockIdx.y, h = hq / (H / g.Hkv), tid = threadIdx.x;
  const int len = g.len(seq_len, b);
  const int64_t bh = (int64_t)b * H + hq;
  if (tid < D) qs[tid] = h2f<DT>(__ldg(q + bh * D + tid));
  float m = -INFINITY, l = 0.0f, o = 0.0f;
  for (int t0 = 0; t0 < len; t0 += 128) {
    __syncthreads();  // qs is in; ps of the previous keys has been read
    const int t = t0 + tid;
    float s = -INFINITY;
    if (t < len)
      s = kv8_dot<D>(k + g.row(b, h, t), qs) *
          (__ldg(ks + g.scale(b, h, t / g.blk)) * scale * kLog2e);
    float mx = s;
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    mx = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float ref = mx == -INFINITY ? 0.0f : mx;
    const float p = t < len ? exp2f(s - ref) : 0.0f;
    const float alpha = exp2f(m - ref);
    l = fmaf(l, alpha, p);
    o *= alpha;
    m = mx;
    ps[tid] = t < len ? p * __ldg(vs + g.scale(b, h, t / g.blk)) : 0.0f;
    __syncthreads();
    if (tid < D)
      for (int i = 0; i < min(128, len - t0); ++i)
        o = fmaf(ps[i], e4m3x2_decode(__ldg(v + g.row(b, h, t0 + i) + tid)).x, o);
  }
#pragma unroll
  for (int w = 16; w >= 1; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
  __syncthreads();
  if ((tid & 31) == 0) red[tid >> 5] = l;
  __syncthreads();
  l = red[0] + red[1] + red[2] + red[3];
  if (tid < D) out[bh * D + tid] = f2h<DT>(len > 0 ? o / l : 0.0f);
  if (tid == 0) lse[bh] = len > 0 ? m * kLn2 + logf(l) : -INFINITY;
}

// weight[b, h, t] += sum over the group's heads of exp(s - lse).
template <int DT, int D>
__global__ void __launch_bounds__(128) kv8_weight_kernel(
    const uint16_t* __restrict__ q, Kv8Geom g, int H, const uint8_t* __restrict__ k,
    const float* __restrict__ ks, const int32_t* __restrict__ seq_len, float scale,
    const float* __restrict__ lse, float* __restrict__ weight) {
  __shared__ float qs[D];
  const int h = blockIdx.y, b = blockIdx.z, G = H / g.Hkv, t = blockIdx.x * 128 + threadIdx.x;
  const int len = g.len(seq_len, b);
  if ((int)blockIdx.x * 128 >= len) return;
  float sum = 0.0f;
  for (int r = 0; r < G; ++r) {
    const int64_t bh = (int64_t)b * H + h * G + r;
    __syncthreads();
    if (threadIdx.x < D) qs[threadIdx.x] = h2f<DT>(__ldg(q + bh * D + threadIdx.x));
    __syncthreads();
    if (t < len)
      sum += expf(kv8_dot<D>(k + g.row(b, h, t), qs) *
                      (__ldg(ks + g.scale(b, h, t / g.blk)) * scale) -
                  __ldg(lse + bh));
  }
  if (t < len) weight[((int64_t)b * g.Hkv + h) * g.capacity + t] += sum;
}

// ------------------------------------------------------------------ evict --

// Order-preserving map of a weight to an unsigned key; NaN counts as -inf,
// -0 as +0.
__device__ __forceinline__ uint32_t kv8_key(float w) {
  const uint32_t u = __float_as_uint(w != w ? -INFINITY : w + 0.0f);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

constexpr int kKv8SelThreads = 1024;

// kept[b, h, i], i < min(len, budget): the tokens that stay, ascending: the
// first `sink`, the last `recent`, and the heaviest of the others, ties to
// the lower token.  One CTA per (kv head, sequence): a radix select of 8 bits
// a pass over the candidates' keys, then every warp writes the survivors of
// one contiguous stretch.
__global__ void __launch_bounds__(kKv8SelThreads) kv8_select_kernel(
    const float* __restrict__ weight, Kv8Geom g, const int32_t* __restrict__ seq_len, int budget,
    int sink, int recent, int32_t* __restrict__ kept, int32_t* __restrict__ len_out) {
  __shared__ int hist[256], s_gt[32], s_eq[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_rem, s_done;
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int len = g.len(seq_len, b);
  const int64_t bh = (int64_t)b * g.Hkv + h;
  const float* w = weight + bh * g.capacity;
  int32_t* out = kept + bh * budget;
  if (h == 0 && tid == 0) len_out[b] = min(len, budget);
  if (len <= budget) {
    for (int t = tid; t < len; t += kKv8SelThreads) out[t] = t;
    return;
  }
  const int lo = sink, hi = len - recent;  // candidates [lo, hi): more than are wanted
  int rem = budget - sink - recent;
  uint32_t prefix = 0, pmask = 0;
  if (rem == 0) {
    prefix = pmask = 0xFFFFFFFFu;  // no key of a number is all ones: none is taken
  } else {
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = 24 - 8 * pass;
      for (int i = tid; i < 256; i += kKv8SelThreads) hist[i] = 0;
      __syncthreads();
      for (int base = lo; base < hi; base += kKv8SelThreads) {
        const int t = base + tid;
        const uint32_t key = t < hi ? kv8_key(__ldg(w + t)) : 0u;
        const int digit = t < hi && (key & pmask) == prefix ? (int)((key >> shift) & 255u) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, digit);
        if (digit >= 0 && lane == __ffs(same) - 1) atomicAdd(&hist[digit], __popc(same));
      }
      __syncthreads();
      if (warp == 0) {
        int64_t above;
        const int sel = select_digit(hist, rem, &above);
        if (lane == 0) {
          s_rem = rem - (int)above;
          s_prefix = prefix | ((uint32_t)sel << shift);
          s_done = hist[sel] == rem - (int)above;
        }
      }
      __syncthreads();
      prefix = s_prefix;
      rem = s_rem;
      pmask |= 255u << shift;
      if (s_done) break;  // the whole bucket is taken: the lower bits decide nothing
      __syncthreads();    // hist and s_done are rewritten by the next pass
    }
  }
  // A token stays if protected, above the threshold, or one of the first
  // `rem` at it.
  const int per = (int)ceil_div(len, 32 * 32) * 32;
  const int from = warp * per, to = min(len, from + per);
  auto look = [&](int t, bool& gt, bool& eq) {
    gt = eq = false;
    if (t >= to) return;
    if (t < lo || t >= hi) {
      gt = true;
      return;
    }
    const uint32_t key = kv8_key(__ldg(w + t)) & pmask;
    gt = key > prefix;
    eq = key == prefix;
  };
  int ngt = 0, neq = 0;
  for (int t = from + lane; t - lane < to; t += 32) {
    bool gt, eq;
    look(t, gt, eq);
    ngt += __popc(__ballot_sync(0xffffffffu, gt));
    neq += __popc(__ballot_sync(0xffffffffu, eq));
  }
  if (lane == 0) {
    s_gt[warp] = ngt;
    s_eq[warp] = neq;
  }
  __syncthreads();
  int gt0 = 0, eq0 = 0;
  for (int i = 0; i < warp; ++i) {
    gt0 += s_gt[i];
    eq0 += s_eq[i];
  }
  const unsigned below = (1u << lane) - 1u;
  for (int t = from + lane; t - lane < to; t += 32) {
    bool gt, eq;
    look(t, gt, eq);
    const unsigned mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
    const int e = eq0 + __popc(me & below);
    // survivors before this token: all above, and the first rem of the equal
    if (gt || (eq && e < rem)) out[gt0 + __popc(mg & below) + min(e, rem)] = t;
    gt0 += __popc(mg);
    eq0 += __popc(me);
  }
}

// One CTA per (block of the new cache, kv head, sequence): the kept tokens'
// values, re-encoded under the new block's own scale.
template <int D>
__global__ void __launch_bounds__(kKv8Threads) kv8_gather_kernel(
    Kv8Geom g, Kv8Geom go, const uint8_t* __restrict__ k, const uint8_t* __restrict__ v,
    const float* __restrict__ ks, const float* __restrict__ vs, const float* __restrict__ weight,
    const int32_t* __restrict__ seq_len, const int32_t* __restrict__ kept, int budget,
    uint8_t* __restrict__ ko, uint8_t* __restrict__ vo, float* __restrict__ kso,
    float* __restrict__ vso, float* __restrict__ wo) {
  constexpr int TPR = D / 8, RPP = kKv8Threads / TPR, PASSES = 128 / RPP;
  __shared__ float red[kKv8Threads / 32];
  const int j = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int n = min(g.len(seq_len, b), budget);
  const int i0 = j * g.blk;
  if (i0 >= n) return;
  const int i1 = min(n, i0 + g.blk);
  const int row = threadIdx.x / TPR, c = 8 * (threadIdx.x % TPR);
  const int64_t bh = (int64_t)b * g.Hkv + h;
  int src[PASSES];
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int i = i0 + p * RPP + row;
    src[p] = i < i1 ? __ldg(kept + bh * budget + i) : -1;
    if (src[p] >= 0 && c == 0) wo[bh * go.capacity + i] = __ldg(weight + bh * g.capacity + src[p]);
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const uint8_t* codes = (kv ? v : k) + c;
    const float* scales = kv ? vs : ks;
    float x[PASSES][8];
    float a = 0.0f;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      uint2 w = make_uint2(0, 0);
      float s = 0.0f;
      if (src[p] >= 0) {
        w = __ldg(reinterpret_cast<const uint2*>(codes + g.row(b, h, src[p])));
        s = __ldg(scales + g.scale(b, h, src[p] / g.blk));
      }
      kv8_decode8(w, x[p]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[p][e] *= s;
        a = fmaxf(a, finite_f(x[p][e]) ? fabsf(x[p][e]) : 0.0f);
      }
    }
    const float s = kv8_scale(block_max(a, red)), inv = kv8_inv(s);
#pragma unroll
    for (int p = 0; p < PASSES; ++p)
      if (src[p] >= 0)
        *reinterpret_cast<uint2*>((kv ? vo : ko) + c + go.row(b, h, i0 + p * RPP + row)) =
            kv8_encode8(x[p], inv);
    if (threadIdx.x == 0) (kv ? vso : kso)[go.scale(b, h, j)] = s;
  }
}

}  // namespace thrift
