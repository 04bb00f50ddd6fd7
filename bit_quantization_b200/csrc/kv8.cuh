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
#include <cfloat>

#include "select.cuh"
#include "tc.cuh"

namespace thrift {

// Every kernel here may be scheduled while the kernel before it in the stream
// ends, and waits for it before it reads or writes anything that one may have
// written.  Only one that another kernel of the same call follows lets that
// one be scheduled early, after its own wait: so the second may read ahead of
// its wait what the call's first kernel does not write, and a call's results
// are complete for whatever follows it.

// ------------------------------------------------------------ conversions --

// Smallest 2^e, e >= -120, with a <= 448 * 2^e = 1.75 * 2^(e + 8); a >= 0
// finite.  The carry out of the mantissa is the step to the next e.
__device__ __forceinline__ float kv8_scale(float a) {
  const int e = (int)((__float_as_uint(a) + 0x1FFFFFu) >> 23) - 135;
  return __uint_as_float((uint32_t)(max(e, -120) + 127) << 23);
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

// 2^x, to two units in the last place; results below 2^-126 are 0.
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
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

// Eight finite 16-bit values -> eight codes under 1 / scale.
template <int DT>
__device__ __forceinline__ uint2 kv8_encode8_finite(uint4 r, float inv) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = e4m3x2(h2f<DT>((uint16_t)(w[i] & 0xFFFFu)) * inv, h2f<DT>((uint16_t)(w[i] >> 16)) * inv);
  return make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
}

// Larger of |x| in each 16-bit half, as bits (infinities and NaN on top).
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t w) {
  return __vmaxu2(a, w & 0x7FFF7FFFu);
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

constexpr int64_t kKv8MaxRow = 1 << 24;  // bytes from a token to the next, less than

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
    return min(capacity, max(0, ld_behind(lens + b)));
  }
};

// ----------------------------------------------------------------- append --
//
// A CTA of four warps takes a tile of max(64, blk) rows of one tensor (K or
// V), kv head and sequence; each warp a quarter of it, whose values stay in
// registers between the maximum and the encoding, so that they are read once.
// A block's maximum is joined from its warps (one, two or four) in shared
// memory: every row is loaded before the one barrier of the CTA.  Measured: 8000
// tokens of 8 heads of 128 (49 MB in and out) 12.1 us with the lengths' kernel,
// bound by the latency of load, barrier and store in 2000 short CTAs.

constexpr int kKv8Warps = 4, kKv8Threads = 32 * kKv8Warps;
__host__ __device__ constexpr int kv8_tile(int blk) { return blk > 64 ? blk : 64; }

// Maximum over the warps of this warp's block: `n` neighbours from a multiple
// of n on.
__device__ __forceinline__ float kv8_join(const float* red, int warp, int n) {
  float a = red[warp & ~(n - 1)];
  for (int i = 1; i < n; ++i) a = fmaxf(a, red[(warp & ~(n - 1)) + i]);
  return a;
}
__device__ __forceinline__ float warp_max(float a) {  // a >= 0
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));
}

// Rows already in a block are re-encoded only when the new ones raise its
// scale.
template <int DT, int D, int TILE>
__global__ void __launch_bounds__(kKv8Threads) kv8_append_kernel(
    const uint16_t* __restrict__ kn, const uint16_t* __restrict__ vn, Kv8Geom g, int max_new,
    const int32_t* __restrict__ cache_len, const int32_t* __restrict__ n_new, uint8_t* k,
    uint8_t* v, float* ks, float* vs, float* __restrict__ weight, bool more) {
  constexpr int TPR = D / 8, RPP = 32 / TPR;  // threads a row (8 values each), rows a pass
  constexpr int ROWS = TILE / kKv8Warps, PASSES = ROWS / RPP;
  __shared__ float red[kKv8Warps];
  const int h = blockIdx.y >> 1, kv = blockIdx.y & 1, b = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = lane / TPR, c = 8 * (lane % TPR);
  pdl_wait();
  if (more) pdl_trigger();
  const int len = g.len(cache_len, b);
  const int n = n_new ? min(max_new, max(0, ld_behind(n_new + b))) : max_new;
  const int end = (int)min((int64_t)g.capacity, (int64_t)len + n);
  const int64_t tile0 = (int64_t)(len / g.blk) * g.blk + (int64_t)blockIdx.x * TILE;
  if (tile0 >= end || end == len) return;
  const int w0 = (int)tile0 + warp * ROWS;  // this warp's rows [w0, w0 + ROWS)
  const int wpb = g.blk > ROWS ? g.blk / ROWS : 1;
  const uint16_t* src = (kv ? vn : kn) + ((int64_t)b * max_new * g.Hkv + h) * D + c;
  uint8_t* codes = (kv ? v : k) + c;
  if (weight && !kv)
    for (int t = w0 + lane; t < w0 + ROWS; t += 32)
      if (t >= len && t < end) weight[((int64_t)b * g.Hkv + h) * g.capacity + t] = 0.0f;
  uint4 raw[PASSES];
  float a = 0.0f;
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int t = w0 + p * RPP + row;
    raw[p] = make_uint4(0, 0, 0, 0);
    if (t >= len && t < end)
      raw[p] = ld_behind(reinterpret_cast<const uint4*>(src + (int64_t)(t - len) * g.Hkv * D));
  }
  uint32_t bits = 0;
#pragma unroll
  for (int p = 0; p < PASSES; ++p)
    bits = max_abs2(max_abs2(max_abs2(max_abs2(bits, raw[p].x), raw[p].y), raw[p].z), raw[p].w);
  bits = max(bits & 0xFFFFu, bits >> 16);
  const bool odd = __any_sync(0xffffffffu, bits >= (DT == 1 ? 0x7F80u : 0x7C00u));
  a = h2f<DT>((uint16_t)bits);
  if (odd) {  // a value that is not finite: the others' maximum
    a = 0.0f;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      float x[8];
      unpack8<DT>(raw[p], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) a = fmaxf(a, finite_f(x[i]) ? fabsf(x[i]) : 0.0f);
    }
  }
  const int t0 = w0 / g.blk * g.blk;  // the warp's block
  float* scales = (kv ? vs : ks) + g.scale(b, h, 0) + w0 / g.blk;
  const float was = t0 < len && w0 < end ? *scales : 0.0f;
  if (lane == 0) red[warp] = 0.0f;
  a = warp_max(a);
  if (lane == 0) red[warp] = a;
  __syncthreads();  // every warp has read its block's scale, too
  if (t0 >= end) return;
  const float s = fmaxf(was, kv8_scale(kv8_join(red, warp, wpb))), inv = 1.0f / s;
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int t = w0 + p * RPP + row;
    if (t < len || t >= end) continue;
    uint2* to = reinterpret_cast<uint2*>(codes + g.row(b, h, t));
    if (odd) {
      float x[8];
      unpack8<DT>(raw[p], x);
      *to = kv8_encode8(x, inv);
    } else {
      *to = kv8_encode8_finite<DT>(raw[p], inv);
    }
  }
  if (t0 < len && s != was) {
    const float ratio = was / s;
    for (int t = w0 + row; t < min(len, w0 + ROWS); t += RPP) {
      uint2* at = reinterpret_cast<uint2*>(codes + g.row(b, h, t));
      float x[8];
      kv8_decode8(*at, x);
      *at = kv8_encode8(x, ratio);
    }
  }
  if (lane == 0 && w0 == t0) *scales = s;
}

// The few tokens of a generation step: one CTA a sequence, a warp a tensor
// and kv head, which takes a block at a time.  It ends with the new length
// (every warp has read the old one by then), so that a step is one launch:
// 3.2 us for 64 sequences of 8 heads, against 6.1 with the tiles above.
constexpr int kKv8StepTokens = 8;

template <int DT, int D>
__global__ void __launch_bounds__(1024) kv8_append_step_kernel(
    const uint16_t* __restrict__ kn, const uint16_t* __restrict__ vn, Kv8Geom g, int max_new,
    const int32_t* cache_len, const int32_t* __restrict__ n_new, uint8_t* k, uint8_t* v, float* ks,
    float* vs, float* __restrict__ weight, int32_t* new_len) {
  constexpr int TPR = D / 8, RPP = 32 / TPR, PASSES = kKv8StepTokens / RPP;
  const int b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = lane / TPR, c = 8 * (lane % TPR);
  pdl_wait();
  const int len = min(g.capacity, max(0, cache_len[b]));
  const int n = n_new ? min(max_new, max(0, ld_behind(n_new + b))) : max_new;
  const int end = (int)min((int64_t)g.capacity, (int64_t)len + n);
  for (int u = warp; u < 2 * g.Hkv; u += blockDim.x >> 5) {
    const int h = u >> 1, kv = u & 1;
    const uint16_t* src = (kv ? vn : kn) + ((int64_t)b * max_new * g.Hkv + h) * D + c;
    uint8_t* codes = (kv ? v : k) + g.row(b, h, 0);
    float* scales = (kv ? vs : ks) + g.scale(b, h, 0);
    if (weight && !kv && len + lane < end)
      weight[((int64_t)b * g.Hkv + h) * g.capacity + len + lane] = 0.0f;
    for (int t0 = len / g.blk * g.blk; t0 < end; t0 += g.blk) {
      const int first = max(t0, len), last = min(end, t0 + g.blk);
      if (first >= last) break;
      float x[PASSES][8], a = 0.0f;
      const float was = t0 < len ? scales[t0 / g.blk] : 0.0f;
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int t = first + p * RPP + row;
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (t < last)
          raw = ld_behind(reinterpret_cast<const uint4*>(src + (int64_t)(t - len) * g.Hkv * D));
        unpack8<DT>(raw, x[p]);
#pragma unroll
        for (int i = 0; i < 8; ++i) a = fmaxf(a, finite_f(x[p][i]) ? fabsf(x[p][i]) : 0.0f);
      }
      const float s = fmaxf(was, kv8_scale(warp_max(a))), inv = 1.0f / s;
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        const int t = first + p * RPP + row;
        if (t < last) *reinterpret_cast<uint2*>(codes + t * g.st + c) = kv8_encode8(x[p], inv);
      }
      if (t0 < len && s != was) {
        const float ratio = was / s;
#pragma unroll 8
        for (int t = t0 + row; t < len; t += RPP) {
          uint2* at = reinterpret_cast<uint2*>(codes + t * g.st + c);
          float y[8];
          kv8_decode8(*at, y);
          *at = kv8_encode8(y, ratio);
        }
      }
      if (lane == 0) scales[t0 / g.blk] = s;
    }
  }
  __syncthreads();
  if (new_len && threadIdx.x == 0) new_len[b] = end;
}

// new_len[b] = min(capacity, len + n).  new_len may be cache_len itself.
__global__ void kv8_advance_kernel(Kv8Geom g, int max_new, const int32_t* cache_len,
                                   const int32_t* __restrict__ n_new, int32_t* new_len) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  pdl_wait();  // the append still reads cache_len
  if (b >= g.B) return;
  const int n = n_new ? min(max_new, max(0, ld_behind(n_new + b))) : max_new;
  const int len = min(g.capacity, max(0, cache_len[b]));
  new_len[b] = (int)min((int64_t)g.capacity, (int64_t)len + n);
}

// ----------------------------------------------------------------- decode --
//
// One new query token per sequence attends to its cached tokens: per (kv head,
// sequence) the 256 (d = 128) bytes of a token are read once for all G query
// heads of the group, which bounds the kernel (4 G d products a token are
// 0.3 of the tensor cores' time at G = 16, far less below).  So the kernel is
// built to keep loads in flight: every warp streams its own tokens from memory
// to registers, 32 (d = 64: 64) at a time, the next ones' keys while the
// values of these are used and the other way round; nothing is staged, no warp
// waits for another before its tokens are done.  Measured: 4 sequences of
// 131072 tokens, 8 kv heads of 128, G = 4: 172 us, 6.2 TB/s, and 180 to 190
// once the card is at its power limit (a tenth of a second on); 32 of 4000 to 8192 with
// weights 86 us; G = 16 244 us, 4.4 TB/s, bound by the latency of 8 warps an
// SM; more heads read the cache once per 16 of them (32 heads over one kv head,
// 16 x 32768 tokens: 71 us, a reading is 20).
//
//   S^T [16 tokens, 8 heads] = K Q^T, O^T [16 channels, 8 heads] += V^T P^T
//
// run on register products (16 x 8 x 16, fp32 sums) whose operands are the
// registers that were loaded: K's codes become exact fp16 pairs in one
// instruction, V's after the bytes of two tokens are laced (the d axis of S
// and the channel of O are numbered as the loads leave them), and P^T is the
// transpose of the probabilities as S^T leaves them.  q enters as fp16, bf16
// brought there by a power of two of the row's largest value (an element
// 2^-28 below it and less keeps an error of 2^-39 of it).  A probability
// enters as fp16, relative to the running maximum and times 2^15, the top of
// fp16's range: within 2^-11 of itself down to 2^-29 of the largest, and within
// 2^-40 of the largest below.  (Taken as it is, at most 1, all below 2^-25 of a
// token that outweighs the others would be lost from O and not from the sum of
// probabilities: with one 20 above 500 others and no value, an eighth of the
// output.  A second product with what the rounding leaves takes fp16 outputs
// from 2.8e-4 of their norm to the 2.1e-4 of an fp32 form, and 8 to 10% more
// time: not kept.)  Sums of it are fp32, of the unrounded ones; O is kept in units of
// the scale of the V block at hand, and moves to another block's by an exact
// power of two, as it comes back from the factor 2^15.

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kKv8ProbUp = 32768.0f;  // of a probability's fp16 form
constexpr int kKv8DecWarps = 4;
__host__ __device__ constexpr int kv8_dec_ctas(int nt) { return nt > 1 ? 2 : 3; }  // an SM
constexpr int kKv8MaxCtas = 512;
// While every (sequence, kv head) has an SM and its capacity is at most four
// steps of a CTA of 8 warps (1024 tokens, d = 64: 2048), such a CTA takes all
// of one (up to 8 heads).  The length is not known on the host, so that the
// rule weighs a whole run of a cache, from empty to full.  8 pairs, d = 128,
// G = 4, in a graph: 3.8, 6.5, 8.2, 9.3 us for 64, 512, 768, 1024 tokens against
// 5.7, 6.9, 6.9, 6.9 for the split and its merge (d = 64, G = 8: 3.7, 6.4, 9.9
// for 128, 1024, 2048 against 6.2, 7.2, 7.2); a call from the host, which has a
// launch less, 15.1 against 17.6 at every length.  So either form is at most 3
// us behind the other up to there; at twice that capacity a full cache is 7 us
// behind (14.2 against 7.9 at 2048).  With more pairs than SMs the second round
// of CTAs costs more: 64 sequences of 8 heads and 1024 tokens 40.6 against 34.0.
constexpr int kKv8SoleWarps = 8, kKv8SoleSteps = 4;
constexpr int kKv8HeadGroup = 16;                 // query heads in one pass over the cache

// Tokens a warp takes at a time, and a CTA.
__host__ __device__ constexpr int kv8_step(int d) { return 4096 / d; }
__host__ __device__ constexpr int kv8_unit(int d) { return kKv8DecWarps * kv8_step(d); }

struct Kv8Dec {
  Kv8Geom g;
  int H, G, HG, Gc;  // query heads, a group's, its parts of at most 16, a part's
  const uint16_t* q;
  const uint8_t* k;
  const uint8_t* v;
  const float* ks;
  const float* vs;
  const int32_t* len;
  float scale;      // log2 e times the softmax scale
  float* part_o;    // [CTA][2][Gc][d], relative to the part's own maximum
  float* part_ml;   // [CTA][2][Gc][2] (maximum in log2 units, sum)
  float2* norm;     // [B, H] (maximum, sum) where one CTA has had all, or NULL
  float* scores;    // [B, Hkv, HG, capacity, Gc rounded to even] (log2 units), or NULL
  float* weight;
  uint16_t* out;
  float* lse;
  int ctas;     // of the pass over the cache
  int weights;  // CTAs of the finish that add up weights
  int lhc;      // log2 of the heads that a merging CTA of it takes: 0 .. 3
};

// The work of a step is a row of units (sequence, kv head, part of the group,
// kv8_unit tokens), dealt to the CTAs in equal runs whatever the lengths are.
// Every stretch of tokens costs a CTA about one unit more than its tokens
// (first loads, q, the join of the warps), so kKv8Head units without tokens
// precede those of each (kv head, part): many short sequences would otherwise
// fall to few CTAs.  A CTA has at most two stretches that others share, its
// first and its last; one that is its own it finishes itself.
// Lengths that another stream changes meanwhile give wrong results but no
// access out of bounds.
constexpr int kKv8Head = 1;
struct Kv8Plan {
  int ctas, run, longer;  // the first `longer` CTAs take run + 1 units, the others run
  __device__ __forceinline__ void set(int units, int n) {
    ctas = n;
    run = units / n;
    longer = units % n;
  }
  __device__ __forceinline__ int first(int cta) const { return run * cta + min(cta, longer); }
  __device__ __forceinline__ int owner(int unit) const {
    const int lead = longer * (run + 1);
    return min(ctas - 1, unit < lead ? unit / (run + 1) : longer + (unit - lead) / max(1, run));
  }
};

// Units of one (kv head, part) of a sequence.
template <int D>
__device__ __forceinline__ int kv8_units(const Kv8Dec& p, int b) {
  const int len = p.g.len(p.len, b);
  return len ? (int)ceil_div(len, kv8_unit(D)) + kKv8Head : 0;
}

// Units of all sequences, and of those before sequence `upto`, by every warp
// for itself.
template <int D>
__device__ __forceinline__ int2 kv8_count(const Kv8Dec& p, int upto) {
  int all = 0, before = 0;
#pragma unroll 4
  for (int b = threadIdx.x & 31; b < p.g.B; b += 32) {
    const int n = kv8_units<D>(p, b);
    all += n;
    before += b < upto ? n : 0;
  }
  const int per = p.g.Hkv * p.HG;
  return make_int2(per * __reduce_add_sync(0xffffffffu, all),
                   per * __reduce_add_sync(0xffffffffu, before));
}

// Four E4M3 codes -> four fp16 values (exact), the two low bytes first.
__device__ __forceinline__ void e4m3x4_f16(uint32_t c, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(c));
}
// Two fp16 values -> two E4M3 codes, as e4m3x2.
__device__ __forceinline__ uint32_t f16_e4m3x2(__half2 h) {
  uint16_t out;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(out) : "r"(*reinterpret_cast<uint32_t*>(&h)));
  return out;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Tokens on their way through the registers: read once, and like ld_behind
// loaded behind the wait.
__device__ __forceinline__ uint4 ld_stream16(const uint8_t* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
__device__ __forceinline__ uint2 ld_stream8(const uint8_t* p) {
  uint2 r;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
               : "=r"(r.x), "=r"(r.y)
               : "l"(p));
  return r;
}

// NT: heads of a part in eights.  A part of 16 heads takes 250 registers a
// thread: two CTAs of four warps an SM, the others three.
//
// SOLE: a CTA a (sequence, kv head, part), of W warps, and nothing left to
// finish: for caches so short and so few of them that the second launch would
// cost more than the split gains.
template <int DT, int D, int NT, int W, bool SOLE>
__global__ void __launch_bounds__(32 * W, SOLE ? 1 : kv8_dec_ctas(NT))
    kv8_decode_kernel(const Kv8Dec p) {
  constexpr int STEP = kv8_step(D), UNIT = W * STEP, NG = STEP / 16;
  constexpr int KS = D / 16;  // products along d
  constexpr int VW = D / 32;  // words of a token's channels a thread holds
  constexpr int QR = 8 * NT / W;  // rows of q a warp prepares
  static_assert(SOLE || UNIT == kv8_unit(D), "units as planned");
  __shared__ float s_o[W][8 * NT][D + 1];
  __shared__ float s_ml[W][8 * NT][2];
  __shared__ float s_qs[8 * NT];
  __shared__ __align__(16) uint16_t s_q[8 * NT][D];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, t = lane & 3;
  const int Gp = (p.Gc + 1) & ~1, per = p.g.Hkv * p.HG;
  const int lb = 31 - __clz(p.g.blk);  // blk is a power of two
  pdl_wait();
  // the finish may read the lengths: nothing before this writes them now
  if (!SOLE) pdl_trigger();
  int b, n, pair, j, u, uend;
  if constexpr (SOLE) {
    b = blockIdx.x / per;
    pair = blockIdx.x - b * per;
    n = (int)ceil_div(p.g.len(p.len, b), UNIT) + kKv8Head;
    j = u = 0;
    uend = n;
    if (n == kKv8Head) {  // an empty sequence
      const int part = pair % p.HG, empty = min(p.Gc, p.G - part * p.Gc);
      const int64_t first = (int64_t)b * p.H + pair / p.HG * p.G + part * p.Gc;
      for (int e = tid; e < empty * D; e += 32 * W) p.out[first * D + e] = 0;
      if (tid < empty) p.lse[first + tid] = -INFINITY;
      return;
    }
  } else {
    Kv8Plan plan;
    plan.set(kv8_count<D>(p, 0).x, p.ctas);
    u = plan.first(blockIdx.x);
    uend = plan.first(blockIdx.x + 1);
    if (u >= uend) return;
    int rel = u;
    b = n = 0;
    // the sequence of unit u
    for (int b0 = 0;; b0 += 32) {  // 32 sequences at a time
      const int mine = b0 + lane < p.g.B ? kv8_units<D>(p, b0 + lane) : 0;
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      const unsigned past = __ballot_sync(0xffffffffu, upto * per > rel);
      const int at = past ? __ffs(past) - 1 : 31;
      const int before = __shfl_sync(0xffffffffu, upto - mine, at);
      n = __shfl_sync(0xffffffffu, mine, at);
      if (past) {
        b = b0 + at;
        rel -= before * per;
        break;
      }
      if (b0 + 32 >= p.g.B) return;
      rel -= (before + n) * per;
    }
    pair = rel / n;  // (kv head, part)
    j = rel - pair * n;  // unit of it
    if (j + uend - u <= kKv8Head) return;  // no tokens
  }

  // the stretch of one sequence, kv head and part that is at hand, the
  // registers its tokens stream through, and its rows of q as they are
  int len, jn, heads, t0, tend;
  int64_t bh;  // the first query head
  bool sole;   // nobody else has tokens of this sequence, kv head and part
  const uint8_t *kb, *vb;
  const float *ksp, *vsp;
  float* sc;
  uint4 kw[NG][2][D / 64];
  uint32_t vw[NG][4][VW];
  float ksc[NG], vsc[NG];
  uint32_t qraw[QR][D / 64];
  // addresses: the sequence's and step's part is the warp's, a thread adds 32 bits
  const uint32_t st = (uint32_t)p.g.st, koff = gr * st + 16 * t, voff = 2 * t * st + (D / 8) * gr;
  auto load_k = [&](int first) {
    const uint8_t* base = kb + (int64_t)first * p.g.st;
    if (first + STEP <= len) {
#pragma unroll
      for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int x = 0; x < D / 64; ++x)
            kw[i][r][x] = ld_stream16(base + (koff + (16 * i + 8 * r) * st + 64 * x));
    } else {
#pragma unroll
      for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int x = 0; x < D / 64; ++x) {
            kw[i][r][x] = make_uint4(0, 0, 0, 0);
            if (first + 16 * i + 8 * r + gr < len)
              kw[i][r][x] = ld_stream16(base + (koff + (16 * i + 8 * r) * st + 64 * x));
          }
    }
#pragma unroll
    for (int i = 0; i < NG; ++i)
      ksc[i] = first + 16 * i < len ? ld_behind(ksp + ((first + 16 * i) >> lb)) : 1.0f;
  };
  auto load_v = [&](int first) {
    const uint8_t* base = vb + (int64_t)first * p.g.st;
    auto one = [&](uint32_t (&w)[VW], uint32_t off) {
      if constexpr (D == 128) {
        const uint4 x = ld_stream16(base + off);
        w[0] = x.x;
        w[1] = x.y;
        w[2] = x.z;
        w[3] = x.w;
      } else {
        const uint2 x = ld_stream8(base + off);
        w[0] = x.x;
        w[1] = x.y;
      }
    };
    if (first + STEP <= len) {
#pragma unroll
      for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          one(vw[i][r], voff + (16 * i + (r & 1) + 8 * (r >> 1)) * st);
    } else {
#pragma unroll
      for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int tok = 16 * i + (r & 1) + 8 * (r >> 1);
#pragma unroll
          for (int x = 0; x < VW; ++x) vw[i][r][x] = 0;
          if (first + tok + 2 * t < len) one(vw[i][r], voff + tok * st);
        }
    }
#pragma unroll
    for (int i = 0; i < NG; ++i)
      vsc[i] = first + 16 * i < len ? ld_behind(vsp + ((first + 16 * i) >> lb)) : 0.0f;
  };
  auto open = [&] {
    const int h = pair / p.HG, part = pair - h * p.HG;
    len = p.g.len(p.len, b);
    jn = min(n - j, uend - u);
    heads = min(p.Gc, p.G - part * p.Gc);
    bh = (int64_t)b * p.H + h * p.G + part * p.Gc;
    sole = j <= kKv8Head && j + jn == n;
    const uint16_t* q = p.q + bh * D + lane * (D / 32);
#pragma unroll
    for (int i = 0; i < QR; ++i) {  // channels lane * D / 32 on
      const int r = warp + W * i;
#pragma unroll
      for (int x = 0; x < D / 64; ++x)
        qraw[i][x] = r < heads ? ld_behind(reinterpret_cast<const uint32_t*>(q + r * D) + x) : 0u;
    }
    kb = p.k + p.g.row(b, h, 0);
    vb = p.v + p.g.row(b, h, 0);
    ksp = p.ks + p.g.scale(b, h, 0);
    vsp = p.vs + p.g.scale(b, h, 0);
    sc = p.scores ? p.scores + ((int64_t)b * per + pair) * p.g.capacity * Gp : nullptr;
    t0 = max(0, j - kKv8Head) * UNIT + warp * STEP;
    tend = min(len, (j + jn - kKv8Head) * UNIT);
    if (t0 < tend) {
      load_k(t0);
      load_v(t0);
    }
  };
  open();
  for (int seg = 0;; ++seg) {
    // ---- q as fp16, a warp a row, while the first tokens arrive
#pragma unroll
    for (int i = 0; i < QR; ++i) {
      const int r = warp + W * i;
      float x[D / 32], top = 0.0f;
      bool bad = false;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) {
        x[e] = h2f<DT>((uint16_t)(e & 1 ? qraw[i][e >> 1] >> 16 : qraw[i][e >> 1] & 0xFFFFu));
        top = fmaxf(top, fabsf(x[e]));
        bad |= !finite_f(x[e]);
      }
      bad = __any_sync(0xffffffffu, bad);
      float f = 1.0f, un = 1.0f;
      if (DT == 1) {  // the largest value to [2^14, 2^15)
        const int e = (int)(__reduce_max_sync(0xffffffffu, __float_as_uint(top)) >> 23);
        const int sh = min(max(141 - e, -126), 126);
        f = __uint_as_float((uint32_t)(sh + 127) << 23);
        un = __uint_as_float((uint32_t)(127 - sh) << 23);
      }
#pragma unroll
      for (int e = 0; e < D / 32; e += 2)
        *reinterpret_cast<uint32_t*>(&s_q[r][lane * (D / 32) + e]) =
            bad ? 0u : pack_f16(x[e] * f, x[e + 1] * f);
      if (lane == 0) s_qs[r] = bad ? NAN : un * p.scale;
    }
    __syncthreads();
    uint2 qf[NT][KS];
    float qs[NT][2];
#pragma unroll
    for (int a = 0; a < NT; ++a) {
#pragma unroll
      for (int s = 0; s < KS; ++s)
        qf[a][s] = *reinterpret_cast<const uint2*>(
            &s_q[8 * a + gr][64 * (s >> 2) + 16 * t + 4 * (s & 3)]);
      qs[a][0] = s_qs[8 * a + 2 * t];
      qs[a][1] = s_qs[8 * a + 2 * t + 1];
    }
    float o[NT][KS][4], m[NT][2], l[NT][2];
    float unit = 0.0f, umax = 0.0f;  // O is in units of `unit`
#pragma unroll
    for (int a = 0; a < NT; ++a) {
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[a][s][e] = 0.0f;
      m[a][0] = m[a][1] = -INFINITY;
      l[a][0] = l[a][1] = 0.0f;
    }
    for (; t0 < tend; t0 += UNIT) {
      float sv[NG][NT][4];
#pragma unroll
      for (int i = 0; i < NG; ++i) {
#pragma unroll
        for (int a = 0; a < NT; ++a)
#pragma unroll
          for (int e = 0; e < 4; ++e) sv[i][a][e] = 0.0f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const uint4 A = kw[i][0][s >> 2], B = kw[i][1][s >> 2];
          const uint32_t wa = (s & 3) == 0 ? A.x : (s & 3) == 1 ? A.y : (s & 3) == 2 ? A.z : A.w;
          const uint32_t wb = (s & 3) == 0 ? B.x : (s & 3) == 1 ? B.y : (s & 3) == 2 ? B.z : B.w;
          uint32_t a0, a1, a2, a3;
          e4m3x4_f16(wa, a0, a2);
          e4m3x4_f16(wb, a1, a3);
#pragma unroll
          for (int a = 0; a < NT; ++a)
            mma_16816(sv[i][a], a0, a1, a2, a3, qf[a][s].x, qf[a][s].y);
        }
#pragma unroll
        for (int a = 0; a < NT; ++a)
#pragma unroll
          for (int e = 0; e < 4; ++e) sv[i][a][e] *= qs[a][e & 1] * ksc[i];
      }
      if (t0 + STEP > len) {
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
          for (int a = 0; a < NT; ++a)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (t0 + 16 * i + gr + 8 * (e >> 1) >= len) sv[i][a][e] = -INFINITY;
      }
      if (t0 + UNIT < tend) load_k(t0 + UNIT);
      if (sc) {
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int tok = t0 + 16 * i + 8 * r + gr;
#pragma unroll
            for (int a = 0; a < NT; ++a)
              if (tok < len && 8 * a + 2 * t < Gp)
                *reinterpret_cast<float2*>(sc + (int64_t)tok * Gp + 8 * a + 2 * t) =
                    make_float2(sv[i][a][2 * r], sv[i][a][2 * r + 1]);
          }
      }
      // ---- running maximum and sum
      float mx[NT][2];
      bool grew = false;
#pragma unroll
      for (int a = 0; a < NT; ++a)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = sv[0][a][e];
#pragma unroll
          for (int i = 0; i < NG; ++i) x = fmaxf(x, fmaxf(sv[i][a][e], sv[i][a][e + 2]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          mx[a][e] = fmaxf(m[a][e], x);
          grew |= mx[a][e] > m[a][e];
        }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int a = 0; a < NT; ++a) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float al = mx[a][e] > m[a][e] ? exp2f(m[a][e] - mx[a][e]) : 1.0f;
            m[a][e] = mx[a][e];
            l[a][e] *= al;
            mx[a][e] = al;
          }
#pragma unroll
          for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[a][s][e] *= mx[a][e & 1];
        }
      }
      float ref[NT][2];
#pragma unroll
      for (int a = 0; a < NT; ++a)
#pragma unroll
        for (int e = 0; e < 2; ++e) ref[a][e] = m[a][e] == -INFINITY ? 0.0f : m[a][e];
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        if (t0 + 16 * i >= len) break;
        if (vsc[i] != unit) {
          umax = fmaxf(umax, vsc[i]);
          // a block 2^60 below the largest so far counts in that one's units
          const float nu = vsc[i] < umax * 0x1p-60f ? umax * 0x1p-60f : vsc[i];
          const float f = unit == 0.0f ? 0.0f : unit / nu;
          unit = nu;
#pragma unroll
          for (int a = 0; a < NT; ++a)
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[a][s][e] *= f;
        }
        uint32_t b0[NT], b1[NT];
#pragma unroll
        for (int a = 0; a < NT; ++a) {
          float pr[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            pr[e] = ex2(sv[i][a][e] - ref[a][e & 1]);
            l[a][e & 1] += pr[e];
          }
          const float up = vsc[i] == unit ? kKv8ProbUp : kKv8ProbUp * (vsc[i] / unit);
#pragma unroll
          for (int e = 0; e < 4; ++e) pr[e] *= up;
          b0[a] = transpose_8x8(pack_f16(pr[0], pr[1]));
          b1[a] = transpose_8x8(pack_f16(pr[2], pr[3]));
        }
#pragma unroll
        for (int x = 0; x < VW; ++x) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t lo = __byte_perm(vw[i][0][x], vw[i][1][x], y ? 0x7362 : 0x5140);
            const uint32_t hi = __byte_perm(vw[i][2][x], vw[i][3][x], y ? 0x7362 : 0x5140);
            uint32_t a0, a1, a2, a3;
            e4m3x4_f16(lo, a0, a1);
            e4m3x4_f16(hi, a2, a3);
#pragma unroll
            for (int a = 0; a < NT; ++a) mma_16816(o[a][2 * x + y], a0, a1, a2, a3, b0[a], b1[a]);
          }
        }
      }
      if (t0 + UNIT < tend) load_v(t0 + UNIT);
    }
    // ---- the next stretch's first tokens are on their way ...
    const int done = heads;
    const int64_t first_head = bh;
    const bool mine = sole;
    u += jn;
    j = 0;
    bool more = !SOLE && uend - u > kKv8Head;
    if (more && ++pair == per) {
      pair = n = 0;
      while (n == 0 && ++b < p.g.B) n = kv8_units<D>(p, b);
      more = n > 0;
    }
    if (more) open();
    // ---- ... while the CTA's warps join this one's parts
    const float down = unit * (1.0f / kKv8ProbUp);
#pragma unroll
    for (int a = 0; a < NT; ++a)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[a][e];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (gr == 0) {
          s_ml[warp][8 * a + 2 * t + e][0] = m[a][e];
          s_ml[warp][8 * a + 2 * t + e][1] = x;
        }
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            s_o[warp][8 * a + 2 * t + e][(D / 8) * gr + 2 * s + r] = o[a][s][2 * r + e] * down;
      }
    __syncthreads();
    const int64_t slot = 2 * (int64_t)blockIdx.x + (seg > 0);
    float* po = p.part_o + slot * p.Gc * D;
    float* pm = p.part_ml + slot * p.Gc * 2;
    for (int e = tid; e < done * D; e += 32 * W) {
      const int r = e / D, c = e % D;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < W; ++w) M = fmaxf(M, s_ml[w][r][0]);
      const float ref = M == -INFINITY ? 0.0f : M;
      float acc = 0.0f, L = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        // a warp without tokens has the maximum -inf and adds 0
        const float x = ex2(s_ml[w][r][0] - ref);
        acc += s_o[w][r][c] * x;
        L += s_ml[w][r][1] * x;
      }
      if (SOLE || mine) {
        p.out[first_head * D + e] = f2h<DT>(acc / L);
        if (c == 0) {
          p.lse[first_head + r] = M * kLn2 + logf(L);
          if (p.norm) p.norm[first_head + r] = make_float2(M, L);
        }
      } else {
        po[e] = acc;
        if (c == 0) {
          pm[2 * r] = M;
          pm[2 * r + 1] = L;
        }
      }
    }
    if (!more) break;
  }
}

// What is left once every part is there, by role of the CTA.  The first
// p.weights, for the weights: kKv8WeightTokens tokens of one (sequence, kv
// head), weight += their probabilities summed over the group's heads, from the
// scores that the pass over the keys has left.  The others: the parts of
// 2^p.lhc query heads of one (sequence, kv head, part of the group) merged, the
// 8 warps dealt to the heads: out and lse.
constexpr int kKv8WeightTokens = 2048;

template <int DT, int D, bool WEIGHTS>
__global__ void __launch_bounds__(256, WEIGHTS ? 6 : 4) kv8_finish_kernel(const Kv8Dec p) {
  constexpr int VEC = D / 32;
  __shared__ float s_o[8][D], s_m[8], s_l[8];
  __shared__ float2 s_norm[kKv8HeadGroup];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (WEIGHTS && (int)blockIdx.x < p.weights) {
    const int chunks = (int)ceil_div(p.g.capacity, kKv8WeightTokens);
    const int pair = (int)blockIdx.x / chunks, b = pair / p.g.Hkv, h = pair % p.g.Hkv;
    const int len = p.g.len(p.len, b), first = ((int)blockIdx.x % chunks) * kKv8WeightTokens;
    if (first >= len) return;
    const int n = kv8_units<D>(p, b), Gp = (p.Gc + 1) & ~1;
    const int2 count = kv8_count<D>(p, b);
    Kv8Plan plan;
    plan.set(count.x, p.ctas);
    float sum[kKv8WeightTokens / 256];
#pragma unroll
    for (int k = 0; k < kKv8WeightTokens / 256; ++k) sum[k] = 0.0f;
    pdl_wait();
    for (int part = 0; part < p.HG; ++part) {
      const int heads = min(p.Gc, p.G - part * p.Gc), u0 = count.y + (h * p.HG + part) * n;
      const int a = plan.owner(u0 + kKv8Head), z = plan.owner(u0 + n - 1);
      __syncthreads();  // s_norm has been read
      // maximum and 1 / sum of a head, its CTAs over the lanes
      for (int r = warp; r < heads; r += 8) {
        float M = -INFINITY, L = 0.0f;
        if (a == z && lane == 0) {
          const float2 ml = p.norm[(int64_t)b * p.H + h * p.G + part * p.Gc + r];
          M = ml.x;
          L = ml.y;
        }
        for (int c = a + lane; c <= z && a < z; c += 32) {
          const int64_t slot = 2 * (int64_t)c + (plan.first(c) < u0);
          const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + (slot * p.Gc + r) * 2);
          const float mn = fmaxf(M, ml.x), ref = mn == -INFINITY ? 0.0f : mn;
          L = L * exp2f(M - ref) + ml.y * exp2f(ml.x - ref);
          M = mn;
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
          const float m2 = __shfl_xor_sync(0xffffffffu, M, o);
          const float l2 = __shfl_xor_sync(0xffffffffu, L, o);
          const float mn = fmaxf(M, m2), ref = mn == -INFINITY ? 0.0f : mn;
          L = L * exp2f(M - ref) + l2 * exp2f(m2 - ref);
          M = mn;
        }
        if (lane == 0) s_norm[r] = make_float2(M, 1.0f / L);
      }
      __syncthreads();
      const float* s = p.scores + (((int64_t)pair * p.HG + part) * p.g.capacity + first + tid) * Gp;
      for (int r = 0; r < heads; r += 2) {
        const float2 n0 = s_norm[r], n1 = r + 1 < heads ? s_norm[r + 1] : make_float2(0.0f, 0.0f);
        float2 x[kKv8WeightTokens / 256];
#pragma unroll
        for (int k = 0; k < kKv8WeightTokens / 256; ++k)
          x[k] = first + 256 * k + tid < len
                     ? *reinterpret_cast<const float2*>(s + (int64_t)256 * k * Gp + r)
                     : make_float2(-INFINITY, -INFINITY);
#pragma unroll
        for (int k = 0; k < kKv8WeightTokens / 256; ++k) {
          sum[k] = fmaf(exp2f(x[k].x - n0.x), n0.y, sum[k]);
          if (r + 1 < heads) sum[k] = fmaf(exp2f(x[k].y - n1.x), n1.y, sum[k]);
        }
      }
    }
    float* w = p.weight + (int64_t)pair * p.g.capacity;
#pragma unroll
    for (int k = 0; k < kKv8WeightTokens / 256; ++k) {
      const int t = first + 256 * k + tid;
      if (t < len) w[t] += sum[k];
    }
    return;
  }
  const int groups = (p.Gc + (1 << p.lhc) - 1) >> p.lhc, per = p.g.Hkv * p.HG;
  const int i = blockIdx.x - (WEIGHTS ? p.weights : 0);
  const int b = i / groups / per, pair = i / groups % per;
  const int r0 = i % groups << p.lhc;  // the first of its heads in the part
  const int heads = min(1 << p.lhc, min(p.Gc, p.G - pair % p.HG * p.Gc) - r0);
  const int64_t bh = (int64_t)b * p.H + pair / p.HG * p.G + pair % p.HG * p.Gc + r0;
  const int n = kv8_units<D>(p, b);
  const int2 count = kv8_count<D>(p, b);
  Kv8Plan plan;
  plan.set(count.x, p.ctas);
  const int u0 = count.y + pair * n;
  const int a = n ? plan.owner(u0 + kKv8Head) : 0, z = n ? plan.owner(u0 + n - 1) : -1;
  const int split = 8 >> p.lhc, r = warp >> (3 - p.lhc);  // this warp's head
  pdl_wait();
  if (a == z || heads <= 0) return;
  float m = -INFINITY, l = 0.0f, o[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) o[e] = 0.0f;
  constexpr int BATCH = 4;  // parts whose loads are in flight together
  for (int c0 = a + (warp & (split - 1)); c0 <= z && r < heads; c0 += BATCH * split) {
    float2 ml[BATCH];
    float po[BATCH][VEC];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int c = c0 + k * split;
      ml[k] = make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int e = 0; e < VEC; ++e) po[k][e] = 0.0f;
      if (c <= z) {
        const int64_t slot = 2 * (int64_t)c + (plan.first(c) < u0);  // not its CTA's first stretch
        const int64_t at = slot * p.Gc + r0 + r;
        ml[k] = *reinterpret_cast<const float2*>(p.part_ml + at * 2);
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
          const float2 v = *reinterpret_cast<const float2*>(p.part_o + at * D + VEC * lane + e);
          po[k][e] = v.x;
          po[k][e + 1] = v.y;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const float mn = fmaxf(m, ml[k].x), ref = mn == -INFINITY ? 0.0f : mn;
      const float x = exp2f(m - ref), y = exp2f(ml[k].x - ref);
#pragma unroll
      for (int e = 0; e < VEC; ++e) o[e] = o[e] * x + po[k][e] * y;
      l = l * x + ml[k].y * y;
      m = mn;
    }
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) s_o[warp][VEC * lane + e] = o[e];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  for (int e = tid; e < heads * D; e += 256) {
    const int w0 = e / D * split, c = e % D;
    float M = -INFINITY, acc = 0.0f, L = 0.0f;
    for (int w = w0; w < w0 + split; ++w) M = fmaxf(M, s_m[w]);
    const float ref = M == -INFINITY ? 0.0f : M;
    for (int w = w0; w < w0 + split; ++w) {
      const float x = exp2f(s_m[w] - ref);
      acc += s_o[w][c] * x;
      L += s_l[w] * x;
    }
    p.out[bh * D + e] = f2h<DT>(n ? acc / L : 0.0f);
    if (c == 0) p.lse[bh + e / D] = n ? M * kLn2 + logf(L) : -INFINITY;
  }
}

// ------------------------------------------------------------------ evict --

// Order-preserving map of a weight to an unsigned key; NaN counts as -inf,
// -0 as +0.
__device__ __forceinline__ uint32_t kv8_key(float w) {
  const uint32_t u = __float_as_uint(w != w ? -INFINITY : w + 0.0f);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

constexpr int kKv8SelThreads = 1024, kKv8SelBins = 2048;
constexpr int kKv8SelCluster = 8;  // CTAs that share a head's tokens, at most

// Inclusive sum over the lanes.
__device__ __forceinline__ int warp_scan(int x) {
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if ((int)(threadIdx.x & 31) >= o) x += y;
  }
  return x;
}

// kept[b, h, i], i < min(len, budget): the tokens that stay, ascending: the
// first `sink`, the last `recent`, and the heaviest of the others, ties to
// the lower token.  A cluster of CTAs per (kv head, sequence), a warp a
// contiguous stretch of tokens: a radix select of 11, 11 and 10 bits over the
// candidates' keys, whose histograms are added over distributed shared memory
// (every CTA arrives at the same digit), then every warp writes the survivors
// of its stretch behind those of the lower ones.  KEEP: the tokens whose keys
// a thread holds in registers from one read; 0: every pass reads them again.
// Latency bounds it (a pass over histograms and barriers takes 2 to 3 us):
// 8 us for 64 heads of 4352 tokens, 14 for 8 heads of 131072.
template <int KEEP>
__global__ void __launch_bounds__(kKv8SelThreads) kv8_select_kernel(
    const float* __restrict__ weight, Kv8Geom g, const int32_t* __restrict__ seq_len, int budget,
    int sink, int recent, int32_t* __restrict__ kept, int32_t* __restrict__ len_out, int cl) {
  __shared__ uint32_t hist[2][kKv8SelBins];
  __shared__ uint32_t coarse[2][64], s_theirs[64 * kKv8SelCluster];
  __shared__ int s_gt[32], s_eq[32], s_bin, s_above;
  __shared__ __align__(8) uint32_t s_count[2];  // of this CTA
  __shared__ uint32_t s_prefix;
  __shared__ int s_rem, s_done;
  const int rank = blockIdx.x % cl, h = blockIdx.x / cl, b = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  const int len = g.len(seq_len, b);
  const int64_t bh = (int64_t)b * g.Hkv + h;
  const float* w = weight + bh * g.capacity;
  int32_t* out = kept + bh * budget;
  if (blockIdx.x == 0 && tid == 0) len_out[b] = min(len, budget);
  if (len <= budget) {
    for (int t = rank * kKv8SelThreads + tid; t < len; t += cl * kKv8SelThreads) out[t] = t;
    return;
  }
  const int lo = sink, hi = len - recent;  // candidates [lo, hi): more than are wanted
  const int steps = (int)ceil_div(len, cl * kKv8SelThreads);  // of 32 tokens a warp
  const int from = (int)min((int64_t)len, ((int64_t)rank * 32 + warp) * 32 * steps);
  const int to = (int)min((int64_t)len, (int64_t)from + 32 * steps);
  // Keys of this thread's tokens: all ones for a protected one (no number's
  // key is), 0 (nor is that) behind the stretch.
  auto key_of = [&](int t, float x) {
    const uint32_t k = kv8_key(x);
    return t >= to ? 0u : t < lo || t >= hi ? 0xFFFFFFFFu : k;
  };
  uint32_t key[KEEP > 0 ? KEEP : 1];
  if constexpr (KEEP > 0) {
    float x[KEEP];  // every load is on its way before the first is waited for
#pragma unroll
    for (int i = 0; i < KEEP; ++i) x[i] = ld_behind(w + min(from + 32 * i + lane, len - 1));
#pragma unroll
    for (int i = 0; i < KEEP; ++i) key[i] = key_of(from + 32 * i + lane, x[i]);
  }
  // f(token, key) for this thread's tokens, 32 consecutive ones a warp
  auto each = [&](auto f) {
    if constexpr (KEEP > 0) {
#pragma unroll
      for (int i = 0; i < KEEP; ++i)
        if (i < steps) f(from + 32 * i + lane, key[i]);
    } else {
      for (int i = 0; i < steps; i += 8) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = ld_behind(w + min(from + 32 * (i + j) + lane, len - 1));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int t = from + 32 * (i + j) + lane;
          f(t, key_of(t, x[j]));
        }
      }
    }
  };
  int rem = budget - sink - recent;
  uint32_t prefix = 0, pmask = 0;
  bool all = false;  // of the keys at the threshold
  if (rem == 0) {
    prefix = 0xFFFFFFFEu;  // above every number
    pmask = 0xFFFFFFFFu;
  } else {
    for (int i = tid; i < 2 * kKv8SelBins; i += kKv8SelThreads) (&hist[0][0])[i] = 0;
    __syncthreads();
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t mask = pass == 2 ? 1023u : 2047u;
      uint32_t* mine = hist[pass & 1];
      each([&](int t, uint32_t k) {
        if (k - 1u < 0xFFFFFFFEu && (k & pmask) == prefix)
          atomicAdd(&mine[(k >> shift) & mask], 1u);
      });
      // sums of 32 bins, two a warp; then of all CTAs: the 64 sums to find the 32
      // bins that hold the threshold, and those bins
      __syncthreads();
      uint32_t* sums = coarse[pass & 1];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t x = __reduce_add_sync(0xffffffffu, mine[64 * warp + 32 * i + lane]);
        if (lane == 0) sums[2 * warp + i] = x;
      }
      if (cl > 1)
        cluster_sync();
      else
        __syncthreads();
      auto theirs = [&](const uint32_t* at, int r) {
        if (r == rank) return *at;
        return r < cl ? __float_as_uint(ld_cluster(reinterpret_cast<const float*>(at), r)) : 0u;
      };
      if (tid < 64 * kKv8SelCluster) s_theirs[tid] = theirs(sums + (tid & 63), tid >> 6);
      __syncthreads();
      if (warp == 0) {
        const int top = 63 - 2 * lane;  // the lane's upper bin of the two
        int c0 = 0, c1 = 0;
#pragma unroll
        for (int r = 0; r < kKv8SelCluster; ++r) {
          c0 += (int)s_theirs[64 * r + top];
          c1 += (int)s_theirs[64 * r + top - 1];
        }
        const int above0 = warp_scan(c0 + c1) - c0 - c1, above1 = above0 + c0;
        if (above0 < rem && rem <= above1 + c1) {  // one lane
          s_bin = rem <= above1 ? top : top - 1;
          s_above = rem <= above1 ? above0 : above1;
        }
      }
      __syncthreads();
      const int bin0 = 32 * s_bin;
      if (tid < 32 * kKv8SelCluster) s_theirs[tid] = theirs(mine + bin0 + (tid & 31), tid >> 5);
      __syncthreads();
      if (warp == 0) {
        int c = 0;
#pragma unroll
        for (int r = 0; r < kKv8SelCluster; ++r) c += (int)s_theirs[32 * r + 31 - lane];
        const int above = s_above + warp_scan(c) - c;
        if (above < rem && rem <= above + c) {  // one lane
          s_rem = rem - above;
          s_prefix = prefix | (uint32_t)(bin0 + 31 - lane) << shift;
          s_done = c == s_rem;
        }
      }
      // the other buffer, free since every CTA of the cluster has come here
      if (pass == 1)
        for (int i = tid; i < kKv8SelBins; i += kKv8SelThreads) hist[0][i] = 0;
      __syncthreads();
      prefix = s_prefix;
      rem = s_rem;
      pmask |= mask << shift;
      all = s_done;
      if (all) break;  // the whole bucket is taken: the lower bits decide nothing
    }
  }
  // A token stays if protected, above the threshold, or one of the first
  // `rem` at it.
  if (all) {
    --prefix;  // the threshold itself is above this one
    pmask = 0xFFFFFFFFu;
    rem = 0;
  }
  int ngt = 0, neq = 0;
  each([&](int t, uint32_t k) {
    ngt += __popc(__ballot_sync(0xffffffffu, (k & pmask) > prefix));
    if (!all) neq += __popc(__ballot_sync(0xffffffffu, (k & pmask) == prefix));
  });
  if (lane == 0) {
    s_gt[warp] = ngt;
    s_eq[warp] = neq;
  }
  __syncthreads();
  int gt0 = __reduce_add_sync(0xffffffffu, lane < warp ? s_gt[lane] : 0);
  int eq0 = __reduce_add_sync(0xffffffffu, lane < warp ? s_eq[lane] : 0);
  if (cl > 1) {
    if (warp == 0) {
      const uint32_t gt = __reduce_add_sync(0xffffffffu, (uint32_t)s_gt[lane]);
      const uint32_t eq = __reduce_add_sync(0xffffffffu, (uint32_t)s_eq[lane]);
      if (lane == 0) {
        s_count[0] = gt;
        s_count[1] = eq;
      }
    }
    cluster_sync();
    const uint2 c = lane < rank ? ld_cluster2(s_count, lane) : make_uint2(0, 0);
    gt0 += (int)__reduce_add_sync(0xffffffffu, c.x);
    eq0 += (int)__reduce_add_sync(0xffffffffu, c.y);
  }
  const unsigned below = (1u << lane) - 1u;
  // in bounds whatever another stream may do to the weights meanwhile
  auto put = [&](int at, bool stays, int t) {
    if (stays && at < budget) out[at] = t;
  };
  each([&](int t, uint32_t k) {
    const bool gt = (k & pmask) > prefix;
    const unsigned mg = __ballot_sync(0xffffffffu, gt);
    if (all) {
      put(gt0 + __popc(mg & below), gt, t);
      gt0 += __popc(mg);
      return;
    }
    const bool eq = (k & pmask) == prefix;
    const unsigned me = __ballot_sync(0xffffffffu, eq);
    const int e = eq0 + __popc(me & below);
    // survivors before this token: all above, and the first rem of the equal
    put(gt0 + __popc(mg & below) + min(e, rem), gt || (eq && e < rem), t);
    gt0 += __popc(mg);
    eq0 += __popc(me);
  });
  if (cl > 1) cluster_sync();  // nobody leaves while its counts are read
}

// The kept tokens of a tile of the new cache, re-encoded under the scales of
// their new blocks: warps and tiles as in the append.  The maximum is taken
// over fp16 pairs (codes are exact fp16 numbers, and the larger of a number
// and a NaN is the number), one product with its scale a row.  Measured: 32768
// tokens of 8 heads (134 MB in and out) 25 us, 5.4 TB/s, bound by the chain of
// token number, codes, barrier and store, ten CTAs an SM deep (tiles of 128
// rows for the larger blocks: 1.5 us slower).
template <int D, int TILE>
__global__ void __launch_bounds__(kKv8Threads) kv8_gather_kernel(
    Kv8Geom g, Kv8Geom go, const uint8_t* __restrict__ k, const uint8_t* __restrict__ v,
    const float* __restrict__ ks, const float* __restrict__ vs, const float* __restrict__ weight,
    const int32_t* __restrict__ seq_len, const int32_t* __restrict__ kept, int budget,
    uint8_t* __restrict__ ko, uint8_t* __restrict__ vo, float* __restrict__ kso,
    float* __restrict__ vso, float* __restrict__ wo) {
  constexpr int TPR = D / 16, RPP = 32 / TPR;  // threads a row (16 codes each), rows a pass
  constexpr int ROWS = TILE / kKv8Warps, PASSES = ROWS / RPP;
  __shared__ float red[kKv8Warps];
  const int h = blockIdx.y >> 1, kv = blockIdx.y & 1, b = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = lane / TPR, c = 16 * (lane % TPR);
  const int n = min(g.len(seq_len, b), budget);
  const int w0 = (int)blockIdx.x * TILE + warp * ROWS;  // this warp's rows
  // Also by a CTA without rows: where every sequence is empty nothing else
  // would keep what follows this kernel from overtaking the select, which
  // still writes the lengths.
  pdl_wait();
  if ((int)blockIdx.x * TILE >= n) return;
  const int wpb = g.blk > ROWS ? g.blk / ROWS : 1;
  const int64_t bh = (int64_t)b * g.Hkv + h;
  const uint8_t* codes = (kv ? v : k) + g.row(b, h, 0) + c;
  const float* scales = (kv ? vs : ks) + g.scale(b, h, 0);
  const int lb = 31 - __clz(g.blk);  // blk is a power of two
  int src[PASSES];
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int i = w0 + p * RPP + row;
    src[p] = i < n ? min(max(0, ld_behind_l2(kept + bh * budget + i)), g.capacity - 1) : -1;
  }
  uint4 w[PASSES];
  float s[PASSES];
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    w[p] = make_uint4(0, 0, 0, 0);
    s[p] = 0.0f;
    if (src[p] >= 0) {
      w[p] = ld_stream16(codes + src[p] * g.st);
      s[p] = __ldg(scales + (src[p] >> lb));
    }
  }
  if (!kv && c == 0) {
#pragma unroll
    for (int p = 0; p < PASSES; ++p)
      if (src[p] >= 0)
        wo[bh * go.capacity + w0 + p * RPP + row] = __ldg(weight + bh * g.capacity + src[p]);
  }
  float a = 0.0f;
  uint32_t nan = 0;  // a bit of every byte that is a NaN
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const uint32_t x[4] = {w[p].x, w[p].y, w[p].z, w[p].w};
    __half2 top = __float2half2_rn(0.0f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t m = x[j] & 0x7F7F7F7Fu;
      nan |= (m + 0x01010101u) & 0x80808080u;
      uint32_t lo, hi;
      e4m3x4_f16(m, lo, hi);
      top = __hmax2(top, *reinterpret_cast<const __half2*>(&lo));
      top = __hmax2(top, *reinterpret_cast<const __half2*>(&hi));
    }
    const float2 f = __half22float2(top);
    const float y = fmaxf(f.x, f.y) * fabsf(s[p]);
    // 256 * 2^120, what the largest bf16 values round to, is no fp32 number
    a = fmaxf(a, finite_f(y) ? y : finite_f(s[p]) ? FLT_MAX : 0.0f);
  }
  const bool odd = __any_sync(0xffffffffu, nan != 0);
  a = warp_max(a);
  if (lane == 0) red[warp] = a;
  __syncthreads();
  if (w0 / g.blk * g.blk >= n) return;
  const float so = kv8_scale(kv8_join(red, warp, wpb));
  uint8_t* to = (kv ? vo : ko) + go.row(b, h, w0) + c;
  // Rows whose scale stays are copied; the others are one product by the ratio
  // of the scales, in two factors where it is no fp16 number (products below
  // 2^-10 end as zeros, however far).
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int e = (int)(__float_as_uint(s[p]) >> 23) - (int)(__float_as_uint(so) >> 23);
    if (odd || __any_sync(0xffffffffu, src[p] >= 0 && e != 0)) {
      const int e1 = max(-14, min(15, e)), e2 = max(-14, min(15, e - e1));
      const __half2 f1 = __half2half2(__ushort_as_half((uint16_t)((e1 + 15) << 10)));
      const __half2 f2 = __half2half2(__ushort_as_half((uint16_t)((e2 + 15) << 10)));
      const bool far = __any_sync(0xffffffffu, e2 != 0);
      uint32_t x[4] = {w[p].x, w[p].y, w[p].z, w[p].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t lo, hi;
        e4m3x4_f16(x[j], lo, hi);
        __half2 l = __hmul2(*reinterpret_cast<const __half2*>(&lo), f1);
        __half2 u = __hmul2(*reinterpret_cast<const __half2*>(&hi), f1);
        if (far) {
          l = __hmul2(l, f2);
          u = __hmul2(u, f2);
        }
        x[j] = f16_e4m3x2(l) | (f16_e4m3x2(u) << 16);
      }
      w[p] = make_uint4(x[0], x[1], x[2], x[3]);
    }
    if (src[p] >= 0) *reinterpret_cast<uint4*>(to + (p * RPP + row) * go.st) = w[p];
  }
  if (lane == 0 && w0 % g.blk == 0) (kv ? vso : kso)[go.scale(b, h, w0 >> lb)] = so;
}

}  // namespace thrift
