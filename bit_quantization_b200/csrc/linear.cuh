// y = x W^T with NVFP4 weights as nvfp4_quantize leaves them (E2M1 codes
// [N, K/2], UE4M3 scales [N, K/16] of 16-element blocks, fp32 tensor scale)
// and few 16-bit rows x [M, K]: the projections of a generation step.
//
//   y[m, n] = g * sum_k x[m, k] e2m1(code[n, k]) ue4m3(scale[n, k / 16])
//
// A weight is read once and used M times: the bytes of the weights (0.5625 a
// weight) bound it, so nothing may stand between them and the tensor cores.
// The block-scaled FP4 products take codes and scales as they are, as the
// 128-row operand.  What they ask for is x in FP4 too, and x is given to them
// exactly enough as a sum of FP4 rows: with s a power of two such that a
// 16-block of x lies within 4 s, the digits
//   d_0 = e2m1(x / s), d_1 = e2m1(8 (x / s - d_0)), ...
// are at most 4 (E2M1 steps by at most 1 up to there, which leaves 1/2, and 8
// times 1/2 is 4 again), and six of them leave at most 2^-17 of the block's
// largest value.  All digits of a block have the scale s; column 6 m + i of
// the product is digit i of row m, and 8^-i is applied to its fp32 sum.  Rows
// are first brought by a power of two to s <= 2^8, so that s down to 2^-9 is a
// UE4M3 number: blocks further below keep an error of 2^-34 of the row's
// largest value.
//
// Converting the codes in registers for 16-bit products was measured too: 84
// us for 4 x 4096 x 128256 and 178 for 16 rows, bound by instructions.
#pragma once
#include <cuda.h>

#include "tc.cuh"

namespace thrift {

using PFN_encode_tiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                      const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                      const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                      CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

constexpr int kLinMaxM = 64;        // rows a call
constexpr int kLinMaxK = 1 << 19;
constexpr int kLinGroup = 16;       // rows of x in one pass over the weights
constexpr int kLinDigits = 6;
constexpr int kLinChunk = 256;      // K of one stage: 128 bytes of codes a weight row
constexpr int kLinMaxCtas = 256;    // one an SM
constexpr int kLinDigitThreads = 512;  // 8 values of x each
constexpr uint32_t kLinABytes = 128 * (kLinChunk / 2);  // codes of 128 weight rows
constexpr uint32_t kLinSfBytes = (kLinChunk / 64) * 512;  // a scale-factor image

// Digit columns of up to `rows` rows of x, a multiple of 16.
__host__ __device__ constexpr int lin_cols(int rows) { return (kLinDigits * rows + 15) / 16 * 16; }
// x of one chunk: digits (rows of 128 bytes, swizzled), then their scales.
__host__ __device__ constexpr uint32_t lin_img(int cols) { return cols * 128 + kLinSfBytes; }

// Workspace: per CTA and quarter of its rows, arrivals at a shared tile
// (uint32 [kLinMaxCtas][4]); per row of x its unit (fp32 [64]); the images of
// x [group][chunk]; partial sums of shared tiles [CTA][2][rows][128].
constexpr size_t kLinOffUnit = kLinMaxCtas * 16, kLinOffImg = kLinOffUnit + 1024;

struct LinParams {
  const uint16_t* x;
  const uint8_t* scales;
  const float* gs;
  uint16_t* y;
  uint8_t* ws;
  int64_t img;  // images of x: ws + img.  Partial sums: ws + part
  int64_t part;
  int M, K, N;
  int cols, chunks;
  int run, longer;  // units a CTA takes; the first `longer` of them one more
};

// A unit of work: chunk c of weight tile `tile` for group `grp` of rows of x.
struct LinUnit {
  int c, tile, grp;
  __device__ __forceinline__ void next(int chunks, int ntiles) {
    if (++c == chunks) {
      c = 0;
      if (++tile == ntiles) {
        tile = 0;
        ++grp;
      }
    }
  }
};

// A byte of two E2M1 codes -> their values.
__device__ __forceinline__ float2 e2m1x2_decode(uint32_t c) {
  uint32_t h;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t}"
      : "=r"(h)
      : "r"(c));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// ----------------------------------------------------------------- digits --

// `parts` CTAs a row of x: each finds the row's largest value for itself (from
// L2, which is quicker than asking the others), then every thread writes the
// digits of 8 values, two threads the scale of a block of 16.
template <int DT>
__global__ void __launch_bounds__(kLinDigitThreads)
    lin_digits_kernel(const LinParams p, int parts) {
  __shared__ uint32_t s_max;
  const int m = blockIdx.x / parts, rank = blockIdx.x % parts, tid = threadIdx.x;
  if (tid == 0) s_max = 0;
  pdl_wait();
  pdl_trigger();  // the products may fetch weights: nothing before this writes them now
  if (blockIdx.x == 0)
    for (int i = tid; i < kLinMaxCtas * 4; i += kLinDigitThreads)
      reinterpret_cast<uint32_t*>(p.ws)[i] = 0;
  __syncthreads();
  const uint4* src = reinterpret_cast<const uint4*>(p.x + (int64_t)m * p.K);
  const int n8 = p.K / 8, first = rank * kLinDigitThreads + tid, step = parts * kLinDigitThreads;
  uint32_t a = 0;  // bits of |x|: ordered, infinities and NaN on top
#pragma unroll 4
  for (int i = tid; i < n8; i += kLinDigitThreads) {
    const uint4 v = ld_behind(src + i);
    const uint32_t w = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
    a = __vmaxu2(a, w);
  }
  a = __reduce_max_sync(0xffffffffu, max(a & 0xFFFFu, a >> 16));
  if ((tid & 31) == 0) atomicMax(&s_max, a);
  __syncthreads();
  a = s_max;
  const bool finite = a < (DT == 1 ? 0x7F80u : 0x7C00u);
  // the largest value to [2^9, 2^10), in two factors: 2^135 is not an fp32 number
  const float top = h2f<DT>((uint16_t)a);
  const int E = top > 0.0f && finite ? (int)(__float_as_uint(top) >> 23) - 127 : 0;
  const int e = 9 - E, e1 = e >> 1, e2 = e - e1;
  const float f1 = __uint_as_float((uint32_t)(127 + e1) << 23);
  const float f2 = __uint_as_float((uint32_t)(127 + e2) << 23);
  if (rank == 0 && tid == 0)
    reinterpret_cast<float*>(p.ws + kLinOffUnit)[m] = finite ? 1.0f / f1 / f2 : NAN;
  const int grp = m / kLinGroup, col = kLinDigits * (m % kLinGroup);
  uint8_t* img = p.ws + p.img + (int64_t)grp * p.chunks * lin_img(p.cols);
  // the last chunk is written to its end: its weights are zeros there, x too
  for (int i = first; i < p.chunks * (kLinChunk / 8); i += step) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (i < n8 && finite) v = ld_behind(src + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float x[8], top8 = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = h2f<DT>((uint16_t)(j & 1 ? w[j >> 1] >> 16 : w[j >> 1] & 0xFFFFu)) * f1 * f2;
      top8 = fmaxf(top8, fabsf(x[j]));
    }
    top8 = fmaxf(top8, __shfl_xor_sync(0xffffffffu, top8, 1));
    // s = 2^ex: top in [2 s, 4 s) within s's range
    const int ex = min(8, max(-9, (int)(__float_as_uint(top8) >> 23) - 128));
    const float inv = __uint_as_float((uint32_t)(127 - ex) << 23);
    const uint32_t sf = ex >= -6 ? (uint32_t)(ex + 7) << 3 : 1u << (ex + 9);
    const int c = i / (kLinChunk / 8), k8 = i % (kLinChunk / 8);
    uint8_t* at = img + (int64_t)c * lin_img(p.cols);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= inv;
#pragma unroll
    for (int d = 0; d < kLinDigits; ++d) {
      uint32_t code = 0;
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const uint32_t b = e2m1x2(x[j], x[j + 1]);
        const float2 q = e2m1x2_decode(b);
        x[j] = (x[j] - q.x) * 8.0f;
        x[j + 1] = (x[j + 1] - q.y) * 8.0f;
        code |= b << (4 * j);
      }
      *reinterpret_cast<uint32_t*>(at + swz_offset(col + d, 4 * k8, 128)) = code;
      if (!(k8 & 1)) at[p.cols * 128 + sf_offset(col + d, k8 >> 1)] = (uint8_t)sf;
    }
  }
}

// ---------------------------------------------------------------- product --
//
// Work is a row of units (group of 16 rows of x, tile of 128 weight rows,
// chunk of 256 along K) in that order, dealt to the CTAs (one an SM) in equal
// runs, so that every SM streams the same number of bytes whatever N and K
// are.  A run covers parts of tiles: a tile that is not one CTA's alone is
// added up from partial sums by the last of its CTAs to arrive, in the order
// of the CTAs, so that results repeat bit for bit.
//
// One warp has codes (a tensor map, 128-byte swizzle) and x (plain copies of
// ready images) brought to a ring of stages by the copy unit; four warps put
// the scales, a row a thread, into the order the tensor cores want; one warp
// issues; four warps read the sums.  Measured: 4 x 4096 x 128256 52 us (5.7 TB/s
// of weights; 60 while the scales came 16 bytes a row at a time, 50 without their
// loads), 16 rows 54; 1 x 4096 x 1024 7 us, of which bytes are 0.4: two
// dependent kernels, and 2 to 3 us for the join of shared tiles.

template <int ROWS>
struct LinLayout {
  static constexpr int COLS = lin_cols(ROWS);
  static constexpr uint32_t B = kLinABytes, SFB = B + COLS * 128, SFA = SFB + kLinSfBytes;
  static constexpr uint32_t STAGE = SFA + kLinSfBytes;
  static constexpr int STAGES = (int)(205 * 1024 / STAGE) < 8 ? (int)(205 * 1024 / STAGE) : 8;
  static constexpr uint32_t OFF_BAR = STAGES * STAGE;
  static constexpr uint32_t SMEM = OFF_BAR + (2 * STAGES + 4) * 8 + 16 + 1024;
  // tensor memory: two sums, two sets of scale factors
  static constexpr uint32_t T_SF = 192, T_COLS = 256;
  static_assert(2 * COLS <= T_SF && STAGE % 1024 == 0, "layout");
};

constexpr int kLinSfWarp = 2, kLinEpiWarp = 6, kLinThreads = 32 * 10;

template <int DT, int ROWS>
__global__ void __launch_bounds__(kLinThreads, 1) linear_kernel(
    const __grid_constant__ CUtensorMap map, const LinParams p) {
  using L = LinLayout<ROWS>;
  extern __shared__ uint8_t lin_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(lin_raw) + 1023) &
                                           ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::OFF_BAR);
  uint64_t* empty = full + L::STAGES;
  uint64_t* sum_full = empty + L::STAGES;
  uint64_t* sum_empty = sum_full + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sum_empty + 2);
  volatile int* s_abort = reinterpret_cast<int*>(s_tmem + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < L::STAGES; ++i) {
      mbar_init(full + i, 1 + 4);  // the copies, and a warp for 32 rows' scales
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sum_full + i, 1);
      mbar_init(sum_empty + i, 128);
    }
    *s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, L::T_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  const int chunks = p.chunks, ntiles = (int)ceil_div(p.N, 128), cta = blockIdx.x;
  const int n = p.run + (cta < p.longer);
  const int u0 = p.run * cta + min(cta, p.longer);
  LinUnit u;
  u.c = u0 % chunks;
  u.tile = u0 / chunks % ntiles;
  u.grp = u0 / chunks / ntiles;

  if (warp == 0) {
    if (lane == 0) {
      auto codes = [&](int sl, const LinUnit& q) {
        tma_load_2d(sm + sl * L::STAGE, &map, q.c * (kLinChunk / 2), q.tile * 128, full + sl);
      };
      auto digits = [&](int sl, const LinUnit& q) {
        bulk_g2s(sm + sl * L::STAGE + L::B,
                 p.ws + p.img + ((int64_t)q.grp * chunks + q.c) * lin_img(L::COLS),
                 lin_img(L::COLS), full + sl);
      };
      const int ahead = min(n, L::STAGES);
      LinUnit q = u;
      for (int k = 0; k < ahead; ++k) {  // the weights do not wait for the digits
        mbar_arrive_expect_tx(full + k, kLinABytes + lin_img(L::COLS));
        codes(k, q);
        q.next(chunks, ntiles);
      }
      pdl_wait();
      for (int k = 0; k < ahead; ++k) {
        digits(k, u);
        u.next(chunks, ntiles);
      }
      int k = ahead, sl = 0, par = 0;
      for (; k < n; ++k) {
        if (sl == L::STAGES) {
          sl = 0;
          par ^= 1;
        }
        if (!mbar_wait(empty + sl, par, s_abort)) break;
        mbar_arrive_expect_tx(full + sl, kLinABytes + lin_img(L::COLS));
        codes(sl, u);
        digits(sl, u);
        u.next(chunks, ntiles);
        ++sl;
      }
      // every copy has landed before the CTA ends
      int dummy = 0;
      for (int i = max(0, k - L::STAGES); i < k; ++i)
        mbar_wait(full + i % L::STAGES, (i / L::STAGES) & 1, &dummy, 200000000ull);
    }
  } else if (warp == 1) {
    const bool leader = elect_one();
    const uint32_t base = smem_u32(sm);
    const uint64_t d_sf = make_sdesc(base, 512, 128, SW_NONE);
    const uint64_t d_ab = make_sdesc(base, 16, 1024, SW_128B);
    constexpr uint32_t id = idesc_nvf4(128, L::COLS);
    int seg = 0, sl = 0, par = 0, c = u.c;
    for (int k = 0; k < n; ++k) {
      const bool first = k == 0 || c == 0, last = k + 1 == n || c + 1 == chunks;
      if (first && seg >= 2 &&
          !__all_sync(0xffffffffu, mbar_wait(sum_empty + (seg & 1), ((seg >> 1) - 1) & 1, s_abort)))
        break;
      if (!__all_sync(0xffffffffu, mbar_wait(full + sl, par, s_abort))) break;
      tc_fence_after();
      if (leader) {
        const uint32_t stg = sl * L::STAGE, sf = tmem + L::T_SF + 32 * (k & 1);
#pragma unroll
        for (int j = 0; j < kLinChunk / 64; ++j) {
          tc_cp_32x128b_x4(sf + 4 * j, d_sf + ((stg + L::SFA + 512 * j) >> 4));
          tc_cp_32x128b_x4(sf + 16 + 4 * j, d_sf + ((stg + L::SFB + 512 * j) >> 4));
        }
#pragma unroll
        for (int j = 0; j < kLinChunk / 64; ++j)
          mma_nvf4(tmem + L::COLS * (seg & 1), d_ab + (stg >> 4) + 2 * j,
                   d_ab + ((stg + L::B) >> 4) + 2 * j, id, sf + 4 * j, sf + 16 + 4 * j,
                   !first || j > 0);
        tc_commit(empty + sl);
        if (last) tc_commit(sum_full + (seg & 1));
      }
      __syncwarp();
      seg += last;
      c = c + 1 == chunks ? 0 : c + 1;
      if (++sl == L::STAGES) {
        sl = 0;
        par ^= 1;
      }
    }
  } else if (warp < kLinEpiWarp) {
    // ------------------------------------------------- weights' scales --
    const int row = tid - 32 * kLinSfWarp;
    const int64_t lds = p.K / 16;
    const bool whole = p.K % kLinChunk == 0;  // 16 aligned bytes a row and chunk
    auto load = [&](int k) {  // units in order
      uint4 v = make_uint4(0, 0, 0, 0);
      if (k >= n) return v;
      const int64_t r = u.tile * 128 + row;
      const int c = u.c;
      u.next(chunks, ntiles);
      if (r >= p.N) return v;
      const uint8_t* s = p.scales + r * lds + c * 16;
      if (whole) return __ldg(reinterpret_cast<const uint4*>(s));
      uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c * 16 + 2 * i < lds)
          w[i >> 1] |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(s) + i) << (16 * (i & 1));
      return make_uint4(w[0], w[1], w[2], w[3]);
    };
    // four units' scales (mostly 64 neighbouring bytes of a row) are loaded
    // together while the four before are stored
    constexpr int AHEAD = 4;
    uint4 next[AHEAD], ring[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) next[i] = load(i);
    bool ok = true;
    int sl = 0, par = 1;  // of the stage's previous use; none in the first round
    for (int k0 = 0; k0 < n && ok; k0 += AHEAD) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) ring[i] = next[i];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) next[i] = load(k0 + AHEAD + i);
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int k = k0 + i;
        if (k >= n || !ok) continue;
        const uint4 v = ring[i];
        if (k >= L::STAGES)
          ok = __all_sync(0xffffffffu, mbar_wait(empty + sl, par, s_abort));
        if (!ok) continue;
        uint32_t* to = reinterpret_cast<uint32_t*>(sm + sl * L::STAGE + L::SFA + sf_offset(row, 0));
        to[0] = v.x;
        to[128] = v.y;
        to[256] = v.z;
        to[384] = v.w;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full + sl);
        if (++sl == L::STAGES) {
          sl = 0;
          par ^= 1;
        }
      }
    }
  } else {
    // ------------------------------------------------------------- sums --
    auto owner = [&](int unit) {
      const int lead = p.longer * (p.run + 1);
      return unit < lead ? unit / (p.run + 1) : p.longer + (unit - lead) / p.run;
    };
    pdl_wait();
    const int quarter = warp & 3, row = 32 * quarter + lane;
    const float g = __ldg(p.gs);
    uint32_t* arrived = reinterpret_cast<uint32_t*>(p.ws);
    const float* unit = reinterpret_cast<const float*>(p.ws + kLinOffUnit);
    float* part = reinterpret_cast<float*>(p.ws + p.part) + row;
    int seg = 0;
    for (int k = 0; k < n; ++seg) {
      const int len = min(n - k, chunks - u.c), grp = u.grp, t = grp * ntiles + u.tile;
      const int64_t w = (int64_t)u.tile * 128 + row;
      const int M = min(kLinGroup, p.M - grp * kLinGroup);
      uint16_t* y = p.y + (int64_t)grp * kLinGroup * p.N + w;
      k += len;
      u.c = chunks - 1;
      u.next(chunks, ntiles);
      if (!__all_sync(0xffffffffu, mbar_wait(sum_full + (seg & 1), (seg >> 1) & 1, s_abort))) break;
      tc_fence_after();
      float acc[L::COLS];
#pragma unroll
      for (int i = 0; i < L::COLS; i += 16)
        tmem_ld16(tmem + L::COLS * (seg & 1) + i + ((uint32_t)(32 * quarter) << 16), acc + i);
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive(sum_empty + (seg & 1));
      float v[ROWS];
#pragma unroll
      for (int m = 0; m < ROWS; ++m) {
        v[m] = 0.0f;
#pragma unroll
        for (int d = kLinDigits - 1; d >= 0; --d)
          v[m] = fmaf(v[m], 0.125f, acc[kLinDigits * m + d]);
      }
      if (len < chunks) {
        // a shared tile: CTAs a .. b have a part of it
        const int first = t * chunks, a = owner(first), b = owner(first + chunks - 1);
        const bool second = p.run * a + min(a, p.longer) < first;  // not a's first tile
        float* mine = part + (int64_t)(2 * cta + (seg > 0)) * ROWS * 128;
#pragma unroll
        for (int m = 0; m < ROWS; ++m)
          if (m < M) __stcg(mine + m * 128, v[m]);
        __syncwarp();
        uint32_t before = 0;
        if (lane == 0) before = atom_add_acq_rel(arrived + 4 * a + quarter, 1u);
        if (__shfl_sync(0xffffffffu, before, 0) != (uint32_t)(b - a)) continue;
        __syncwarp();  // what lane 0 has acquired is the warp's
        // in the order of the CTAs, the loads of BATCH of them together
        constexpr int BATCH = 16 / ROWS;
        const float* theirs = part + (int64_t)2 * a * ROWS * 128;
#pragma unroll
        for (int m = 0; m < ROWS; ++m)
          v[m] = m < M ? ld_behind_l2(theirs + (second * ROWS + m) * 128) : 0.0f;
        for (int i = 1; i <= b - a; i += BATCH) {
          float got[BATCH][ROWS];
#pragma unroll
          for (int j = 0; j < BATCH; ++j)
#pragma unroll
            for (int m = 0; m < ROWS; ++m)
              got[j][m] = i + j <= b - a && m < M
                              ? ld_behind_l2(theirs + (int64_t)(2 * (i + j) * ROWS + m) * 128)
                              : 0.0f;
#pragma unroll
          for (int j = 0; j < BATCH; ++j)
#pragma unroll
            for (int m = 0; m < ROWS; ++m) v[m] += got[j][m];
        }
      }
      if (w < p.N) {
#pragma unroll
        for (int m = 0; m < ROWS; ++m)
          if (m < M) y[(int64_t)m * p.N] = f2h<DT>(v[m] * g * unit[grp * kLinGroup + m]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, L::T_COLS);
}

}  // namespace thrift
