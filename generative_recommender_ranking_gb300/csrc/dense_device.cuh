// dense_device.cuh -- what the kernels of the matrix products share: the gate's activation, the stores
// of result rows and the walk over the tiles.
#pragma once

#include <cuda_bf16.h>

#include "dense.cuh"
#include "ptx_sm103.cuh"
#include "rec_attn_internal.cuh"

namespace recattn {

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Pairs of fp32 for the packed instructions (two values an issue).
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair_of(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ f32x2 pair_of_bits(uint32_t a, uint32_t b) {
  return pair_of(__uint_as_float(a), __uint_as_float(b));
}
__device__ __forceinline__ float2 values_of(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 fma_pairs(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ f32x2 mul_pairs(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add_pairs(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(f32x2 v) {
  const float2 f = values_of(v);
  return pack_bf16(f.x, f.y);
}

// The hardware's 2^x and 1 / x (off by 2^-22 and 2^-23; results and operands below the normal numbers are zero).
__device__ __forceinline__ float exp2_hw(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_hw(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ f32x2 exp2_hw(f32x2 x) {
  const float2 v = values_of(x);
  return pair_of(exp2_hw(v.x), exp2_hw(v.y));
}
// Of two values from 1 to 2^62, by the reciprocal of their product (the special-function unit, at an eighth of
// the others' rate, bounds the epilogues).
__device__ __forceinline__ f32x2 rcp_hw(f32x2 x) {
  const float2 v = values_of(x);
  const float r = rcp_hw(v.x * v.y);
  return mul_pairs(pair_of(v.y, v.x), pair_of(r, r));
}
__device__ __forceinline__ f32x2 min_pairs(f32x2 a, float most) {  // (NaN: most)
  const float2 v = values_of(a);
  return pair_of(fminf(v.x, most), fminf(v.y, most));
}
__device__ __forceinline__ f32x2 both(float v) { return pair_of(v, v); }

// Phi(g) of the normal distribution, and e^(-g^2/2): for z = |g| / sqrt(2), erfc(z) / 2 = e^(-z^2) t (c1 + t (c2 + t (c3 +
// t (c4 + t c5)))), t = 1 / (1 + q z), the form of Abramowitz and Stegun 7.1.26.  Its own coefficients bound the absolute
// error alone (0.4% of Phi at -6, 3.7% at -13); these were fitted by a linear program to e^(z^2) erfc(z) / 2 up to z =
// 9.45: Phi is off by 8e-7 at most, and the side below zero by 4e-4 of itself too (a fifth of a bf16 rounding), down to
// -13.2 where the exponential is zero.  (A sixth term, 2e-7 and 2.5e-4, took the e4m3 block of 512 to 1024 columns on
// 320016 rows from 754 to 805 us, for registers.)  The exponential is shared with the slope.
__device__ __forceinline__ f32x2 normal_cdf(f32x2 g, f32x2& density) {
  const f32x2 t = rcp_hw(fma_pairs(both(0.70710678f * 0.4975f), min_pairs(g & 0x7fffffff7fffffffull, 1e18f), both(1.f)));
  density = exp2_hw(mul_pairs(mul_pairs(g, g), both(-0.72134752f)));  // log2(e) / 2
  f32x2 s = fma_pairs(t, both(-0.0957419881f), both(0.264943538f));
  s = fma_pairs(t, s, both(0.0297439802f));
  s = fma_pairs(t, s, both(0.162609824f));
  s = fma_pairs(t, s, both(0.138444008f));
  s = mul_pairs(mul_pairs(t, s), density);
  const float2 v = values_of(g), w = values_of(s);
  return pair_of(v.x > 0.f ? 1.f - w.x : w.x, v.y > 0.f ? 1.f - w.y : w.y);
}

// a b + c, from 0 to 1.
__device__ __forceinline__ float fma_sat(float a, float b, float c) {
  float r;
  asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// 1 / (1 + e^-g) less 2^-60, where it would stay from -41.6 down: a gate that is closed by a large value has the
// weight 0 and no gradient, whatever its size.  (From -34 up that is less than half a bf16 step of it; the exact form
// from e^-|g| takes five more instructions: 320016 rows through an e4m3 block of 512 x 1024 750 us against 724.)
// e: e^-g, up to 2^60.
__device__ __forceinline__ f32x2 logistic(f32x2 g, f32x2& e) {
  e = exp2_hw(min_pairs(mul_pairs(g, both(-1.44269504f)), 60.f));
  const float2 v = values_of(add_pairs(e, both(1.f)));
  const float r = rcp_hw(v.x * v.y), floor = -0x1.00002p-60f;  // (2^-60 and the reciprocal's error)
  return pair_of(fma_sat(r, v.y, floor), fma_sat(r, v.x, floor));
}

// act(g) of two values, and its derivative, for results in 16 bits and fewer.  silu: g / (1 + e^-g).  gelu: g Phi(g).
template <int ACT>
__device__ __forceinline__ f32x2 act_value(f32x2 g) {
  if (ACT == REC_ATTN_SILU) {
    f32x2 e;
    return mul_pairs(g, logistic(g, e));
  }
  f32x2 density;
  return mul_pairs(g, normal_cdf(g, density));
}
template <int ACT>
__device__ __forceinline__ f32x2 act_both(f32x2 g, f32x2& slope) {
  if (ACT == REC_ATTN_SILU) {
    // 1 - p as e^-g p: p of an open gate may be 2^-24 short of one, which a large g would make a slope of its own
    f32x2 e;
    const f32x2 p = logistic(g, e), v = mul_pairs(g, p);
    slope = fma_pairs(v, mul_pairs(e, p), p);
    return v;
  }
  f32x2 density;
  const f32x2 p = normal_cdf(g, density);
  slope = fma_pairs(g, mul_pairs(density, both(0.39894228f)), p);
  return mul_pairs(g, p);
}
// The same for fp32 results: Phi by the complementary error function, and the library's exponential and division keep
// its last bits.
template <int ACT>
__device__ __forceinline__ float act32(float g, float& slope) {
  if (ACT == REC_ATTN_SILU) {
    const float p = 1.f / (1.f + expf(-g)), v = g * p;
    slope = fmaf(v, 1.f - p, p);
    return v;
  }
  const float p = 0.5f * erfcf(-0.70710678f * g);
  slope = fmaf(g, 0.39894228f * expf(-0.5f * g * g), p);
  return g * p;
}

// 32 columns of a row in bf16; `left` columns of the result remain from the first on (a multiple of
// 8).  wide: the row starts on a 32-byte boundary.  Whole sectors are written, of other rows (every second one, where
// the width is an odd multiple of 8) between the first and the last 16 bytes: dx of 40000 x 520 with hidden 1024
// 239 -> 234 us, and twice as much where more is stored.
__device__ __forceinline__ void store_bf16(__nv_bfloat16* dst, const uint32_t (&w)[16], int left, bool wide) {
  char* const at = reinterpret_cast<char*>(dst);
  if (left >= 32 && (wide || (reinterpret_cast<uintptr_t>(dst) & 31) == 0)) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
      ptx::st_global_v8(at + 32 * c, w[8 * c], w[8 * c + 1], w[8 * c + 2], w[8 * c + 3], w[8 * c + 4], w[8 * c + 5],
                        w[8 * c + 6], w[8 * c + 7]);
  } else if (left >= 32) {
    *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
    ptx::st_global_v8(at + 16, w[4], w[5], w[6], w[7], w[8], w[9], w[10], w[11]);
    *reinterpret_cast<uint4*>(at + 48) = make_uint4(w[12], w[13], w[14], w[15]);
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (8 * c < left) reinterpret_cast<uint4*>(dst)[c] = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  }
}

// 16 columns.
__device__ __forceinline__ void store_bf16(__nv_bfloat16* dst, const uint32_t (&w)[8], int left, bool wide) {
  if (left >= 16 && (wide || (reinterpret_cast<uintptr_t>(dst) & 31) == 0)) {
    ptx::st_global_v8(dst, w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7]);
  } else {
#pragma unroll
    for (int c = 0; c < 2; ++c)
      if (8 * c < left) reinterpret_cast<uint4*>(dst)[c] = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  }
}

// Tiles in bands of 16 row tiles, row tiles fastest: the CTAs at work together share a band's rows and the
// columns' weights in the L2.  A walk from tile t on in equal steps, without a division at each.
struct TileWalk {
  int tiles_m, band_size, band, in;  // in: tiles of the band before this one
  __device__ __forceinline__ TileWalk(int t, int rows, int columns) : tiles_m(rows), band_size(16 * columns) {
    band = t / band_size;
    in = t - band * band_size;
  }
  __device__ __forceinline__ void advance(int step) {
    in += step;
    while (in >= band_size) {
      in -= band_size;
      ++band;
    }
  }
  __device__ __forceinline__ int2 at() const {  // row and column tile
    const int rows = tiles_m - 16 * band;
    return rows >= 16 ? make_int2(band * 16 + (in & 15), in >> 4) : make_int2(band * 16 + in % rows, in / rows);
  }
};

struct Unit {
  int m0, n0, kb0, kb1, split;
};

// A pair's units in turn; m0: this CTA's first row.  (Parts of the summed axis: all tiles of one, then of the
// next; the first a.kblocks % a.splits parts have a block more.  PARTS false: there is one.)
template <int TN, typename Args, bool PARTS = true>
struct Units {
  const Args& a;
  int i, n, step, tiles, split;
  uint32_t rank;
  TileWalk walk;
  __device__ __forceinline__ Units(const Args& args, uint32_t r)
      : a(args), i((int)blockIdx.x / 2), n(args.tiles_m * args.tiles_n * (PARTS ? args.splits : 1)), step((int)gridDim.x / 2),
        tiles(args.tiles_m * args.tiles_n), split(0), rank(r), walk(i, args.tiles_m, args.tiles_n) {
    settle();
  }
  __device__ __forceinline__ bool left() const { return i < n; }
  __device__ __forceinline__ void next() {
    i += step;
    walk.advance(step);
    settle();
  }
  __device__ __forceinline__ void settle() {  // a walk past the tiles goes on in the next part
    if (!PARTS || a.splits == 1 || i < (split + 1) * tiles || i >= n) return;
    split = i / tiles;
    walk = TileWalk(i - split * tiles, a.tiles_m, a.tiles_n);
  }
  __device__ __forceinline__ Unit get() const {
    const int2 at = walk.at();
    Unit u;
    u.split = split;
    u.m0 = (at.x * 2 + (int)rank) * kTile;
    u.n0 = at.y * TN;
    u.kb0 = 0;
    u.kb1 = a.kblocks;
    if (!PARTS) return u;
    const int q = a.kblocks / a.splits, more = a.kblocks - q * a.splits;
    u.kb0 = split * q + min(split, more);
    u.kb1 = u.kb0 + q + (split < more ? 1 : 0);
    return u;
  }
};

}  // namespace recattn
