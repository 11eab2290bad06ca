// simt_tile.cuh -- 64 x 64 tiles of fp32 products on the CUDA cores, for the fp32 attention
// kernels (attn_simt.cu, attn_bwd.cu).  256 threads; thread (ty, tx) of 16 x 16 holds rows 4 ty ..
// and columns 4 tx .. of a score tile, or D / 16 columns of an accumulator, in row pairs (fma.rn.f32x2).
//
// Operands whose rows run along the product's K dimension are stored transposed, element (r, d) at
// d * 64 + 4 * ((r / 4) ^ (d / 4 % 16)) + r % 4: a thread's four rows at one d are 16 bytes, and
// neither the transposing stores (two lanes a bank) nor the loads (none) wait for one another.
#pragma once

#include "attn_common.cuh"

namespace recattn {
namespace simt {

constexpr int kB = 64;         // rows and columns of a score tile
constexpr int kThreads = 256;
constexpr int kPerTile = kTile / kB;

using f2 = unsigned long long;
__device__ __forceinline__ f2 pair(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 both(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Four consecutive rows (4 * block ..) of a transposed operand at d.
__device__ __forceinline__ int at(int block, int d) { return d * kB + ((block ^ ((d >> 2) & 15)) << 2); }

// The 64 rows at src (`stride` floats apart; zeros from row `valid` on): into registers, so that a
// step's loads run under the last one's products, and from there, times scale, to shared memory:
// transposed into T and / or as they are into R (either may be null).
template <int D>
struct Rows {
  static constexpr int kChunks = kB * (D / 4) / kThreads;
  float4 x[kChunks];
  __device__ __forceinline__ void fetch(const float* src, long long stride, int valid) {
#pragma unroll
    for (int n = 0; n < kChunks; ++n) {
      const int i = (int)threadIdx.x + n * kThreads, r = i / (D / 4), e = i % (D / 4) * 4;
      x[n] = r < valid ? *reinterpret_cast<const float4*>(src + r * stride + e) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  __device__ __forceinline__ void put(float scale, float* T, float* R) const {
#pragma unroll
    for (int n = 0; n < kChunks; ++n) {
      const int i = (int)threadIdx.x + n * kThreads, r = i / (D / 4), e = i % (D / 4) * 4;
      const float4 y = make_float4(x[n].x * scale, x[n].y * scale, x[n].z * scale, x[n].w * scale);
      if (T) {
        float* t = T + at(r >> 2, e) + (r & 3);
        t[0] = y.x; t[kB] = y.y; t[2 * kB] = y.z; t[3 * kB] = y.w;
      }
      if (R) *reinterpret_cast<float4*>(R + r * D + e) = y;
    }
  }
};
template <int D>
__device__ __forceinline__ void load_tile(const float* src, long long stride, int valid, float scale, float* T, float* R) {
  Rows<D> x;
  x.fetch(src, stride, valid);
  x.put(scale, T, R);
}

// s[p][j] += sum_d A(rows 4 ty + 2 p, + 1; d) B(row 4 tx + j; d), both transposed.
template <int D>
__device__ __forceinline__ void scores(const float* A, const float* B, int ty, int tx, f2 (&s)[2][4]) {
#pragma unroll 8
  for (int d = 0; d < D; ++d) {
    const float4 a = *reinterpret_cast<const float4*>(A + at(ty, d)), b = *reinterpret_cast<const float4*>(B + at(tx, d));
    const f2 a0 = pair(a.x, a.y), a1 = pair(a.z, a.w);
    const f2 bb[4] = {pair(b.x, b.x), pair(b.y, b.y), pair(b.z, b.z), pair(b.w, b.w)};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s[0][j] = fma2(a0, bb[j], s[0][j]);
      s[1][j] = fma2(a1, bb[j], s[1][j]);
    }
  }
}

// The thread's 4 x 4 values, transposed for accumulate(): P(row, column) at (4 ty + row, 4 tx + column).
__device__ __forceinline__ void store_scores(float* P, int ty, int tx, const float (&x)[4][4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<float4*>(P + at(ty, 4 * tx + j)) = make_float4(x[0][j], x[1][j], x[2][j], x[3][j]);
}

// o[p][j] += sum_c P(rows 4 ty + 2 p, + 1; c) V(row c, column N tx + j), V as it is, N = D / 16.
template <int D>
__device__ __forceinline__ void accumulate(const float* P, const float* V, int ty, int tx, f2 (&o)[2][D / 16]) {
  constexpr int N = D / 16;
#pragma unroll 8
  for (int c = 0; c < kB; ++c) {
    const float4 p = *reinterpret_cast<const float4*>(P + at(ty, c));
    const f2 p0 = pair(p.x, p.y), p1 = pair(p.z, p.w);
    float v[N];
    if constexpr (N == 4) {
      const float4 x = *reinterpret_cast<const float4*>(V + c * D + N * tx);
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else {
      const float2 x = *reinterpret_cast<const float2*>(V + c * D + N * tx);
      v[0] = x.x; v[1] = x.y;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const f2 vv = pair(v[j], v[j]);
      o[0][j] = fma2(p0, vv, o[0][j]);
      o[1][j] = fma2(p1, vv, o[1][j]);
    }
  }
}

// The same without the pairs whose weight is -0, the mark of a pair that the mask hides: for rows of V
// with values that are not finite.
constexpr float kHidden = -0.f;
template <int D>
__device__ __forceinline__ void accumulate_seen(const float* P, const float* V, int ty, int tx, f2 (&o)[2][D / 16]) {
  constexpr int N = D / 16;
#pragma unroll 1
  for (int c = 0; c < kB; ++c) {
    const float4 p = *reinterpret_cast<const float4*>(P + at(ty, c));
    auto add = [](float w, float v, float y) {
      return __float_as_uint(w) == __float_as_uint(kHidden) ? y : fmaf(w, v, y);
    };
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float v = V[c * D + N * tx + j];
      const float2 a = both(o[0][j]), b = both(o[1][j]);
      o[0][j] = pair(add(p.x, v, a.x), add(p.y, v, a.y));
      o[1][j] = pair(add(p.z, v, b.x), add(p.w, v, b.y));
    }
  }
}

// A row over the 16 threads that share it.
__device__ __forceinline__ float row_max(float x) {
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// What the mask needs of 64 tokens: position, time, type (-1 past the request's end) and, of
// queries, the delay bound.
struct Tokens {
  long long t[kB], thr[kB];
  int ty[kB], thr_ok[kB];
  int pos0;
  __device__ __forceinline__ void load(const long long* t_, const int8_t* ty_, long long tok0, int pos, int len, long long delay) {
    for (int i = threadIdx.x; i < kB; i += kThreads) {
      const bool in = pos + i < len;
      t[i] = in ? t_[tok0 + i] : 0;
      ty[i] = in ? (int)ty_[tok0 + i] : -1;
      bool ok;
      delay_bound(t[i], delay, ok, thr[i]);
      thr_ok[i] = ok;
    }
    if (threadIdx.x == 0) pos0 = pos;
  }
};
__device__ __forceinline__ bool visible(const MaskP& m, const Tokens& q, int i, const Tokens& k, int j) {
  return vis_pred(m, q.pos0 + i, q.t[i], q.ty[i], q.thr_ok[i] != 0, q.thr[i], k.pos0 + j, k.t[j], k.ty[j]);
}


// The visibility bits of a query's keys 4 c .. 4 c + 3 within a key tile, from the mask table's rows of
// the pair (`row`: the query's row of its tile).
__device__ __forceinline__ uint32_t table_bits(const uint32_t* mtab, int slot, int row, int c) {
  return mtab[((long long)slot * kTile + row) * 4 + (c >> 3)] >> (4 * (c & 7)) & 15u;
}

}  // namespace simt
}  // namespace recattn
