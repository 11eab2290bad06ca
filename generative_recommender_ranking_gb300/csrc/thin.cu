// thin.cu -- the feed-forward products for up to eight rows.
//
// The weights go from memory straight into registers, 16 bytes a lane, and mma.sync m16n8k16 takes 16
// rows of them as its first operand and the 8 token rows as its second: no shared memory, tensor map,
// TMEM or cluster stands between the launch and the first load, which few.cu's products pay for with
// 2 to 4 us.  The order of the summed axis is free, so a lane's 16 bytes are the values it owns in both
// operands and nothing is shuffled.  A block has 16 columns of the result (gated: the 16 gate rows and
// the 16 up rows of w); its eight warps take blocks of 128 of the summed axis in turn and are added up
// in shared memory, in their order.  e4m3 values are fp16 values: they are converted, summed block by
// block and added in fp32 times the block's scales.
// One row of 512 x 1024, both products: 7 us on the device (latency; a call from Python takes 16); of
// 4096 x 8192: 42 us (4.8 TB/s).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "dense_device.cuh"
#include "few.cuh"
#include "launchers.cuh"

namespace recattn {

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kCols = 16;    // columns of the result a block
constexpr int kChunk = 128;  // of the summed axis, a warp's turn

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four e4m3 values as two pairs of fp16.
__device__ __forceinline__ uint2 halves(uint32_t w) {
  const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
  const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
  return make_uint2((uint32_t)lo.x | (uint32_t)lo.y << 16, (uint32_t)hi.x | (uint32_t)hi.y << 16);
}

// 16 bytes each of rows g and g + 8 of w, and of a row of x, into d.
template <bool E4M3>
__device__ __forceinline__ void product(float (&d)[4], const uint4 a, const uint4 b, const uint4 x) {
  if constexpr (E4M3) {
    const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w}, wx[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint2 ha = halves(wa[i]), hb = halves(wb[i]), hx = halves(wx[i]);
      mma_f16(d, ha.x, hb.x, ha.y, hb.y, hx.x, hx.y);
    }
  } else {
    mma_bf16(d, a.x, b.x, a.y, b.y, x.x, x.y);
    mma_bf16(d, a.z, b.z, a.w, b.w, x.z, x.w);
  }
}

template <bool E4M3, bool GATED, int ACT>
__global__ void __launch_bounds__(kThreads, 2) k_thin(const FewArgs a) {
  constexpr int kSize = E4M3 ? 1 : 2, kPer = 16 / kSize;        // values in 16 bytes
  constexpr int kLoads = kChunk / (4 * kPer);                   // 16-byte loads of a row's chunk, a lane
  constexpr int kMats = GATED ? 2 : 1;                          // gate and up
  constexpr int kAhead = GATED ? 1 : E4M3 ? 4 : 2;              // blocks whose weights a warp has on their way
  __shared__ float s_sum[kWarps][kMats * 4][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * kCols;
  const int chunks = (a.K + kChunk - 1) / kChunk;
  ptx::successor_may_start();
  const char* const w = static_cast<const char*>(a.w);
  const char* const x = static_cast<const char*>(a.x) + (long long)g * a.K * kSize;
  float acc[kMats][4] = {};
  uint4 wv[kAhead][kMats][2][kLoads];
  const auto load = [&](uint4 (&to)[kMats][2][kLoads], int c) {
#pragma unroll
    for (int m = 0; m < kMats; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int n = n0 + g + 8 * r;
        const char* row = w + ((long long)m * a.N + n) * a.K * kSize;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int k = c * kChunk + (4 * i + t) * kPer;
          to[m][r][i] = n < a.N && k < a.K ? __ldcs(reinterpret_cast<const uint4*>(row + (long long)k * kSize))
                                           : make_uint4(0, 0, 0, 0);
        }
      }
  };
#pragma unroll
  for (int h = 0; h < kAhead; ++h)
    if (warp + kWarps * h < chunks) load(wv[h], warp + kWarps * h);
  if (a.follows) ptx::predecessor_done();
  for (int c0 = warp; c0 < chunks; c0 += kWarps * kAhead) {
    uint4 xv[kAhead][kLoads];
#pragma unroll
    for (int h = 0; h < kAhead; ++h)
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int k = (c0 + kWarps * h) * kChunk + (4 * i + t) * kPer;
        xv[h][i] = g < a.rows && k < a.K ? *reinterpret_cast<const uint4*>(x + (long long)k * kSize) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
    for (int h = 0; h < kAhead; ++h) {
      const int c = c0 + kWarps * h;
      if (c >= chunks) break;
      float sum[kMats][4] = {};
#pragma unroll
      for (int m = 0; m < kMats; ++m)
#pragma unroll
        for (int i = 0; i < kLoads; ++i) product<E4M3>(E4M3 ? sum[m] : acc[m], wv[h][m][0][i], wv[h][m][1][i], xv[h][i]);
      if (c + kWarps * kAhead < chunks) load(wv[h], c + kWarps * kAhead);
      if constexpr (E4M3) {
#pragma unroll
        for (int m = 0; m < kMats; ++m) {
          const float sw = __ldg(a.w_scale + (long long)((m * a.N + n0) / kChunk) * chunks + c);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = 2 * t + e;
            const float f = row < a.rows ? sw * a.x_scale[(long long)row * chunks + c] : 0.f;
            acc[m][e] = fmaf(sum[m][e], f, acc[m][e]);
            acc[m][2 + e] = fmaf(sum[m][2 + e], f, acc[m][2 + e]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < kMats; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) s_sum[warp][m * 4 + e][lane] = acc[m][e];
  __syncthreads();
  // result (row, column) = (2 t + (e & 1), g + 8 (e >> 1)); 16 neighbouring threads: a row's columns
  if (threadIdx.x >= 8 * kCols) return;
  const int col = threadIdx.x % kCols, row = threadIdx.x / kCols;
  const int at = (col >> 3) * 2 + (row & 1), from = (col & 7) * 4 + (row >> 1);
  float v = 0.f, u = 0.f;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) {
    v += s_sum[k][at][from];
    if (GATED) u += s_sum[k][4 + at][from];
  }
  if (row >= a.rows || n0 + col >= a.N) return;
  if (GATED) v = values_of(act_value<ACT>(pair_of(v, v))).x * u;
  static_cast<__nv_bfloat16*>(a.out)[(long long)row * a.N + n0 + col] = __float2bfloat16_rn(v);
}

cudaError_t go(void (*fn)(FewArgs), const FewArgs& a, cudaStream_t st) {
  return launch_pairs(1, a.follows != 0, fn, (a.N + kCols - 1) / kCols, kThreads, 0, st, a);
}

}  // namespace

// Up to eight rows; of e4m3 up to 16 MB of weights.  Against few.cu's (one row, weights not in the L2):
// bf16 512 x 1024, both products, 9.2 and 13.3 us; 4096 x 8192 42 and 52.  e4m3, one product: 0.5 MB
// 6.0 and 8.2; 16 MB 12.3 both; 32 MB 16.4 and 14.3 (the conversions to fp16 tell).
bool few_is_thin(bool e4m3, bool gated, const FewArgs& a) {
  return a.rows <= 8 && (!e4m3 || (!gated && (long long)a.N * a.K <= (16LL << 20)));
}

cudaError_t launch_thin(bool e4m3, bool gated, const FewArgs& a, cudaStream_t st) {
  if (e4m3) return go(k_thin<true, false, 0>, a, st);
  if (!gated) return go(k_thin<false, false, 0>, a, st);
  return go(a.act == REC_ATTN_SILU ? k_thin<false, true, REC_ATTN_SILU> : k_thin<false, true, REC_ATTN_GELU>, a, st);
}

}  // namespace recattn
