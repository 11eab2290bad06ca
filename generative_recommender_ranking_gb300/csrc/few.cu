// few.cu -- the feed-forward products for few rows (serving a handful of tokens).
//
// Every weight is used once for each row, so the weights' bytes bound the time: they go from memory
// straight into registers, 16 bytes a lane.  bf16 and e4m3 take mma.sync m16n8k16 with 16 rows of
// weights as its first operand and 8 token rows as its second (a tile of the tensor cores' tcgen05
// kind would hold 128 rows of which few are tokens, and needs the weights in shared memory first).
// The order of the summed axis is free, so a lane's 16 bytes are the values it owns in both operands
// and nothing is shuffled.  A block has 16 columns of the result (gated: the 16 gate rows and the 16 up
// rows of w); its eight warps take blocks of 128 of the summed axis in turn and are added up in
// shared memory, in their order.  e4m3 values are fp16 values: they are converted, summed block by
// block and added in fp32 times the block's scales.  fp32 multiplies on the CUDA cores.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "dense_epilogue.cuh"
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

// TILES: groups of 8 token rows.
template <bool E4M3, bool GATED, int ACT, int TILES>
__global__ void __launch_bounds__(kThreads, 2) k_few(const FewArgs a) {
  constexpr int kSize = E4M3 ? 1 : 2, kPer = 16 / kSize;        // values in 16 bytes
  constexpr int kLoads = kChunk / (4 * kPer);                   // 16-byte loads of a row's chunk, a lane
  constexpr int kMats = GATED ? 2 : 1;                          // gate and up
  __shared__ float s_sum[kWarps][kMats * TILES * 4][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * kCols;
  const int chunks = (a.K + kChunk - 1) / kChunk;
  ptx::successor_may_start();
  const char* const w = static_cast<const char*>(a.w);
  const char* const x = static_cast<const char*>(a.x);
  float acc[kMats][TILES][4] = {};
  uint4 wv[kMats][2][kLoads];
  const auto load = [&](int c) {
#pragma unroll
    for (int m = 0; m < kMats; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int n = n0 + g + 8 * r;
        const char* row = w + ((long long)m * a.N + n) * a.K * kSize;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int k = c * kChunk + (4 * i + t) * kPer;
          wv[m][r][i] = n < a.N && k < a.K ? __ldcs(reinterpret_cast<const uint4*>(row + (long long)k * kSize)) : make_uint4(0, 0, 0, 0);
        }
      }
  };
  if (warp < chunks) load(warp);
  if (a.follows) ptx::predecessor_done();
  for (int c = warp; c < chunks; c += kWarps) {
    float sum[kMats][TILES][4] = {};
#pragma unroll
    for (int j = 0; j < TILES; ++j) {
      const int row = 8 * j + g;
      uint4 xv[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int k = c * kChunk + (4 * i + t) * kPer;
        xv[i] = row < a.rows && k < a.K ? *reinterpret_cast<const uint4*>(x + ((long long)row * a.K + k) * kSize) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int m = 0; m < kMats; ++m)
#pragma unroll
        for (int i = 0; i < kLoads; ++i) product<E4M3>(E4M3 ? sum[m][j] : acc[m][j], wv[m][0][i], wv[m][1][i], xv[i]);
    }
    if (c + kWarps < chunks) load(c + kWarps);
    if constexpr (E4M3) {
#pragma unroll
      for (int m = 0; m < kMats; ++m) {
        const float sw = __ldg(a.w_scale + (long long)((m * a.N + n0) / kChunk) * chunks + c);
#pragma unroll
        for (int j = 0; j < TILES; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = 8 * j + 2 * t + e;
            const float f = row < a.rows ? sw * a.x_scale[(long long)row * chunks + c] : 0.f;
            acc[m][j][e] = fmaf(sum[m][j][e], f, acc[m][j][e]);
            acc[m][j][2 + e] = fmaf(sum[m][j][2 + e], f, acc[m][j][2 + e]);
          }
      }
    }
  }
#pragma unroll
  for (int m = 0; m < kMats; ++m)
#pragma unroll
    for (int j = 0; j < TILES; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) s_sum[warp][(m * TILES + j) * 4 + e][lane] = acc[m][j][e];
  __syncthreads();
  // result (row, column) = (8 j + 2 t + (e & 1), g + 8 (e >> 1)); 16 neighbouring threads: a row's columns
  for (int i = threadIdx.x; i < 8 * TILES * kCols; i += kThreads) {
    const int col = i % kCols, row = i / kCols;
    const int at = (row >> 3) * 4 + (col >> 3) * 2 + (row & 1), from = (col & 7) * 4 + ((row & 7) >> 1);
    float v = 0.f, u = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      v += s_sum[k][at][from];
      if (GATED) u += s_sum[k][TILES * 4 + at][from];
    }
    if (row >= a.rows || n0 + col >= a.N) continue;
    const long long o = (long long)row * a.N + n0 + col;
    if (GATED) v = act_value<ACT>(v) * u;
    if (GATED && E4M3) static_cast<float*>(a.out)[o] = v;
    else static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(v);
  }
}

// fp32: a warp has kCols32 columns of the result (gated: as many pairs) and 1 / kWarps of the summed axis;
// a lane four neighbouring values of it.
constexpr int kCols32 = 2;
template <bool GATED, int ACT, int ROWS>
__global__ void __launch_bounds__(kThreads, 2) k_few32(const FewArgs a) {
  constexpr int kMats = GATED ? 2 : 1;
  __shared__ float s_sum[kWarps][kMats * kCols32 * ROWS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * kCols32;  // (N is a multiple of 4)
  ptx::successor_may_start();
  const float* const w = static_cast<const float*>(a.w);
  const float* const x = static_cast<const float*>(a.x);
  float acc[kMats][kCols32][ROWS] = {};
  if (a.follows) ptx::predecessor_done();
#pragma unroll 2
  for (int k = (warp * 32 + lane) * 4; k < a.K; k += kThreads * 4) {
    float4 wv[kMats][kCols32];
#pragma unroll
    for (int m = 0; m < kMats; ++m)
#pragma unroll
      for (int c = 0; c < kCols32; ++c)
        wv[m][c] = __ldcs(reinterpret_cast<const float4*>(w + ((long long)m * a.N + n0 + c) * a.K + k));
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (r >= a.rows) break;
      const float4 xv = *reinterpret_cast<const float4*>(x + (long long)r * a.K + k);
#pragma unroll
      for (int m = 0; m < kMats; ++m)
#pragma unroll
        for (int c = 0; c < kCols32; ++c)
          acc[m][c][r] = fmaf(xv.x, wv[m][c].x, fmaf(xv.y, wv[m][c].y, fmaf(xv.z, wv[m][c].z, fmaf(xv.w, wv[m][c].w, acc[m][c][r]))));
    }
  }
#pragma unroll
  for (int m = 0; m < kMats; ++m)
#pragma unroll
    for (int c = 0; c < kCols32; ++c)
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        float v = acc[m][c][r];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) s_sum[warp][(m * kCols32 + c) * ROWS + r] = v;
      }
  __syncthreads();
  if (threadIdx.x >= kCols32 * ROWS) return;
  const int c = threadIdx.x % kCols32, r = threadIdx.x / kCols32;
  if (r >= a.rows) return;
  float v = 0.f, u = 0.f;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) {
    v += s_sum[k][c * ROWS + r];
    if (GATED) u += s_sum[k][(kCols32 + c) * ROWS + r];
  }
  if (GATED) {
    float slope;
    v = act32<ACT>(v, slope) * u;
  }
  static_cast<float*>(a.out)[(long long)r * a.N + n0 + c] = v;
}

cudaError_t go(void (*fn)(FewArgs), const FewArgs& a, int cols, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((a.N + cols - 1) / cols));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = a.follows ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, fn, a);
}

template <bool E4M3, bool GATED, int ACT>
cudaError_t by_rows(const FewArgs& a, cudaStream_t st) {
  if (a.rows <= 8) return go(k_few<E4M3, GATED, ACT, 1>, a, kCols, st);
  if (a.rows <= 16) return go(k_few<E4M3, GATED, ACT, 2>, a, kCols, st);
  if (a.rows <= 24) return go(k_few<E4M3, GATED, ACT, 3>, a, kCols, st);
  return go(k_few<E4M3, GATED, ACT, 4>, a, kCols, st);
}
template <bool E4M3>
cudaError_t by_kind(bool gated, const FewArgs& a, cudaStream_t st) {
  if (!gated) return by_rows<E4M3, false, 0>(a, st);
  return a.act == REC_ATTN_SILU ? by_rows<E4M3, true, REC_ATTN_SILU>(a, st) : by_rows<E4M3, true, REC_ATTN_GELU>(a, st);
}
template <bool GATED, int ACT>
cudaError_t by_rows32(const FewArgs& a, cudaStream_t st) {
  if (a.rows <= 2) return go(k_few32<GATED, ACT, 2>, a, kCols32, st);
  return go(k_few32<GATED, ACT, kFewRows32>, a, kCols32, st);
}

}  // namespace

cudaError_t launch_few(FewType type, bool gated, const FewArgs& a, cudaStream_t st) {
  if (type == FewType::kBf16) return by_kind<false>(gated, a, st);
  if (type == FewType::kE4m3) return by_kind<true>(gated, a, st);
  if (!gated) return by_rows32<false, 0>(a, st);
  return a.act == REC_ATTN_SILU ? by_rows32<true, REC_ATTN_SILU>(a, st) : by_rows32<true, REC_ATTN_GELU>(a, st);
}

}  // namespace recattn
