// few32.cu -- the feed-forward products for few rows in fp32, on the CUDA cores.
//
// Every weight is used once for each row, so the weights' bytes bound the time: a lane multiplies four
// neighbouring values of a weight row with each token row; a block's eight warps share the summed axis
// and are added up in their order.  Past eight rows the tensor cores take over
// (dense_fp32.cu): on 4096 x 4096 they take 168 us for nine rows and 170 for 64, this way 16 rows a block 111 us for
// nine rows and 32 a block 477 for 24.
// Both products, us on the device with the weights not in the L2: 512 x 1024, one, two, four and eight rows, 5.2, 5.3,
// 8.7 and 10.6; 4096 x 4096 39.0, 39.1, 70.6 and 84.0 (201 MB: 30 at the copy's rate); 4096 x 8192 71, 72, 126 and 179 (403
// MB: 59).  One row reads 5.0 and 4.2 TB/s under ncu; eight 2.6 and 1.6: two blocks an SM (94 to 124 registers a thread)
// have too few loads on their way, and the warps wait for them.
#include "dense_device.cuh"
#include "few.cuh"
#include "launchers.cuh"

namespace recattn {

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;

// A warp has kCols columns of the result (gated: as many pairs) and 1 / kWarps of the summed axis;
// a lane four neighbouring values of it.
constexpr int kCols = 2;
template <bool GATED, int ACT, int ROWS>
__global__ void __launch_bounds__(kThreads, 2) k_few32(const FewArgs a) {
  constexpr int kMats = GATED ? 2 : 1;
  __shared__ float s_sum[kWarps][kMats * kCols * ROWS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.x * kCols;  // (N is a multiple of 4)
  ptx::successor_may_start();
  const float* const w = static_cast<const float*>(a.w);
  const float* const x = static_cast<const float*>(a.x);
  float acc[kMats][kCols][ROWS] = {};
  if (a.follows) ptx::predecessor_done();
#pragma unroll 2
  for (int k = (warp * 32 + lane) * 4; k < a.K; k += kThreads * 4) {
    float4 wv[kMats][kCols];
#pragma unroll
    for (int m = 0; m < kMats; ++m)
#pragma unroll
      for (int c = 0; c < kCols; ++c)
        wv[m][c] = __ldcs(reinterpret_cast<const float4*>(w + ((long long)m * a.N + n0 + c) * a.K + k));
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (r >= a.rows) break;
      const float4 xv = *reinterpret_cast<const float4*>(x + (long long)r * a.K + k);
#pragma unroll
      for (int m = 0; m < kMats; ++m)
#pragma unroll
        for (int c = 0; c < kCols; ++c)
          acc[m][c][r] = fmaf(xv.x, wv[m][c].x,
                              fmaf(xv.y, wv[m][c].y, fmaf(xv.z, wv[m][c].z, fmaf(xv.w, wv[m][c].w, acc[m][c][r]))));
    }
  }
#pragma unroll
  for (int m = 0; m < kMats; ++m)
#pragma unroll
    for (int c = 0; c < kCols; ++c)
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        float v = acc[m][c][r];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) s_sum[warp][(m * kCols + c) * ROWS + r] = v;
      }
  __syncthreads();
  if (threadIdx.x >= kCols * ROWS) return;
  const int c = threadIdx.x % kCols, r = threadIdx.x / kCols;
  if (r >= a.rows) return;
  float v = 0.f, u = 0.f;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) {
    v += s_sum[k][c * ROWS + r];
    if (GATED) u += s_sum[k][(kCols + c) * ROWS + r];
  }
  if (GATED) {
    float slope;
    v = act32<ACT>(v, slope) * u;
  }
  static_cast<float*>(a.out)[(long long)r * a.N + n0 + c] = v;
}

cudaError_t go(void (*fn)(FewArgs), const FewArgs& a, cudaStream_t st) {
  return launch_pairs(1, a.follows != 0, fn, (a.N + kCols - 1) / kCols, kThreads, 0, st, a);
}

template <bool GATED, int ACT>
cudaError_t by_rows(const FewArgs& a, cudaStream_t st) {
  if (a.rows <= 2) return go(k_few32<GATED, ACT, 2>, a, st);
  return go(k_few32<GATED, ACT, kFewRows32>, a, st);
}

}  // namespace

cudaError_t launch_few32(bool gated, const FewArgs& a, cudaStream_t st) {
  if (!gated) return by_rows<false, 0>(a, st);
  return a.act == REC_ATTN_SILU ? by_rows<true, REC_ATTN_SILU>(a, st) : by_rows<true, REC_ATTN_GELU>(a, st);
}

}  // namespace recattn
