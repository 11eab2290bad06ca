// few.cuh -- the feed-forward products for few rows: arguments and launchers (internal).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "rec_attn_internal.cuh"

namespace recattn {

// out[r][n] = sum over k of x[r][k] w[n][k]; gated: act(x w[n]) * (x w[N + n]).
struct FewArgs {
  int rows, N, K;
  const void* x;         // [rows][K] bf16, fp32 or e4m3
  const float* x_scale;  // e4m3: [rows][blocks of 128]
  const void* w;         // [N or 2 N][K] in the same type
  const float* w_scale;  // e4m3: [blocks of its rows][blocks]
  int act;
  void* out;             // [rows][N]: bf16; gated e4m3: e4m3; fp32: fp32
  float* out_scale;      // gated e4m3: [rows][N / 128]
  int follows;           // reads the kernel launched just before (its weights' first loads need not wait for it)
  int* status;
  // set by the launcher
  int kblocks, cluster;  // blocks of 128 bytes along the summed axis; CTAs that share them
};
// Most rows of a call, bf16 and e4m3 (few.cu): all that an MMA's N side is laid out for.  33 and 64 rows here, and by the
// kernels of many rows (us on the device, weights not in the L2): bf16 block 512 x 1024 9.9 and 11.9, 14.7 and 15.1; 1408
// x 4104 18.4 and 22.1, 22.5 and 24.1; 4096 x 8192 44.7 and 46.8, 49.6 and 51.4; 4096 x 256 14.3 and 16.2, 27.0 and 27.2.
// e4m3 product 512 x 512 4.6 and 4.9, 5.7 and 6.2; 4096 x 4096 9.8 and 11.2, 13.0 and 14.2; 8192 x 1024 7.3 and 8.0, 8.5
// and 8.9; its block 4096 x 8192 31.3 and 36.2, 38.5 and 40.4.
constexpr int kFewRows = 64;
constexpr int kFewRows32 = 8;  // fp32 (few32.cu)
bool few_is_thin(bool e4m3, bool gated, const FewArgs& a);
cudaError_t launch_thin(bool e4m3, bool gated, const FewArgs& a, cudaStream_t st);
cudaError_t launch_few(bool e4m3, bool gated, FewArgs a, int num_sms, cudaStream_t st);
cudaError_t launch_few32(bool gated, const FewArgs& a, cudaStream_t st);

}  // namespace recattn
