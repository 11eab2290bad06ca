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
constexpr int kFewRows = 64;   // most rows of a call, bf16 and e4m3 (few.cu)
constexpr int kFewRows32 = 8;  // fp32 (few32.cu)
bool few_is_thin(bool e4m3, bool gated, const FewArgs& a);
cudaError_t launch_thin(bool e4m3, bool gated, const FewArgs& a, cudaStream_t st);
cudaError_t launch_few(bool e4m3, bool gated, FewArgs a, int num_sms, cudaStream_t st);
cudaError_t launch_few32(bool gated, const FewArgs& a, cudaStream_t st);

}  // namespace recattn
