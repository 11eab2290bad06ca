// few.cuh -- the feed-forward products for few rows: arguments and launchers (internal).
#pragma once

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
  void* out;             // [rows][N]: bf16; gated e4m3: fp32; fp32: fp32
  int follows;           // reads the kernel launched just before (its weights' first loads need not wait for it)
};
constexpr int kFewRows = 32;    // most rows of a call, bf16 and e4m3
constexpr int kFewRows32 = 8;   // fp32
enum class FewType { kBf16, kE4m3, kFp32 };
cudaError_t launch_few(FewType type, bool gated, const FewArgs& a, cudaStream_t st);

}  // namespace recattn
