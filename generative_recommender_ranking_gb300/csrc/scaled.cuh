// scaled.cuh -- e4m3 matrices with a scale for each block of 128: arguments and launchers (internal).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "rec_attn_internal.cuh"

namespace recattn {

constexpr int kScaleBlock = 128;

struct QuantArgs {
  const void* x;      // [rows][width]
  uint8_t* q;         // [rows][width]
  float* scale;       // [rows or row blocks][blocks]
  long long rows;
  int width, blocks;  // blocks of 128 columns
};
cudaError_t launch_quantize(const QuantArgs& a, int dtype, int block_rows, int num_sms, cudaStream_t st);

struct ScaledArgs {
  int M, N;                // of the result; gated: N = hidden, B has 2 N rows
  int kblocks;             // blocks of 128 along the summed axis
  int tiles_m, tiles_n, splits;
  const float* a_scale;    // [M][kblocks]
  const float* b_scale;    // [blocks of B's rows][kblocks]
  int act;                 // gated
  int wide;                // the outputs' rows start on 32-byte boundaries
  int follows;             // behind a kernel of the same call: launched before that one has ended
  void* out;               // bf16 [M][N]; gated: e4m3
  float* out_scale;        // gated: [M][N / 128]
  float* part;             // [splits][M][N] sums of parts of the summed axis (more than one; not gated)
  int* status;
};
bool encode_scaled(CUtensorMap* m, const void* base, long long rows, long long cols, int box_rows = 128);
// y = a b' of e4m3 operands; gated: act(a g') * (a u') with b = [g; u], in e4m3 with its scales.
cudaError_t launch_scaled(bool gated, const CUtensorMap& ma, const CUtensorMap& mb, ScaledArgs a, int num_sms,
                          cudaStream_t st);

}  // namespace recattn
