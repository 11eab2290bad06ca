// dense.cuh -- the feed-forward block's matrix products: arguments and launchers (internal).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "rec_attn_internal.cuh"

namespace recattn {

// The products of the gated feed-forward block (dense_tc.cu); R rows, W width, H hidden.
enum class DenseOp {
  kGlu,   // h = act(x Wg') * (x Wu')                       [R][H]
  kOut,   // y = h w_out'                                   [R][W]
  kDglu,  // p = [dh u act'(g); dh act(g)], h, dh = dy w_out [R][2H], [R][H]
  kDx,    // dx = p w_in                                    [R][W]
  kDw,    // a' b summed over the rows: dw_in = p' x, dw_out = dy' h
};

struct DenseArgs {
  int M, N;             // rows and columns of the result (kGlu, kDglu: N = H)
  int kblocks;          // blocks of 64 along the summed axis
  int tiles_m, tiles_n, splits;
  int act;              // rec_attn_activation
  int pad;              // columns between the halves of p and behind the rows of p and h (hidden not a
                        // multiple of 16), so that they start on 32-byte boundaries
  int cut;              // kDx, kDw of such a p: hidden
  int wide;             // the outputs' rows start on 32-byte boundaries
  int follows;          // behind a kernel of the same call: launched before that one has ended
  void* out;            // kGlu: h; kOut, kDx: the result; kDglu: p; kDw: the result (of one split)
  void* out2;           // kDglu: h
  float* part;          // kOut, kDx, kDw: [splits][M][N] sums of parts (more than one split)
  int* status;
};

// A row-major [rows][cols] bf16 operand as a TMA map: boxes of 64 columns x 128 rows, or 64 x 64 where the
// summed axis runs over its rows (mn_major).
// ld: from a row to the next, if that is not cols.
bool encode_dense(CUtensorMap* m, const void* base, long long rows, long long cols, bool mn_major, long long ld = 0);
int* dense_status();

// fp32 operands (dense_fp32.cu): a matrix as three bf16 planes whose sum it is, rows `ld` apart.
struct Planes {
  void* p;              // [3][rows][ld] bf16
  long long rows, cols, ld;
  __host__ __device__ size_t plane() const { return (size_t)rows * ld * 2; }
};
struct Dense32Args {
  DenseArgs d;          // out: float rows (kOut, kDx, kDw); part as for kDw, of any of the three
  Planes h, p;          // what kGlu and kDglu write
};
struct SplitList {
  int n;                // matrices, up to four
  const void* x[4];     // fp32 rows
  Planes to[4];
};
cudaError_t launch_split(const SplitList& l, cudaStream_t st);
// (a K-major A: boxes of 128 rows, other operands 64)
// (rows: of a part of the matrix that starts at a.p)
bool encode_planes(CUtensorMap* m, const Planes& a, int box_rows, long long rows = 0);
cudaError_t launch_dense32(DenseOp op, const CUtensorMap (&maps)[4], Dense32Args a, int num_sms, cudaStream_t st);
int dense32_splits(int M, int N, int kblocks, int num_sms);
cudaError_t launch_dense(DenseOp op, const CUtensorMap (&maps)[4], DenseArgs a, int num_sms, cudaStream_t st);
// Parts of the summed axis for a product in tiles of 256 x 256; block_us: what one of its blocks takes.
constexpr double kBlockUs = 0.4, kScaledBlockUs = 0.5;
int dense_splits(int M, int N, int kblocks, double block_us, int num_sms);
// (launched behind the kernel that wrote the parts, before that one has ended)
cudaError_t launch_dense_sum(const float* part, void* out, long long n, int splits, int dtype, cudaStream_t st);

}  // namespace recattn
