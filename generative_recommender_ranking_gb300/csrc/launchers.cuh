// launchers.cuh -- host entry points of the kernels (internal to the library).
#pragma once

#include <atomic>

#include <cuda.h>

#include "attn_common.cuh"

namespace recattn {

// While it lives, the thread may make calls that a stream capture forbids it otherwise: for what is
// set up once and belongs to no stream (a memory pool, a kernel's attributes), should the first
// call that needs it be captured.
struct OutsideCapture {
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  OutsideCapture() { cudaThreadExchangeStreamCaptureMode(&mode); }
  ~OutsideCapture() { cudaThreadExchangeStreamCaptureMode(&mode); }
  OutsideCapture(const OutsideCapture&) = delete;
  OutsideCapture& operator=(const OutsideCapture&) = delete;
};

// Raises a kernel's limit of dynamic shared memory, once per kernel and device (`done`: a static
// of the caller, one bit per device): the call costs a launch's worth of host time.
inline cudaError_t allow_smem(std::atomic<unsigned long long>& done, const void* fn, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  const OutsideCapture now;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Launches blocks in clusters of `cluster` (1: none); early: before the stream's last kernel has ended
// (the kernel itself waits for it, ptx::predecessor_done).
template <typename... P, typename... A>
cudaError_t launch_pairs(int cluster, bool early, void (*fn)(P...), int blocks, int threads, int smem, cudaStream_t st,
                         A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  if (cluster > 1) {
    at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    at[cfg.numAttrs].val.clusterDim.x = (unsigned)cluster;
    at[cfg.numAttrs].val.clusterDim.y = at[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (early) {
    at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  cfg.attrs = at;
  return cudaLaunchKernelEx(&cfg, fn, static_cast<P>(args)...);
}

// Whether a kernel's threads are launched with so many registers (asked once, kept in `known`): one that splits more
// among its warpgroups than it was launched with would wait for them forever.  The kernels ask for theirs by
// __maxnreg__, so this says no only if a compiler gives them fewer.
inline bool launched_with(std::atomic<int>& known, const void* fn, int regs) {
  int n = known.load(std::memory_order_relaxed);
  if (n == 0) {
    cudaFuncAttributes at{};
    const OutsideCapture now;
    if (cudaFuncGetAttributes(&at, fn) != cudaSuccess) return false;
    known.store(n = at.numRegs, std::memory_order_relaxed);
  }
  return n == regs;
}

// prologue_ok (may be null) is recorded on st once the RoPE prologue, on another stream,
// may start: before the planner when it is one kernel, after its first kernel when a
// long request's tiles are split over several blocks (so the second kernel's blocks,
// launched first, are not queued behind the prologue's).  kv_bytes: size of all keys and values.
cudaError_t launch_plan(const MaskP& mp, int heads, const PlanDev& pd, const long long* offsets_dev,
                        const long long* t, const int8_t* ty, int batch, long long n_tiles, size_t kv_bytes,
                        cudaEvent_t prologue_ok, cudaStream_t st);
cudaError_t launch_build_masks(const MaskP& mp, const PlanDev& pd, int num_sms, cudaStream_t st);
cudaError_t launch_count_pairs(const MaskP& mp, const PlanDev& pd, const long long* t,
                               const int8_t* ty, long long n_tiles, cudaStream_t st);
// pairs: device int[n_pairs][3] (request, query tile, key tile), validated by the caller;
// bits: [n_pairs][128][4]; lcls: the pair's class in its query tile's list (0xff: not
// listed, never loaded); lslot: its mask-table slot (-1: none).
cudaError_t launch_export_masks(const MaskP& mp, const PlanDev& pd, const long long* t, const int8_t* ty,
                                const int* pairs, int n_pairs, int mode, uint32_t* bits, uint8_t* lcls, int* lslot,
                                cudaStream_t st);
cudaError_t launch_rope(const RopeArgs& a, int dtype, long long n_tiles, cudaStream_t st);
cudaError_t launch_rope_fused(const RopeArgs& a, const FusedArgs& f, int dtype, long long n_tiles,
                              cudaStream_t st);
// Serving with a cached history: regions of rows into / out of the combined layout
// (n_chunks 128-row chunks listed in a.chunk_req / a.chunk_row0).
cudaError_t launch_rope_slots(const SlotArgs& a, int dtype, long long n_chunks, cudaStream_t st);
cudaError_t launch_slots_gather(const SlotArgs& a, int dtype, long long n_chunks, cudaStream_t st);
cudaError_t launch_attn_simt(const AttnArgs& a, int head_dim, cudaStream_t st);
cudaError_t launch_bwd_delta(const BwdArgs& a, int head_dim, cudaStream_t st);
cudaError_t launch_attn_bwd_simt(const BwdArgs& a, int head_dim, long long n_tiles, cudaStream_t st);
// Parts of a group's query heads that dK/dV items take apart (a divisor of the group): the
// fewest that give `least` items.  Tensor cores: two an SM (161 tiles of 2 key/value heads, 152 SMs: parts of
// their own for a better balance cost more in their sums, 516 against 494 us a training step);
// fp32, whose items are slow and of unequal length: six.
int bwd_kv_parts(long long n_tiles, int kv_heads, int group, long long least);
cudaError_t launch_bwd_schedule(const BwdSchedArgs& s, int num_sms, cudaStream_t st);
cudaError_t launch_attn_bwd_tc(const BwdArgs& a, const CUtensorMap (&maps)[4], int head_dim, int num_sms,
                               cudaStream_t st);
cudaError_t launch_compress(const CompressArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_bwd_gate(const GateArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_bwd_norm_gate(const NormGateArgs& a, int dtype, cudaStream_t st);
// n_fix 32-row block boundaries (per request ceil(len / 32), from CmpReq::fix_start);
// req_len: device int [B] request lengths.
cudaError_t launch_cmp_fixup(const CmpArgs& c, int batch, const int* req_len, long long n_fix, int heads,
                             int head_dim, cudaStream_t st);
// Candidates against a cached history with shared heads (score.cu).
constexpr int kNeedBlock = 64;     // keys per entry of block_need
constexpr int kScoreMaxReq = 250;  // requests per launch (their tables are kernel parameters: 2 KB)
struct ScoreArgs {
  // the cache
  const long long* hist_off;    // [B + 1] rows of each request in K', V (whole 128-row tiles)
  const int* hist_len;          // [B] its keys; the rows behind them are zero
  const long long* need;        // [Th]: least time of a candidate that sees the key
  const long long* block_need;  // per 64-key block of a request: the largest of its keys' need
  const int* block_off;         // [B + 1] first block of each request
  const long long* t_ref;       // [B] the rotation's reference time
  int* status;
  // the call
  const long long* tc;          // [Nc]
  const void *q, *k, *v;        // [Nc][heads or kv_heads][d], not rotated
  void* out;
  float* lse;
  float2* part_ml;              // [items][rows per item]: maximum and sum; null: one part per row
  float* part_o;                // [items][rows per item][d]: unnormalised outputs
  int heads, kv_heads;
  int rotate;
  int tile_keys, chunk_tiles;   // keys per tile, tiles per item
  int cluster;                  // > 0: an item's tiles are shared by a cluster of so many blocks
  float scale_log2;             // softmax scale * log2(e)
  float omega[kMaxPairs];
  int req0, n_req;              // the launch's requests
  int cand_start[kScoreMaxReq + 1];  // first candidate of each
  int item_start[kScoreMaxReq + 1];  // first block of each: [row group][kv head][run of tiles]
};
struct NeedArgs {
  const long long* hist_off;
  const int *hist_len, *block_off;
  const long long* t;
  const int8_t* ty;
  int batch, use_delay;
  long long delay;
  long long *need, *block_need, *t_ref;
  uint8_t* block_ordered;       // 1: the block's keys stand in order of visibility
  int* status;
};
int score_tile_keys(int head_dim);
int score_rows_per_item(int head_dim, int max_rows);
cudaError_t launch_score_need(const NeedArgs& a, int blocks, cudaStream_t st);
// The many-row path: k_score_pack, k_attn_tc's CAND instantiation (launch_attn_tc with
// a.cand), and with more than one run per row k_score_combine.
cudaError_t launch_score_pack(const ScoreArgs& a, int head_dim, int items, CandItem* desc, void* qp, int* counters,
                              cudaStream_t st);
cudaError_t launch_score_combine(const ScoreArgs& a, int head_dim, int rows_per_item, cudaStream_t st);
cudaError_t launch_score_rows(const CUtensorMap& k, const CUtensorMap& v, const ScoreArgs& a, int head_dim,
                              int rows_per_item, int items, cudaStream_t st);

// Layer norm (layernorm.cu).
struct NormArgs {
  long long rows;
  int width;            // values per row; width * element size a multiple of 16
  float eps;
  const int8_t* ty;     // [rows] token types (the row's gain and bias), or null: one for all
  const void* x;        // [rows][width]
  const float* w;       // [4 or 1][width]
  const float* b;       // [4 or 1][width] or null
  void* y;              // forward output
  const void* dy;       // backward: upstream gradient
  void* dx;
  float* dw;            // [4 or 1][width] or null
  float* db;
  // set by the launchers
  int tpr;              // threads per row
  long long rows_per_block;
  unsigned* seen;       // [blocks]: types whose sums the block wrote
  float* part;          // [blocks][types][2][width]
  float* flush;         // [blocks][row groups][4][2][width] (by type only)
};
// The backward's grid and workspace for a shape.
struct NormBwdPlan {
  int blocks, smem;
  long long rows_per_block;
  size_t off_part, off_flush, bytes;
};
cudaError_t launch_layernorm_fwd(NormArgs a, int dtype, int num_sms, cudaStream_t st);
NormBwdPlan layernorm_bwd_plan(long long rows, int width, int dtype, bool by_type, int num_sms);
cudaError_t launch_layernorm_bwd(NormArgs a, const NormBwdPlan& p, void* ws, int dtype, cudaStream_t st);
cudaError_t launch_wait_timeout(int* status, unsigned long long limit_ns, cudaStream_t st);
cudaError_t launch_attn_tc(const AttnArgs& a, const CUtensorMap& q, const CUtensorMap& k,
                           const CUtensorMap& v, int head_dim, int grid, cudaStream_t st);

// Host helpers shared by the entry points (api.cu): the parameter checks of
// rec_attn_params, and a 2-D TMA map over a [T][cols] bf16 tensor (box 64 columns x
// `rows` rows, 128-byte swizzle).
rec_attn_status check_params(const rec_attn_params* p);
rec_attn_status from_cuda(cudaError_t e);
cudaError_t pool_for(int device, cudaMemPool_t* out);  // the library's memory pool of a device
bool overlaps(const void* a, size_t na, const void* b, size_t nb);
cudaError_t device_and_sms(int* dev, int* sms);  // the current device
bool encode_map(CUtensorMap* m, const void* base, long long T, long long cols, int rows = kTile,
                long long ld = 0);
// 1 when the plan's items run over many key tiles (AttnArgs::long_items).
int long_items(const rec_attn_params& p, int batch, long long n_tiles);

}  // namespace recattn
