// few.cu -- the feed-forward products for few rows (serving a handful of tokens), bf16 and e4m3.
//
// Every weight is used once for each row, so the weights' bytes bound the time.  The operands change
// places: 128 rows of weights are the MMA's M side, the token rows (up to 64, padded to 16, 32 or 64) its
// N side, and two CTAs an SM keep 108 KB each full of weights on their way (TMA).  A
// tile is 128 columns of the result (gated: their gate rows and their up rows, two accumulators); where
// tiles are fewer than SMs, a cluster of 2, 4 or 8 CTAs shares a tile's summed axis, and each then adds
// up its share of the token rows over the CTAs' sums through distributed shared memory, in their order.
// e4m3: each block of 128 is summed by itself and taken into registers times its scales, as in scaled.cu.
// The first weights of a product that follows another are fetched before that one has ended.
// 24 rows of 4096 x 8192, both products: 41 us (4.9 TB/s), e4m3 30.5 with the quantizer (3.3 TB/s): about 6 us of
// each kernel are its launch, its first copies' latency and the join; 67 and 134 MB take 15 and 26 us alone.  One
// CTA an SM with 180 KB: 43; mma.sync from registers (thin.cu) with 24 rows: 61 and 59.  (The gated e4m3 form for more than
// 32 rows holds 128 sums a thread and spills 28 bytes at 168 registers.)
#include <cuda_bf16.h>

#include <atomic>

#include "dense.cuh"
#include "dense_device.cuh"
#include "few.cuh"
#include "launchers.cuh"
#include "ptx_sm103.cuh"
#include "quantize.cuh"
#include "scaled.cuh"
#include "wait.cuh"

namespace recattn {

namespace {

constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s
constexpr int kThreads = 192, kSumWarps = 4;
constexpr int kMat = 128 * 128;              // 128 rows of 128 bytes
constexpr uint32_t kTmem = 256;

enum { kFull = 0, kEmpty = 12, kAccFull = 24, kAccEmpty = 26, kDone = 28, kBars = 29 };

// TOKENS: rows of x that an MMA takes.
template <bool GATED, int TOKENS>
struct Cfg {
  static constexpr int kMats = GATED ? 2 : 1;
  static constexpr int kStage = kMats * kMat + TOKENS * 128;
  static constexpr int kStages = 108 * 1024 / kStage;  // two CTAs an SM
  static constexpr int kDynamic = kStages * kStage + 1024;
  static_assert(kStages * kStage >= kMats * TOKENS * 128 * 4, "the CTA's sums fit the ring");
  static_assert(3 * kDynamic > 228 * 1024, "no more CTAs an SM than TMEM has columns for");
};

// Four floats of another CTA's shared memory, at this one's place `p`.
__device__ __forceinline__ float4 remote_float4(const void* p, int rank) {
  uint32_t at;
  float4 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
__device__ __forceinline__ float4 sum_of(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// One thread: block n of this CTA's on its way into its stage.
template <bool E4M3, bool GATED, int TOKENS>
struct Loader {
  using C = Cfg<GATED, TOKENS>;
  static constexpr int kX = E4M3 ? 128 : 64;  // values in 128 bytes
  const FewArgs& a;
  const CUtensorMap *mw, *mx;
  uint8_t* sm;
  uint64_t* bars;
  int n0, kb0;
  __device__ __forceinline__ void weights(int n) const {
    const int st = n % C::kStages;
    uint8_t* s = sm + st * C::kStage;
    ptx::mbar_arrive_expect_tx(bars + kFull + st, C::kStage);
    ptx::tma_load_2d(s, mw, (kb0 + n) * kX, n0, bars + kFull + st);
    if (GATED) ptx::tma_load_2d(s + kMat, mw, (kb0 + n) * kX, a.N + n0, bars + kFull + st);
  }
  __device__ __forceinline__ void tokens(int n) const {
    const int st = n % C::kStages;
    ptx::tma_load_2d(sm + st * C::kStage + C::kMats * kMat, mx, (kb0 + n) * kX, 0, bars + kFull + st);
  }
};

// The loading warp; the first stages' weights are on their way already.
template <bool E4M3, bool GATED, int TOKENS>
__device__ void load_rest(const FewArgs& a, const Loader<E4M3, GATED, TOKENS>& in, uint64_t* bars,
                          volatile int* abort_flag, int blocks, int lane) {
  using C = Cfg<GATED, TOKENS>;
  const int ahead = min(blocks, C::kStages);
  if (a.follows) ptx::predecessor_done();
  if (lane == 0)
    for (int j = 0; j < ahead; ++j) in.tokens(j);
  __syncwarp();
  int n = ahead;
  for (; n < blocks; ++n) {
    if (!bounded_wait_warp(bars + kEmpty + n % C::kStages, (n / C::kStages + 1) & 1, abort_flag, a.status, kWaitNs)) break;
    if (lane == 0) {
      in.weights(n);
      in.tokens(n);
    }
    __syncwarp();
  }
  // after an abort, copies may still be in flight
  if (lane == 0)
    for (int j = max(0, n - C::kStages); j < n; ++j)
      bounded_drain(bars + kFull + j % C::kStages, (j / C::kStages) & 1, kWaitNs / 4);
  __syncwarp();
}

// bf16: one sum over all blocks; e4m3: a sum for each block, in two buffers.
template <bool E4M3, bool GATED, int TOKENS>
__device__ void issue(const FewArgs& a, uint8_t* sm, uint64_t* bars, uint32_t tmem, volatile int* abort_flag, int blocks) {
  using C = Cfg<GATED, TOKENS>;
  const uint32_t idesc = E4M3 ? ptx::idesc_e4m3_f32(128, TOKENS) : ptx::idesc_bf16_f32(128, TOKENS, false, false);
  const uint32_t s0 = ptx::smem_u32(sm);
  const bool el = ptx::elect_one();
  for (int n = 0; n < blocks; ++n) {
    const int st = n % C::kStages;
    const uint32_t buf = E4M3 ? n & 1 : 0;
    if (E4M3 && !bounded_wait_warp(bars + kAccEmpty + buf, ((n >> 1) & 1) ^ 1, abort_flag, a.status, kWaitNs)) break;
    if (!bounded_wait_warp(bars + kFull + st, (n / C::kStages) & 1, abort_flag, a.status, kWaitNs)) break;
    ptx::tc_fence_after();
    if (el) {
      const uint32_t s = s0 + st * C::kStage;
      const uint64_t dx = ptx::smem_desc_sw128(s + C::kMats * kMat, 16, 1024);
#pragma unroll
      for (int m = 0; m < C::kMats; ++m) {
        const uint64_t dw = ptx::smem_desc_sw128(s + m * kMat, 16, 1024);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          (E4M3 ? ptx::umma_f8 : ptx::umma_f16)(tmem + (buf * C::kMats + m) * TOKENS, ptx::smem_desc_at(dw, 32 * k),
                                                ptx::smem_desc_at(dx, 32 * k), idesc, k > 0 || (!E4M3 && n > 0));
      }
      ptx::umma_commit(bars + kEmpty + st);
      if (E4M3 || n == blocks - 1) ptx::umma_commit(bars + kAccFull + buf);
    }
    __syncwarp();
  }
  if (el) {
    ptx::umma_commit(bars + kDone);
    bounded_drain(bars + kDone, 0, kWaitNs / 4);
  }
  __syncwarp();
}

// Four warps: a thread has one weight row; its sums go to s_sum[matrix][token][row].
template <bool E4M3, bool GATED, int TOKENS>
__device__ void collect(const FewArgs& a, float* s_sum, uint64_t* bars, uint32_t tmem, volatile int* abort_flag, int n0,
                        int kb0, int kb1, int warp, int lane) {
  using C = Cfg<GATED, TOKENS>;
  const int quad = warp & 3;
  const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
  float* const mine = s_sum + quad * 32 + lane;
  if constexpr (E4M3) {
    if (a.follows) ptx::predecessor_done();
    float acc[C::kMats][TOKENS];
#pragma unroll
    for (int m = 0; m < C::kMats; ++m)
#pragma unroll
      for (int j = 0; j < TOKENS; ++j) acc[m][j] = 0.f;
    for (int kb = kb0; kb < kb1; ++kb) {
      const int n = kb - kb0;
      const uint32_t buf = n & 1;
      // lane l: the scales of tokens l and 32 + l
      float sx[(TOKENS + 31) / 32];
#pragma unroll
      for (int h = 0; h < (TOKENS + 31) / 32; ++h)
        sx[h] = 32 * h + lane < a.rows ? a.x_scale[(long long)(32 * h + lane) * a.kblocks + kb] : 0.f;
      float sw[C::kMats];
#pragma unroll
      for (int m = 0; m < C::kMats; ++m) sw[m] = __ldg(a.w_scale + (long long)((m * a.N + n0) / 128) * a.kblocks + kb);
      if (!bounded_wait_warp(bars + kAccFull + buf, (n >> 1) & 1, abort_flag, a.status, kWaitNs)) return;
      ptx::tc_fence_after();
#pragma unroll
      for (int c = 0; c < TOKENS; c += 16) {
#pragma unroll
        for (int m = 0; m < C::kMats; ++m) {
          uint32_t r[16];
          ptx::tmem_ld16(lanes + (buf * C::kMats + m) * TOKENS + c, r);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            acc[m][c + e] = fmaf(__uint_as_float(r[e]),
                                 sw[m] * __shfl_sync(0xffffffffu, sx[(c + e) / 32], (c + e) & 31), acc[m][c + e]);
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bars + kAccEmpty + buf);
    }
#pragma unroll
    for (int m = 0; m < C::kMats; ++m)
#pragma unroll
      for (int j = 0; j < TOKENS; ++j) mine[(m * TOKENS + j) * 128] = acc[m][j];
  } else {
    if (!bounded_wait_warp(bars + kAccFull, 0, abort_flag, a.status, kWaitNs)) return;
    ptx::tc_fence_after();
#pragma unroll
    for (int j = 0; j < C::kMats * TOKENS; j += 16) {
      uint32_t r[16];
      ptx::tmem_ld16(lanes + j, r);
#pragma unroll
      for (int e = 0; e < 16; ++e) mine[(j + e) * 128] = __uint_as_float(r[e]);
    }
    ptx::tc_fence_before();
  }
}

template <bool E4M3, bool GATED, int ACT, int TOKENS>
__global__ void __launch_bounds__(kThreads, 2)
    k_few(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx, const FewArgs a) {
  using C = Cfg<GATED, TOKENS>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kBars];
  __shared__ int s_abort;
  __shared__ uint32_t tmem_slot;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  volatile int* abort_flag = &s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = a.cluster > 1 ? (int)ptx::cluster_rank() : 0, n0 = (int)(blockIdx.x / a.cluster) * 128;
  const int kb0 = a.kblocks * rank / a.cluster, kb1 = a.kblocks * (rank + 1) / a.cluster;
  const Loader<E4M3, GATED, TOKENS> in{a, &mw, &mx, sm, bars, n0, kb0};
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      ptx::mbar_init(bars + kFull + i, 1);
      ptx::mbar_init(bars + kEmpty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bars + kAccFull + i, 1);
      ptx::mbar_init(bars + kAccEmpty + i, kSumWarps);
    }
    ptx::mbar_init(bars + kDone, 1);
    s_abort = 0;
    ptx::fence_barrier_init();
    for (int j = 0; j < min(kb1 - kb0, C::kStages); ++j) in.weights(j);
  }
  // (Before TMEM is taken: a successor's CTA on this SM may take its 256 columns first and wait for this kernel, but shared
  // memory holds two CTAs of these kernels an SM at most, whose columns are 512 together.)
  ptx::successor_may_start();
  if (warp == 1) {
    ptx::tmem_alloc(&tmem_slot, kTmem);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_slot;
  float* const s_sum = reinterpret_cast<float*>(sm);  // over the ring, once every block has been summed
  if (warp == 0) load_rest<E4M3, GATED, TOKENS>(a, in, bars, abort_flag, kb1 - kb0, lane);
  else if (warp == 1) issue<E4M3, GATED, TOKENS>(a, sm, bars, tmem, abort_flag, kb1 - kb0);
  else collect<E4M3, GATED, TOKENS>(a, s_sum, bars, tmem, abort_flag, n0, kb0, kb1, warp, lane);
  __syncthreads();
  if (a.cluster > 1) ptx::cluster_sync();
  // a warp per token row: 128 columns, four a lane
  const int col = n0 + 4 * lane;
  for (int t = rank + a.cluster * warp; t < a.rows; t += a.cluster * (kThreads / 32)) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f), u = v;
    const float4* const at = reinterpret_cast<const float4*>(s_sum + t * 128) + lane;
    for (int r = 0; r < a.cluster; ++r) {
      v = sum_of(v, a.cluster > 1 ? remote_float4(at, r) : *at);
      if (GATED) u = sum_of(u, a.cluster > 1 ? remote_float4(at + TOKENS * 32, r) : at[TOKENS * 32]);
    }
    if (GATED) {
      const float2 a0 = values_of(mul_pairs(act_value<ACT>(pair_of(v.x, v.y)), pair_of(u.x, u.y)));
      const float2 a1 = values_of(mul_pairs(act_value<ACT>(pair_of(v.z, v.w)), pair_of(u.z, u.w)));
      v = make_float4(a0.x, a0.y, a1.x, a1.y);
    }
    const long long o = (long long)t * a.N + col;
    if constexpr (E4M3 && GATED) {
      float top = largest_or_nan(largest_or_nan(largest_or_nan(largest_or_nan(0.f, v.x), v.y), v.z), v.w);
      const bool fine = top <= kFloatMax;
      if (!fine) top = fmaxf(fmaxf(finite_size(v.x), finite_size(v.y)), fmaxf(finite_size(v.z), finite_size(v.w)));
#pragma unroll
      for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
      float inv;
      const float scale = block_scale(top, inv);
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.out) + o) =
          pack_e4m3(v.x * inv, v.y * inv, v.z * inv, v.w * inv, fine);
      if (lane == 0) a.out_scale[(long long)t * (a.N / 128) + n0 / 128] = scale;
    } else if (col < a.N) {
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + o) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (a.cluster > 1) ptx::cluster_sync();  // no CTA leaves while another reads its sums
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmem);
  }
}

template <bool E4M3, bool GATED, int ACT, int TOKENS>
cudaError_t run(const FewArgs& a, cudaStream_t st) {
  using C = Cfg<GATED, TOKENS>;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(done, (const void*)k_few<E4M3, GATED, ACT, TOKENS>, C::kDynamic);
  if (e != cudaSuccess) return e;
  CUtensorMap mw, mx;
  const long long wr = (long long)C::kMats * a.N;
  const bool ok = E4M3 ? encode_scaled(&mw, a.w, wr, a.K) && encode_scaled(&mx, a.x, a.rows, a.K, TOKENS)
                       : encode_map(&mw, a.w, wr, a.K, 128) && encode_map(&mx, a.x, a.rows, a.K, TOKENS);
  if (!ok) return cudaErrorInvalidValue;
  return launch_pairs(a.cluster, a.follows != 0, k_few<E4M3, GATED, ACT, TOKENS>, (a.N + 127) / 128 * a.cluster, kThreads,
                      C::kDynamic, st, mw, mx, a);
}
template <bool E4M3, bool GATED, int ACT>
cudaError_t by_rows(const FewArgs& a, cudaStream_t st) {
  if (a.rows <= 16) return run<E4M3, GATED, ACT, 16>(a, st);
  if (a.rows <= 32) return run<E4M3, GATED, ACT, 32>(a, st);
  return run<E4M3, GATED, ACT, 64>(a, st);
}
template <bool E4M3>
cudaError_t by_kind(bool gated, const FewArgs& a, cudaStream_t st) {
  if (!gated) return by_rows<E4M3, false, 0>(a, st);
  return a.act == REC_ATTN_SILU ? by_rows<E4M3, true, REC_ATTN_SILU>(a, st) : by_rows<E4M3, true, REC_ATTN_GELU>(a, st);
}

}  // namespace

cudaError_t launch_few(bool e4m3, bool gated, FewArgs a, int num_sms, cudaStream_t st) {
  if (few_is_thin(e4m3, gated, a)) return launch_thin(e4m3, gated, a, st);
  a.kblocks = e4m3 ? (a.K + 127) / 128 : (a.K + 63) / 64;
  a.cluster = 1;
  while (a.cluster < 8 && 2 * a.cluster <= a.kblocks && a.cluster * ((a.N + 127LL) / 128) <= num_sms) a.cluster *= 2;
  return e4m3 ? by_kind<true>(gated, a, st) : by_kind<false>(gated, a, st);
}

}  // namespace recattn
