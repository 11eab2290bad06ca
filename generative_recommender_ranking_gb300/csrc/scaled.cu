// scaled.cu -- e4m3 matrices with a scale for each block of 128: the quantizer, and the product on
// the sm_103a tensor cores.
//
// Quantizer: a block's scale is the least power of two that brings its largest value to at most 448,
// so x / scale is exact and each value is rounded once, to the nearest e4m3 (ties to even).  A
// floating-point format loses nothing by a power of two but the last step below 2^-6 of its range.
//
// Product: y[m][n] = sum over blocks b of sa[m][b] sb[n / 128][b] (sum over the block's k of a[m][k]
// b[n][k]).  A pair of CTAs has a tile of 256 x 256; the tensor cores sum one block into one of two TMEM
// buffers; sixteen warps take it up, times its scales, into fp32 sums in registers (64 a thread, two to
// an instruction) while the next block is summed.  So the scales may be any fp32, and no sum of more than
// 128 products is the tensor cores' own.  The gated form takes 128 gate and 128 up columns as a tile and writes
// their product in e4m3 with its scales.
// 16387 x 8192 x 4096: 472 us (2.3 PFLOP/s; without taking sums up 3.5).  A block takes 1060 cycles where its MMAs
// take 540: the sixteen warps bound it (waking, two reads of 32 columns, their multiply-adds, the next block's
// scales), so that two issuing warps with half a tile each changed nothing; more buffers do not fit TMEM.  The
// gated form on 320016 rows of 512 x 1024: 414 us under ncu, half of it the tile's epilogue.  Sixteen warps of 112
// registers read 32 columns at a time; eight warps of 168, or 16 columns at a time: 562 and 603 us where these
// took 508.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <atomic>

#include "dense.cuh"
#include "dense_device.cuh"
#include "launchers.cuh"
#include "ptx_sm103.cuh"
#include "quantize.cuh"
#include "scaled.cuh"
#include "wait.cuh"

namespace recattn {

namespace {

// ------------------------------------------------------------------ quantizer
// Sixteen neighbouring values of a row (widths are multiples of 16): 16 bytes of e4m3.
template <typename E>
struct Run;
template <>
struct Run<__nv_bfloat16> {
  uint4 v[2];
  __device__ __forceinline__ float at(int k) const {
    const uint4 h = v[k >> 3];
    const uint32_t w = (k & 7) < 2 ? h.x : (k & 7) < 4 ? h.y : (k & 7) < 6 ? h.z : h.w;
    return __uint_as_float(k & 1 ? w & 0xffff0000u : w << 16);
  }
};
template <>
struct Run<float> {
  uint4 v[4];
  __device__ __forceinline__ float at(int k) const {
    const uint4 h = v[k >> 2];
    return __uint_as_float((k & 3) == 0 ? h.x : (k & 3) == 1 ? h.y : (k & 3) == 2 ? h.z : h.w);
  }
};
template <typename E>
__device__ __forceinline__ void load_run(Run<E>& r, const void* x, long long i, bool in) {
  constexpr int kN = sizeof(Run<E>) / 16;
#pragma unroll
  for (int k = 0; k < kN; ++k) r.v[k] = in ? __ldcs(static_cast<const uint4*>(x) + i * kN + k) : make_uint4(0, 0, 0, 0);
}
// The largest finite size; fine: there are no others.
template <typename E>
__device__ __forceinline__ float largest(const Run<E>& x, bool& fine) {
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) m = largest_or_nan(m, x.at(k));
  fine = m <= kFloatMax;
  if (!fine) {
    m = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) m = fmaxf(m, finite_size(x.at(k)));
  }
  return m;
}
template <typename E>
__device__ __forceinline__ uint4 quantized(const Run<E>& x, float inv, bool fine) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    w[k] = pack_e4m3(x.at(4 * k) * inv, x.at(4 * k + 1) * inv, x.at(4 * k + 2) * inv, x.at(4 * k + 3) * inv, fine);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int kQuantThreads = 256, kRunBf16 = 4, kRunFp32 = 2;

// A scale per row and 128 columns: 8 lanes a block, RUN blocks of theirs in flight.  HBM-bound: 320016
// rows of 512 bf16 take 76 us (6.5 TB/s).
template <typename E, int RUN>
__global__ void __launch_bounds__(kQuantThreads) k_quantize_rows(QuantArgs a) {
  ptx::successor_may_start();
  const int lane = threadIdx.x & 7, runs = a.width / 16;
  const long long units = a.rows * a.blocks, groups = (long long)gridDim.x * (kQuantThreads / 8);
  const long long first = (long long)blockIdx.x * (kQuantThreads / 8) + (threadIdx.x >> 3);
  for (long long u0 = first; u0 - (threadIdx.x >> 3 & 3) < units; u0 += groups * RUN) {  // (a warp's groups together)
    Run<E> x[RUN];
    long long at[RUN];
#pragma unroll
    for (int j = 0; j < RUN; ++j) {
      const long long u = u0 + j * groups;
      const long long row = units >> 32 ? u / a.blocks : (long long)((uint32_t)u / (uint32_t)a.blocks);
      const int c = (int)(u - row * a.blocks) * 8 + lane;
      const bool in = u < units && c < runs;
      at[j] = in ? row * runs + c : -1;
      load_run(x[j], a.x, at[j], in);
    }
#pragma unroll
    for (int j = 0; j < RUN; ++j) {
      bool fine;
      float top = largest(x[j], fine);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      float inv;
      const float scale = block_scale(top, inv);
      if (at[j] >= 0) {
        reinterpret_cast<uint4*>(a.q)[at[j]] = quantized(x[j], inv, fine);
        if (lane == 0) a.scale[u0 + j * groups] = scale;
      }
    }
  }
}

// A scale per 128 x 128 block: one thread block each, its values in registers meanwhile.
template <typename E>
__global__ void __launch_bounds__(kQuantThreads) k_quantize_blocks(QuantArgs a) {
  __shared__ float s_top[kQuantThreads / 32];
  const int runs = a.width / 16, c = (int)(blockIdx.x % a.blocks) * 8 + (threadIdx.x & 7);
  const long long row0 = (long long)(blockIdx.x / a.blocks) * kScaleBlock + (threadIdx.x >> 3);
  Run<E> x[4];
  float top = 0.f;
  bool all_fine = true;
#pragma unroll
  for (int j = 0; j < 4; ++j) load_run(x[j], a.x, (row0 + 32 * j) * runs + c, row0 + 32 * j < a.rows && c < runs);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    bool fine;
    top = fmaxf(top, largest(x[j], fine));
    all_fine = all_fine && fine;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQuantThreads / 32; ++w) top = fmaxf(top, s_top[w]);
  float inv;
  const float scale = block_scale(top, inv);
  if (threadIdx.x == 0) a.scale[blockIdx.x] = scale;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (row0 + 32 * j < a.rows && c < runs)
      reinterpret_cast<uint4*>(a.q)[(row0 + 32 * j) * runs + c] = quantized(x[j], inv, all_fine);
}

// ------------------------------------------------------------------ product
constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s
constexpr int kBN = 256;                     // columns of B a tile
constexpr int kSlab = 128 * 128;             // 128 rows of a block: 128 bytes each
constexpr int kStage = 2 * kSlab, kStages = 6;  // a CTA's 128 rows of A and its half of B's 256
constexpr int kEpiWarps = 16, kThreads = 128 + 32 * kEpiWarps;
// Registers a thread: what the block is launched with, and then of the loading and issuing warpgroup and
// of the four that hold sums (64 of them, and the 32 that are being taken up).
constexpr int kRegs = 96, kFewRegs = 32, kSumRegs = 112;
static_assert(128 * kFewRegs + 32 * kEpiWarps * kSumRegs <= kThreads * kRegs, "the split is the block's own");
constexpr int kDynamic = kStages * kStage + 1024;
constexpr uint32_t kTmem = 512;               // two buffers of a block's sums

enum { kFull = 0, kEmpty = 6, kAccFull = 12, kAccEmpty = 14, kParts = 16, kDone = 20, kBars = 21 };

// A pair's tiles (parts of their summed axis) in turn; n0: the first column of the result.
template <bool GATED, bool PARTS>
using Work = Units<GATED ? kBN / 2 : kBN, ScaledArgs, PARTS>;

template <bool GATED, bool PARTS>
__device__ void produce(const ScaledArgs& a, const CUtensorMap* ma, const CUtensorMap* mb, uint8_t* sm, uint64_t* bars,
                        volatile int* abort_flag, uint32_t rank, int lane) {
  uint32_t n = 0;
  for (Work<GATED, PARTS> work(a, rank); work.left(); work.next()) {
    const Unit u = work.get();
    // gated: the gate's columns are the first CTA's rows of B, up's the second's
    const int nb = u.n0 + (rank ? (GATED ? a.N : kBN / 2) : 0);
    for (int kb = u.kb0; kb < u.kb1; ++kb, ++n) {
      const int st = n % kStages;
      if (!bounded_wait_warp(bars + kEmpty + st, ((n / kStages) & 1) ^ 1, abort_flag, a.status, kWaitNs)) goto out;
      if (ptx::elect_one()) {
        uint8_t* s = sm + st * kStage;
        const uint32_t bar = ptx::first_of_pair(bars + kFull + st);
        if (rank == 0) ptx::mbar_arrive_expect_tx(bars + kFull + st, 2 * kStage);  // the bytes of both CTAs
        ptx::tma_load_2d_pair(s, ma, kb * 128, u.m0, bar);
        ptx::tma_load_2d_pair(s + kSlab, mb, kb * 128, nb, bar);
      }
      __syncwarp();
    }
  }
out:
  // after an abort, copies may still be in flight (those of a pair count on the first CTA's barriers)
  if (lane == 0 && rank == 0)
    for (uint32_t j = n > kStages ? n - kStages : 0; j < n; ++j)
      bounded_drain(bars + kFull + j % kStages, (j / kStages) & 1, kWaitNs / 4);
  __syncwarp();
}

// The first CTA issues for both.
template <bool GATED, bool PARTS>
__device__ __forceinline__ void issue(const ScaledArgs& a, uint8_t* sm, uint64_t* bars, uint32_t tmem,
                                      volatile int* abort_flag) {
  const uint32_t s0 = ptx::smem_u32(sm), idesc = ptx::idesc_e4m3_f32(2 * kTile, kBN);
  const bool el = ptx::elect_one();
  uint32_t n = 0;
  for (Work<GATED, PARTS> work(a, 0); work.left(); work.next()) {
    const Unit u = work.get();
    for (int kb = u.kb0; kb < u.kb1; ++kb, ++n) {
      const int st = n % kStages;
      const uint32_t buf = n & 1;
      if (!bounded_wait_warp(bars + kAccEmpty + buf, ((n >> 1) & 1) ^ 1, abort_flag, a.status, kWaitNs)) goto out;
      if (!bounded_wait_warp(bars + kFull + st, (n / kStages) & 1, abort_flag, a.status, kWaitNs)) goto out;
      ptx::tc_fence_after();
      if (el) {
        const uint64_t da = ptx::smem_desc_sw128(s0 + st * kStage, 16, 1024);
        const uint64_t db = ptx::smem_desc_sw128(s0 + st * kStage + kSlab, 16, 1024);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          ptx::umma_pair<true>(tmem + buf * kBN, ptx::smem_desc_at(da, 32 * k), ptx::smem_desc_at(db, 32 * k), idesc, k > 0);
        ptx::umma_commit_pair(bars + kEmpty + st);
        ptx::umma_commit_pair(bars + kAccFull + buf);
      }
      __syncwarp();
    }
  }
out:
  if (el) {
    ptx::umma_commit_pair(bars + kDone);
    bounded_drain(bars + kDone, 0, kWaitNs / 4);
  }
  __syncwarp();
}

// A row's scales of four blocks (n are left): every thread of a warp reads another row, 32 sectors, so they
// are read together.  (Plain loads: the kernel may have started before they were written.)
__device__ __forceinline__ float4 next_scales(const float* s, int n, bool aligned) {
  if (aligned) return *reinterpret_cast<const float4*>(s);
  return make_float4(s[0], n > 1 ? s[1] : 0.f, n > 2 ? s[2] : 0.f, n > 3 ? s[3] : 0.f);
}

// Sixteen warps: a thread has one row and a quarter of the tile's columns (gated: 32 gate columns and
// the 32 up columns that belong to them).
template <bool GATED, int ACT, bool PARTS>
__device__ void finish(const ScaledArgs& a, uint64_t* bars, uint32_t tmem, volatile int* abort_flag, float* s_top,
                       uint32_t rank, int warp, int lane) {
  // Scales are read a block, and over a tile's end, ahead: 16387 x 8192 x 4096 500 -> 472 us (487 without the
  // step over the end).  The gated form has no registers for each block's (a block of 512 to 1024 columns on 320016
  // rows 737 -> 757 us); it reads a tile's first when the sums of the one before are done with (717 -> 685).  Parts
  // read none ahead (spills).
  constexpr bool kEarly = !GATED && !PARTS, kFirst = !PARTS;
  const int quad = warp & 3, part = (warp - 4) >> 2;
  const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16) + (GATED ? 32 : 64) * part;
  const uint32_t empty = ptx::first_of_pair(bars + kAccEmpty);
  const bool aligned = (a.kblocks & 3) == 0;  // (a.a_scale is on a 16-byte boundary)
  Work<GATED, PARTS> work(a, rank);
  // the tile, this thread's row of it, and the scales of the row and of its first and second 32 columns' block
  Unit u;
  bool in;
  const float *sa, *sb0, *sb1;
  float4 s4 = make_float4(0.f, 0.f, 0.f, 0.f);
  float b0 = 0.f;
  auto begin = [&] {
    u = work.get();
    const long long row = u.m0 + quad * 32 + lane;
    in = row < a.M;
    sa = a.a_scale + (in ? row : 0) * a.kblocks;
    const int nb = u.n0 / 128 + (GATED ? 0 : part >> 1);
    const bool nb_in = GATED || (long long)nb * 128 < a.N;
    sb0 = a.b_scale + (long long)(nb_in ? nb : 0) * a.kblocks;
    sb1 = GATED ? a.b_scale + (long long)(a.N / 128 + nb) * a.kblocks : sb0;
    if (kFirst && u.kb0 < u.kb1) s4 = next_scales(sa + (u.kb0 & ~3), a.kblocks - (u.kb0 & ~3), aligned);
    if (kEarly && u.kb0 < u.kb1) b0 = __ldg(sb0 + u.kb0);
  };
  uint32_t n = 0;
  if (kFirst && work.left()) begin();
  for (uint32_t it = 0; work.left(); ++it) {
    if (!kFirst) begin();
    f32x2 sums[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) sums[e] = 0ull;
    for (int kb = u.kb0; kb < u.kb1; ++kb, ++n) {
      if (!kEarly && (PARTS ? (kb & 3) == 0 || kb == u.kb0 : (kb & 3) == 0 && kb > 0))
        s4 = next_scales(sa + (kb & ~3), a.kblocks - (kb & ~3), aligned);
      const float sk = (kb & 2) ? (kb & 1 ? s4.w : s4.z) : (kb & 1 ? s4.y : s4.x);
      const float f0 = sk * (kEarly ? b0 : __ldg(sb0 + kb)), f1 = GATED ? sk * __ldg(sb1 + kb) : f0;
      if (kEarly && kb + 1 < u.kb1) {
        b0 = __ldg(sb0 + kb + 1);
        if ((kb & 3) == 3) s4 = next_scales(sa + kb + 1, a.kblocks - kb - 1, aligned);
      }
      const uint32_t buf = n & 1;
      if (!bounded_wait_voted(bars + kAccFull + buf, (n >> 1) & 1, abort_flag, a.status, kWaitNs)) return;
      ptx::tc_fence_after();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t r[32];
        ptx::tmem_ld32(lanes + buf * kBN + c * (GATED ? 128 : 32), r);
        if (c == 1) {  // the buffer goes back before its last columns are added
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive_pair(empty + 8 * buf);
        }
        const f32x2 f = GATED && c ? pair_of(f1, f1) : pair_of(f0, f0);
#pragma unroll
        for (int e = 0; e < 16; ++e)
          sums[16 * c + e] = fma_pairs(pair_of(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])), f, sums[16 * c + e]);
      }
    }
    const Unit at = u;
    const bool here = in;
    const long long row = at.m0 + quad * 32 + lane;
    if (kEarly) {  // the next tile's first scales travel while this tile is written
      work.next();
      if (work.left()) begin();
    }
    if constexpr (GATED) {
      float acc[32], top = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float2 v = values_of(mul_pairs(act_value<ACT>(sums[e]), sums[16 + e]));
        acc[2 * e] = v.x;
        acc[2 * e + 1] = v.y;
        top = largest_or_nan(largest_or_nan(top, v.x), v.y);
      }
      const bool fine = top <= kFloatMax;
      if (!fine) {
        top = 0.f;
#pragma unroll
        for (int e = 0; e < 32; ++e) top = fmaxf(top, finite_size(acc[e]));
      }
      // the other parts' largest values; the tiles take two places in turn
      float* s = s_top + (it & 1) * 512 + quad * 32 + lane;
      s[part * 128] = top;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bars + kParts + quad);
      work.next();
      if (work.left()) begin();
      if (!bounded_wait_voted(bars + kParts + quad, it & 1, abort_flag, a.status, kWaitNs)) return;
      top = fmaxf(fmaxf(s[0], s[128]), fmaxf(s[256], s[384]));
      float inv;
      const float scale = block_scale(top, inv);
      if (here) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          w[e] = pack_e4m3(acc[4 * e] * inv, acc[4 * e + 1] * inv, acc[4 * e + 2] * inv, acc[4 * e + 3] * inv, fine);
        ptx::st_global_v8(static_cast<uint8_t*>(a.out) + row * a.N + at.n0 + part * 32, w[0], w[1], w[2], w[3], w[4],
                          w[5], w[6], w[7]);
        if (part == 0) a.out_scale[row * (a.N / 128) + at.n0 / 128] = scale;
      }
    } else {
      const int col0 = at.n0 + part * 64;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int col = col0 + 16 * c;
        if constexpr (PARTS) {
          ulonglong2* const dst = reinterpret_cast<ulonglong2*>(a.part + ((long long)at.split * a.M + row) * a.N + col);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (here && col + 4 * e < a.N) dst[e] = make_ulonglong2(sums[8 * c + 2 * e], sums[8 * c + 2 * e + 1]);
        } else {
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = pack_bf16(sums[8 * c + e]);
          if (here && col < a.N) store_bf16(static_cast<__nv_bfloat16*>(a.out) + row * a.N + col, w, a.N - col, a.wide);
        }
      }
    }
    if (!kFirst) work.next();
  }
}

template <bool GATED, int ACT, bool PARTS>
__global__ void __maxnreg__(kRegs)
    k_scaled(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb, const ScaledArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kBars];
  __shared__ int s_abort;
  __shared__ uint32_t tmem_slot;
  __shared__ float s_top[GATED ? 1024 : 1];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  volatile int* abort_flag = &s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(bars + kFull + i, 1);
      ptx::mbar_init(bars + kEmpty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bars + kAccFull + i, 1);
      ptx::mbar_init(bars + kAccEmpty + i, 2 * kEpiWarps);
    }
    for (int i = 0; i < 4; ++i) ptx::mbar_init(bars + kParts + i, kEpiWarps / 4);
    ptx::mbar_init(bars + kDone, 1);
    s_abort = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 1) ptx::tmem_alloc_pair(&tmem_slot, kTmem);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();  // both CTAs' barriers are there
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_slot, rank = ptx::cluster_rank();
  ptx::successor_may_start();
  if (a.follows) ptx::predecessor_done();
  if (warp < 4) {
    ptx::fewer_registers<kFewRegs>();
    if (warp == 0) produce<GATED, PARTS>(a, &ma, &mb, sm, bars, abort_flag, rank, lane);
    else if (warp == 1 && rank == 0) issue<GATED, PARTS>(a, sm, bars, tmem, abort_flag);
  } else {
    ptx::more_registers<kSumRegs>();
    finish<GATED, ACT, PARTS>(a, bars, tmem, abort_flag, s_top, rank, warp, lane);
  }
  ptx::tc_fence_before();
  __syncthreads();
  // nothing of one CTA's reaches into the other any more, the last commit too
  if (warp == 1 && rank == 1 && lane == 0) bounded_drain(bars + kDone, 0, kWaitNs / 4);
  __syncwarp();
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, kTmem);
  }
}

template <bool GATED, int ACT, bool PARTS>
cudaError_t run(const CUtensorMap& ma, const CUtensorMap& mb, ScaledArgs a, int num_sms, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(done, (const void*)k_scaled<GATED, ACT, PARTS>, kDynamic);
  if (e != cudaSuccess) return e;
  const int tn = GATED ? kBN / 2 : kBN;
  static std::atomic<int> regs{0};
  if (!launched_with(regs, (const void*)k_scaled<GATED, ACT, PARTS>, kRegs)) return cudaErrorInvalidConfiguration;
  a.tiles_m = (a.M + 2 * kTile - 1) / (2 * kTile);
  a.tiles_n = (a.N + tn - 1) / tn;
  const int tiles = a.tiles_m * a.tiles_n * (PARTS ? a.splits : 1), places = num_sms / 2;
  return launch_pairs(2, a.follows != 0, k_scaled<GATED, ACT, PARTS>, (tiles < places ? tiles : places) * 2, kThreads,
                      kDynamic, st, ma, mb, a);
}

}  // namespace

cudaError_t launch_quantize(const QuantArgs& a, int dtype, int block_rows, int num_sms, cudaStream_t st) {
  const bool bf16 = dtype == REC_ATTN_BF16;
  if (block_rows == 1) {
    const int run = bf16 ? kRunBf16 : kRunFp32;
    const long long units = a.rows * a.blocks, per = kQuantThreads / 8 * run, blocks = (units + per - 1) / per;
    const unsigned grid = (unsigned)(blocks < 32LL * num_sms ? blocks : 32LL * num_sms);
    if (bf16) k_quantize_rows<__nv_bfloat16, kRunBf16><<<grid, kQuantThreads, 0, st>>>(a);
    else k_quantize_rows<float, kRunFp32><<<grid, kQuantThreads, 0, st>>>(a);
  } else {
    const unsigned grid = (unsigned)((a.rows + kScaleBlock - 1) / kScaleBlock * a.blocks);
    if (bf16) k_quantize_blocks<__nv_bfloat16><<<grid, kQuantThreads, 0, st>>>(a);
    else k_quantize_blocks<float><<<grid, kQuantThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_scaled(bool gated, const CUtensorMap& ma, const CUtensorMap& mb, ScaledArgs a, int num_sms,
                          cudaStream_t st) {
  if (!gated) return a.splits > 1 ? run<false, 0, true>(ma, mb, a, num_sms, st) : run<false, 0, false>(ma, mb, a, num_sms, st);
  return a.act == REC_ATTN_SILU ? run<true, REC_ATTN_SILU, false>(ma, mb, a, num_sms, st)
                                : run<true, REC_ATTN_GELU, false>(ma, mb, a, num_sms, st);
}

}  // namespace recattn
