// dense_fp32.cu -- the products of the gated feed-forward block in fp32, on the tensor cores.
//
// An fp32 value is the sum of three bf16 values (8 bits each: hi, mid, lo), and a product of two
// such sums is, to 2^-24 of it, that of six pairs: hi lo, mid mid, lo hi, hi mid, mid hi, hi hi (in
// this order, small ones first).  bf16 MMAs at a sixth of their rate are still five times CUDA cores.
// The tensor cores cut each addition's result off (measured: 2^-24 of the sum for each 16 products,
// always towards zero), so they sum no more than a block of 64; sixteen warps add the blocks up in
// fp32 registers, rounded to nearest.
// A pair of CTAs has a tile of 256 x 128 (gated: 64 gate and 64 up columns; the backward's dh 64); a
// ring of three 64-deep stages holds all six planes, so each is loaded once.  h and p are written as
// planes.  (kDglu spills 4 and 8 bytes at 96 registers a thread.)  1850 rows of 512 x 1024, forward and backward, 148 us (elementary fp32 operations 454): 22 R W H
// multiplied by six is 68 us at the bf16 rate; the rest is eleven kernels of one or two tiles a pair, each with the
// filling of its ring and an epilogue at its end.  7680 rows: tensor pipe 50 to 69%.
#include <cuda_bf16.h>

#include <atomic>

#include "dense.cuh"
#include "dense_device.cuh"
#include "launchers.cuh"
#include "ptx_sm103.cuh"
#include "wait.cuh"

namespace recattn {

namespace {

constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s
constexpr int kBK = 64, kSlab = 64 * 128;    // 64 rows of 128 bytes
constexpr int kPlane = 2 * kSlab;            // 128 rows of one plane
constexpr int kStage = 3 * (kPlane + kSlab), kStages = 3;  // 128 rows of A and this CTA's 64 of B
constexpr int kEpiWarps = 16, kThreads = 64 + 32 * kEpiWarps;
constexpr int kRun = 16;                     // columns that a thread takes up at a time
constexpr int kDynamic = kStages * kStage + 1024;
constexpr int kTileN = 128;
constexpr int kBufs = 4;  // buffers of a block's sums: all of TMEM (40000 rows, 512 x 1024, forward 492 us with two, 457)
constexpr uint32_t kTmem = kBufs * kTileN;

enum { kFull = 0, kEmpty = 3, kAccFull = 6, kAccEmpty = 10, kDone = 14, kBars = 15 };

template <DenseOp OP>
struct Cfg {
  static constexpr bool kPair = OP == DenseOp::kGlu || OP == DenseOp::kDglu;
  static constexpr bool kAMn = OP == DenseOp::kDw, kBMn = OP == DenseOp::kDx || OP == DenseOp::kDw;
  static constexpr int kCols = kPair ? 64 : 128;  // of the result
};

// The three planes of 64 columns (MN) or 64 or 128 rows (the map's box) at mn0, block kb of the summed axis, one
// after the other.
template <bool MN>
__device__ __forceinline__ void load_planes(uint8_t* dst, const CUtensorMap* map, int mn0, int kb, uint32_t bar) {
  if (MN) ptx::tma_load_3d_pair(dst, map, mn0, kb * kBK, 0, bar);
  else ptx::tma_load_3d_pair(dst, map, kb * kBK, mn0, 0, bar);
}

template <DenseOp OP>
__device__ void produce(const DenseArgs& a, const CUtensorMap* ma, const CUtensorMap* mb, const CUtensorMap* ma2,
                        const CUtensorMap* mb2, uint8_t* sm, uint64_t* bars, volatile int* abort_flag, uint32_t rank, int lane) {
  using C = Cfg<OP>;
  uint32_t n = 0;
  for (Units<C::kCols, DenseArgs> units(a, rank); units.left(); units.next()) {
    const Unit u = units.get();
    const int first = OP == DenseOp::kDglu ? a.kblocks : 0;  // blocks of dy and w_out before those of x and w_in
    for (int kb = u.kb0 - first; kb < u.kb1; ++kb, ++n) {
      const int st = n % kStages;
      if (!bounded_wait_warp(bars + kEmpty + st, ((n / kStages) & 1) ^ 1, abort_flag, a.status, kWaitNs)) goto out;
      if (ptx::elect_one()) {
        uint8_t* s = sm + st * kStage;
        const uint32_t bar = ptx::first_of_pair(bars + kFull + st);
        const bool grad = OP == DenseOp::kDglu && kb < 0;
        // (the first CTA's barrier counts the bytes of both; dh has 64 columns, 32 rows of B from each)
        if (rank == 0) ptx::mbar_arrive_expect_tx(bars + kFull + st, 2 * kStage);
        const int nb = C::kPair ? (rank ? a.N : 0) + u.n0 : u.n0 + 64 * (int)rank;  // gated: the gate's rows, up's
        uint8_t* const sb = s + 3 * kPlane;
        // kDx where p's halves do not adjoin: its second half and the up projection have maps of their own
        const int half = OP == DenseOp::kDx && a.pad ? (a.cut + kBK - 1) / kBK : INT32_MAX;
        if (OP == DenseOp::kDx && kb >= half) {
          load_planes<false>(s, ma2, u.m0, kb - half, bar);
          load_planes<true>(sb, mb2, nb, kb - half, bar);
        } else if (grad) {
          load_planes<false>(s, ma2, u.m0, kb + first, bar);
          load_planes<true>(sb, mb2, u.n0 + 32 * (int)rank, kb + first, bar);
        } else {
          load_planes<C::kAMn>(s, ma, u.m0, kb, bar);
          if (C::kAMn) load_planes<true>(s + 3 * kSlab, ma, u.m0 + 64, kb, bar);
          load_planes<C::kBMn>(sb, mb, nb, kb, bar);
        }
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

// The six pairs of a stage's planes into one buffer.
template <bool AMN, bool BMN, int N>
__device__ __forceinline__ void block_mma(uint32_t acc, uint32_t s) {
  const uint32_t idesc = ptx::idesc_bf16_f32(2 * kTile, N, AMN, BMN);
  // A's planes: 128 rows each, or (MN) 64 columns of each and then the other 64
  constexpr int kStepA = AMN ? kSlab : kPlane;
  const uint64_t da = ptx::smem_desc_sw128(s, AMN ? 3 * kSlab : 16, 1024);
  const uint64_t db = ptx::smem_desc_sw128(s + 3 * kPlane, BMN ? kSlab : 16, 1024);
  constexpr int kA[6] = {2, 1, 0, 1, 0, 0}, kB[6] = {0, 1, 2, 0, 1, 0};
#pragma unroll
  for (int j = 0; j < 6; ++j)
#pragma unroll
    for (int k = 0; k < kBK / 16; ++k)
      ptx::umma_pair<false>(acc, ptx::smem_desc_at(da, kA[j] * kStepA + k * (AMN ? 2048 : 32)),
                               ptx::smem_desc_at(db, kB[j] * kSlab + k * (BMN ? 2048 : 32)), idesc, j + k > 0);
}

template <DenseOp OP>
__device__ void issue(const DenseArgs& a, uint8_t* sm, uint64_t* bars, uint32_t tmem, volatile int* abort_flag) {
  using C = Cfg<OP>;
  const uint32_t s0 = ptx::smem_u32(sm);
  const bool el = ptx::elect_one();
  constexpr uint32_t rank = 0;  // the first CTA issues for both
  uint32_t n = 0;
  for (Units<C::kCols, DenseArgs> units(a, rank); units.left(); units.next()) {
    const Unit u = units.get();
    for (int kb = OP == DenseOp::kDglu ? -a.kblocks : u.kb0; kb < u.kb1; ++kb, ++n) {
      const int st = n % kStages;
      const uint32_t buf = n % kBufs;
      if (!bounded_wait_warp(bars + kAccEmpty + buf, ((n / kBufs) & 1) ^ 1, abort_flag, a.status, kWaitNs)) goto out;
      if (!bounded_wait_warp(bars + kFull + st, (n / kStages) & 1, abort_flag, a.status, kWaitNs)) goto out;
      ptx::tc_fence_after();
      if (el) {
        if (OP == DenseOp::kDglu && kb < 0) block_mma<false, true, 64>(tmem + buf * kTileN, s0 + st * kStage);
        else block_mma<C::kAMn, C::kBMn, kTileN>(tmem + buf * kTileN, s0 + st * kStage);
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

// x as hi + mid + lo.  (A finite value past bf16's largest is cut instead of rounded to infinity;
// one that is not finite is in hi alone.)
__device__ __forceinline__ void split3(float x, float& hi, float& mid, float& lo) {
  hi = __bfloat162float(__float2bfloat16_rn(x));
  if (!(fabsf(hi) <= 3.402823466e38f) && fabsf(x) <= 3.402823466e38f) hi = __uint_as_float(__float_as_uint(x) & 0xffff0000u);
  const float r = x - hi;
  const bool fine = fabsf(r) <= 3.402823466e38f;
  mid = fine ? __bfloat162float(__float2bfloat16_rn(r)) : 0.f;
  lo = fine ? r - mid : 0.f;
}
// Four columns of a row into the planes.
__device__ __forceinline__ void store_planes(const Planes& to, long long row, int col, float a, float b, float c, float d) {
  const float x[4] = {a, b, c, d};
  float v[3][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) split3(x[i], v[0][i], v[1][i], v[2][i]);
  char* at = static_cast<char*>(to.p) + (row * to.ld + col) * 2;
#pragma unroll
  for (int p = 0; p < 3; ++p, at += to.plane())
    *reinterpret_cast<uint2*>(at) = make_uint2(pack_bf16(v[p][0], v[p][1]), pack_bf16(v[p][2], v[p][3]));
}
// kRun columns from a 32-byte boundary on, `left` of which there are (whole sectors are written: four
// columns at a time took three times the traffic).
__device__ __forceinline__ void store_planes(const Planes& to, long long row, int col, const float (&x)[kRun], int left) {
  if (left >= kRun) {
    uint32_t w[3][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float a[3], b[3];
      split3(x[2 * e], a[0], a[1], a[2]);
      split3(x[2 * e + 1], b[0], b[1], b[2]);
#pragma unroll
      for (int p = 0; p < 3; ++p) w[p][e] = pack_bf16(a[p], b[p]);
    }
    char* at = static_cast<char*>(to.p) + (row * to.ld + col) * 2;
#pragma unroll
    for (int p = 0; p < 3; ++p, at += to.plane())
      ptx::st_global_v8(at, w[p][0], w[p][1], w[p][2], w[p][3], w[p][4], w[p][5], w[p][6], w[p][7]);
  } else {
#pragma unroll
    for (int c = 0; c < kRun; c += 4)
      if (c < left) store_planes(to, row, col + c, x[c], x[c + 1], x[c + 2], x[c + 3]);
  }
}
__device__ __forceinline__ void store8(float* dst, const float* x) {
  ptx::st_global_v8(dst, __float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]),
                    __float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
}
// The same in fp32; a row that starts between two sectors' borders has them whole but for the first and last (8000 x 516
// with hidden 1024: 136 -> 133 us).
__device__ __forceinline__ void store_floats(float* dst, const float (&x)[kRun], int left) {
  const bool off = (reinterpret_cast<uintptr_t>(dst) & 31) != 0;
  if (left >= kRun && !off) {
#pragma unroll
    for (int c = 0; c < kRun; c += 8) store8(dst + c, x + c);
  } else if (left >= kRun) {
    *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
#pragma unroll
    for (int c = 4; c + 8 < kRun; c += 8) store8(dst + c, x + c);
    *reinterpret_cast<float4*>(dst + kRun - 4) = make_float4(x[kRun - 4], x[kRun - 3], x[kRun - 2], x[kRun - 1]);
  } else {
#pragma unroll
    for (int c = 0; c < kRun; c += 4)
      if (c < left) *reinterpret_cast<float4*>(dst + c) = make_float4(x[c], x[c + 1], x[c + 2], x[c + 3]);
  }
}

template <DenseOp OP, int ACT>
__device__ void finish(const Dense32Args& aa, uint64_t* bars, uint32_t tmem, volatile int* abort_flag, uint32_t rank, int warp,
                       int lane) {
  using C = Cfg<OP>;
  const DenseArgs& a = aa.d;
  const int quad = warp & 3, part = (warp - 2) >> 2;
  const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
  // its columns of the tile: two runs (gated: of the gate's and of up's)
  const int c0 = C::kPair ? kRun * part : 2 * kRun * part, c1 = C::kPair ? 64 + c0 : c0 + kRun;
  const uint32_t empty = ptx::first_of_pair(bars + kAccEmpty);
  uint32_t n = 0;
  // a block's sums of a run, added up
  const auto take = [&](float (&to)[kRun], uint32_t buf, int col) {
    uint32_t r[kRun];
    ptx::tmem_ld16(lanes + buf * kTileN + col, r);
#pragma unroll
    for (int e = 0; e < kRun; ++e) to[e] += __uint_as_float(r[e]);
  };
  const auto taken = [&](uint32_t buf) {
    ptx::tc_fence_before();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive_pair(empty + 8 * buf);
  };
  for (Units<C::kCols, DenseArgs> units(a, rank); units.left(); units.next()) {
    const Unit u = units.get();
    float x0[kRun], x1[kRun], dh[OP == DenseOp::kDglu ? kRun : 1];
#pragma unroll
    for (int e = 0; e < kRun; ++e) x0[e] = x1[e] = 0.f;
    if constexpr (OP == DenseOp::kDglu) {
#pragma unroll
      for (int e = 0; e < kRun; ++e) dh[e] = 0.f;
      for (int kb = 0; kb < a.kblocks; ++kb, ++n) {
        if (!bounded_wait_warp(bars + kAccFull + n % kBufs, (n / kBufs) & 1, abort_flag, a.status, kWaitNs)) return;
        ptx::tc_fence_after();
        take(dh, n % kBufs, c0);
        taken(n % kBufs);
      }
    }
    for (int kb = u.kb0; kb < u.kb1; ++kb, ++n) {
      if (!bounded_wait_warp(bars + kAccFull + n % kBufs, (n / kBufs) & 1, abort_flag, a.status, kWaitNs)) return;
      ptx::tc_fence_after();
      take(x0, n % kBufs, c0);
      take(x1, n % kBufs, c1);
      taken(n % kBufs);
    }
    long long row = u.m0 + quad * 32 + lane;
    if (OP == DenseOp::kDw && a.pad && row >= a.cut) row = row < a.cut + a.pad ? a.M : row - a.pad;  // (between: none)
    if (row >= a.M) continue;
    if constexpr (C::kPair) {
      // in place: x0 becomes du, x1 h and dh dg
      const int col = u.n0 + c0, left = a.N - col;
#pragma unroll
      for (int e = 0; e < kRun; ++e) {
        float slope;
        const float act = act32<ACT>(x0[e], slope), up = x1[e];
        x1[e] = act * up;
        if constexpr (OP == DenseOp::kDglu) {
          x0[e] = dh[e] * act;
          dh[e] = dh[e] * up * slope;
        }
      }
      if (left > 0) {
        store_planes(aa.h, row, col, x1, left);
        if constexpr (OP == DenseOp::kDglu) {
          store_planes(aa.p, row, col, dh, left);
          store_planes(aa.p, row, a.N + a.pad + col, x0, left);
        }
      }
    } else {
      float* const out = (a.splits > 1 ? a.part + (long long)u.split * a.M * a.N : static_cast<float*>(a.out)) + row * a.N;
      if (u.n0 + c0 < a.N) store_floats(out + u.n0 + c0, x0, a.N - u.n0 - c0);
      if (u.n0 + c1 < a.N) store_floats(out + u.n0 + c1, x1, a.N - u.n0 - c1);
    }
  }
}

template <DenseOp OP, int ACT>
__global__ void __launch_bounds__(kThreads, 1)
    k_dense32(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
              const __grid_constant__ CUtensorMap ma2, const __grid_constant__ CUtensorMap mb2, const Dense32Args a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kBars];
  __shared__ int s_abort;
  __shared__ uint32_t tmem_slot;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  volatile int* abort_flag = &s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(bars + kFull + i, 1);
      ptx::mbar_init(bars + kEmpty + i, 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      ptx::mbar_init(bars + kAccFull + i, 1);
      ptx::mbar_init(bars + kAccEmpty + i, 2 * kEpiWarps);
    }
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
  ptx::predecessor_done();
  if (warp == 0) produce<OP>(a.d, &ma, &mb, &ma2, &mb2, sm, bars, abort_flag, rank, lane);
  else if (warp == 1 && rank == 0) issue<OP>(a.d, sm, bars, tmem, abort_flag);
  else if (warp > 1) finish<OP, ACT>(a, bars, tmem, abort_flag, rank, warp, lane);
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

// The planes of up to four matrices in one launch; first[i]: matrix i's first block.
struct SplitArgs {
  const float* x[4];
  Planes to[4];
  int first[5];
};
constexpr int kSplitRun = 4;  // float4s a thread
__global__ void __launch_bounds__(256) k_split(const SplitArgs a) {
  ptx::successor_may_start();
  int m = 0;
#pragma unroll
  for (int i = 1; i < 4; ++i) m += (int)blockIdx.x >= a.first[i];
  const Planes to = a.to[m];
  const float4* const x = reinterpret_cast<const float4*>(a.x[m]);
  const int per_row = (int)(to.cols / 4);
  const long long n = to.rows * per_row, i0 = (long long)((int)blockIdx.x - a.first[m]) * (256 * kSplitRun) + threadIdx.x;
  float4 v[kSplitRun];
#pragma unroll
  for (int k = 0; k < kSplitRun; ++k)
    if (i0 + 256 * k < n) v[k] = __ldcs(x + i0 + 256 * k);
#pragma unroll
  for (int k = 0; k < kSplitRun; ++k) {
    const long long i = i0 + 256 * k;
    if (i >= n) break;
    const long long row = n >> 32 ? i / per_row : (long long)((uint32_t)i / (uint32_t)per_row);
    store_planes(to, row, 4 * (int)(i - row * per_row), v[k].x, v[k].y, v[k].z, v[k].w);
  }
}

template <DenseOp OP, int ACT>
cudaError_t run(const CUtensorMap (&m)[4], Dense32Args a, int num_sms, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(done, (const void*)k_dense32<OP, ACT>, kDynamic);
  if (e != cudaSuccess) return e;
  a.d.tiles_m = (a.d.M + (OP == DenseOp::kDw ? a.d.pad : 0) + 2 * kTile - 1) / (2 * kTile);
  a.d.tiles_n = (a.d.N + Cfg<OP>::kCols - 1) / Cfg<OP>::kCols;
  const int units = a.d.tiles_m * a.d.tiles_n * a.d.splits, places = num_sms / 2;
  return launch_pairs(2, true, k_dense32<OP, ACT>, (units < places ? units : places) * 2, kThreads, kDynamic, st, m[0], m[1],
                      m[2], m[3], a);
}

}  // namespace

cudaError_t launch_split(const SplitList& l, cudaStream_t st) {
  SplitArgs a{};
  long long blocks = 0;
  for (int i = 0; i < 4; ++i) {
    a.first[i] = (int)blocks;
    if (i >= l.n) continue;
    a.x[i] = static_cast<const float*>(l.x[i]);
    a.to[i] = l.to[i];
    blocks += (l.to[i].rows * (l.to[i].cols / 4) + 256 * kSplitRun - 1) / (256 * kSplitRun);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  }
  for (int i = l.n; i < 5; ++i) a.first[i] = INT32_MAX;
  k_split<<<(unsigned)blocks, 256, 0, st>>>(a);
  return cudaGetLastError();
}

// Parts of the summed axis that give every pair of SMs work: each at least four blocks deep.  (At least one, two, four,
// eight and sixteen blocks, us on the device: forward of 500 rows of 128 x 4096 32.3, 26.7, 25.7, 27.6, 33.4; of 200 rows of
// 512 x 1024 26.1, 25.2, 26.3, 29.0, 33.8; with backward, 200 rows of 128 x 4096 86.6, 73.6, 68.8, 71.6, 82.5, 4000 rows of
// 256 x 256 88.0, 86.1, 78.2, 82.2, 99.8, 1850 of 512 x 1024 137, 137, 137, 138, 162.)
int dense32_splits(int M, int N, int kblocks, int num_sms) {
  const long long tiles = (long long)((M + 2 * kTile - 1) / (2 * kTile)) * ((N + kTileN - 1) / kTileN);
  long long s = num_sms / 2 / tiles;
  if (s > kblocks / 4) s = kblocks / 4;
  return s < 1 ? 1 : (int)s;
}

cudaError_t launch_dense32(DenseOp op, const CUtensorMap (&m)[4], Dense32Args a, int num_sms, cudaStream_t st) {
  switch (op) {
    case DenseOp::kGlu:
      return a.d.act == REC_ATTN_SILU ? run<DenseOp::kGlu, REC_ATTN_SILU>(m, a, num_sms, st)
                                      : run<DenseOp::kGlu, REC_ATTN_GELU>(m, a, num_sms, st);
    case DenseOp::kDglu:
      return a.d.act == REC_ATTN_SILU ? run<DenseOp::kDglu, REC_ATTN_SILU>(m, a, num_sms, st)
                                      : run<DenseOp::kDglu, REC_ATTN_GELU>(m, a, num_sms, st);
    case DenseOp::kOut: return run<DenseOp::kOut, 0>(m, a, num_sms, st);
    case DenseOp::kDx: return run<DenseOp::kDx, 0>(m, a, num_sms, st);
    case DenseOp::kDw: return run<DenseOp::kDw, 0>(m, a, num_sms, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace recattn
