// dense_tc.cu -- the matrix products of the gated feed-forward block on the sm_103a tensor cores.
//
// y = (act(x Wg') * (x Wu')) w_out' over packed token rows, and its gradients (dense.cuh lists the
// five products).  A persistent pair of CTAs takes tiles of 256 x 256 (cta_group::2: each CTA loads its 128
// rows of A and half of B, two thirds of what two single CTAs would); a TMA warp keeps a ring of 64-deep
// operand blocks full, one warp of the first CTA issues tcgen05 MMAs into TMEM, eight or sixteen warps read a
// finished tile out while the next one is summed.
//  - kGlu: a tile's 256 columns are 128 gate and the 128 up columns that belong to them, so the
//    activation and the product happen in the epilogue and neither projection reaches memory.
//  - kDglu: nothing of the forward is kept; g and u are summed again (256 columns) beside
//    dh = dy w_out (128 columns).  dh has two buffers and goes first: while it is summed for the
//    next tile the epilogue reads this tile's g and u, which have one.
//  - kDw sums over the rows; they (of kOut and kDx the summed axis, where tiles are few) are split into
//    parts so that all SMs have work, and the parts' sums are added in a fixed order (k_dense_sum).
// Sums are fp32 in TMEM (each addition cut, 2^-24 of the sum for every 16 products: measured 3e-5 over 32768,
// under the 2^-9 of the results' rounding); h and p are rounded to bf16 once, as operands of the next product.
// 320016 rows of 512 x 1024 (us under ncu, rate): kGlu 348-363 (1.9 PFLOP/s, tensor pipe 85%), kOut 183-190 (1.8),
// kDglu 660-685 (1.5; its epilogue, 8 of a tile's 10 thousand cycles, bounds it: three stores and the activation's
// exponential and reciprocal), kDx 348-367 (1.9), kDw 354-373 and 189-197 (1.9 and 1.7).  In a loop the
// board's power cap takes another fifth.  Single CTAs of 128 x 256: kGlu 438, kOut 231, kDx 424, kDw 544.  Clusters of two
// pairs with A multicast between them, and fetching A into the L2 ahead, gained nothing.
#include <atomic>

#include "dense.cuh"
#include "dense_device.cuh"
#include "launchers.cuh"
#include "ptx_sm103.cuh"
#include "wait.cuh"

namespace recattn {

namespace {

__device__ int g_dense_status;

constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s
constexpr int kBK = 64;                      // a block along the summed axis: 128 bytes
constexpr int kSlab = 64 * 128;              // 64 rows of 128 bytes
constexpr int kBN = 256;                     // columns of B a tile; a CTA loads 128 rows of either operand

template <DenseOp OP>
struct Cfg {
  static constexpr bool kPair = OP == DenseOp::kGlu || OP == DenseOp::kDglu;  // gate and up columns
  static constexpr bool kAMn = OP == DenseOp::kDw, kBMn = OP == DenseOp::kDx || OP == DenseOp::kDw;
  static constexpr int kTileN = kPair ? kBN / 2 : kBN;  // columns of the result
  // Warps of the epilogue: 16 where it computes the activation (of kDglu 901 us with 8)
  static constexpr int kEpiWarps = kPair ? 16 : 8, kThreads = 128 + 32 * kEpiWarps;
  // Registers a thread, as the block is launched (what an SM has for it); kDglu: then of the loading and issuing
  // warpgroup and of the four that hold g, u and dh
  static constexpr bool kSplitRegs = OP == DenseOp::kDglu;
  static constexpr int kRegs = 65536 / kThreads / 8 * 8, kFewRegs = 32, kSumRegs = 112;
  static_assert(!kSplitRegs || 128 * kFewRegs + 512 * kSumRegs <= kThreads * kRegs, "the split is the block's own");
  static constexpr int kTileM = 2 * kTile;
  static constexpr int kBRows = kBN / 2;               // of B in this CTA
  static constexpr int kStage = 2 * kSlab + kBRows * 128;
  static constexpr int kStages = 6 * 32 * 1024 / kStage;
  static constexpr int kDynamic = kStages * kStage + 1024;
  static constexpr uint32_t kTmem = 2 * kBN;  // kDglu: g, u and two buffers of dh
};

// Barriers
enum { kFull = 0, kEmpty = 8, kAccFull = 16, kAccEmpty = 18, kGuEmpty = 20, kDone = 21, kBars = 22 };

// ------------------------------------------------------------------ loads
// 128 rows of one operand at mn0 (MN: `rows` columns of it, a multiple of 64), block kb of the summed axis.  One
// copy where a box can hold them: the loading warp needs about 100 cycles a copy (measured: 394 for a block's
// four copies of 64 rows, which bounded the kernels at 570 cycles a block).
template <bool MN>
__device__ __forceinline__ void load_operand(uint8_t* dst, const CUtensorMap* map, int mn0, int rows, int kb, uint32_t bar) {
  if (MN) {
    for (int i = 0; i < rows / 64; ++i) ptx::tma_load_2d_pair(dst + i * kSlab, map, mn0 + 64 * i, kb * kBK, bar);
  } else {
    ptx::tma_load_2d_pair(dst, map, kb * kBK, mn0, bar);
  }
}

template <DenseOp OP>
__device__ void produce(const DenseArgs& a, const CUtensorMap* ma, const CUtensorMap* mb, const CUtensorMap* ma2,
                        const CUtensorMap* mb2, uint8_t* sm, uint64_t* bars, volatile int* abort_flag, uint32_t rank, int lane) {
  using C = Cfg<OP>;
  uint32_t n = 0;
  for (Units<C::kTileN, DenseArgs> units(a, rank); units.left(); units.next()) {
    const Unit u = units.get();
    const int first = OP == DenseOp::kDglu ? a.kblocks : 0;  // blocks of dy and w_out before those of x and w_in
    for (int kb = u.kb0 - first; kb < u.kb1; ++kb, ++n) {
      const int st = n % C::kStages;
      if (!bounded_wait_warp(bars + kEmpty + st, ((n / C::kStages) & 1) ^ 1, abort_flag, a.status, kWaitNs)) goto out;
      if (ptx::elect_one()) {
        uint8_t* s = sm + st * C::kStage;
        const uint32_t bar = ptx::first_of_pair(bars + kFull + st);
        const bool grad = OP == DenseOp::kDglu && kb < 0;
        // (the first CTA's barrier counts the bytes of both)
        if (rank == 0) ptx::mbar_arrive_expect_tx(bars + kFull + st, 2 * (grad ? 2 * kSlab + C::kBRows * 64 : C::kStage));
        // kDx where p's halves do not adjoin: its second half and the up projection have maps of their own
        const int half = OP == DenseOp::kDx && a.pad ? (a.cut + kBK - 1) / kBK : INT32_MAX;
        if (OP == DenseOp::kDx && kb >= half) {
          load_operand<false>(s, ma2, u.m0, kTile, kb - half, bar);
          load_operand<true>(s + 2 * kSlab, mb2, u.n0 + (int)rank * C::kBRows, C::kBRows, kb - half, bar);
        } else if (grad) {
          load_operand<false>(s, ma2, u.m0, kTile, kb + first, bar);
          load_operand<true>(s + 2 * kSlab, mb2, u.n0 + (int)rank * (C::kBRows / 2), C::kBRows / 2, kb + first, bar);
        } else {
          load_operand<C::kAMn>(s, ma, u.m0, kTile, kb, bar);
          if (C::kPair) {  // the gate's columns are the first CTA's rows of B, up's the second's
            load_operand<false>(s + 2 * kSlab, mb, (rank ? a.N : 0) + u.n0, C::kBRows, kb, bar);
          } else {
            load_operand<C::kBMn>(s + 2 * kSlab, mb, u.n0 + (int)rank * C::kBRows, C::kBRows, kb, bar);
          }
        }
      }
      __syncwarp();
    }
  }
out:
  // after an abort, copies may still be in flight (those of a pair count on the first CTA's barriers)
  if (lane == 0 && rank == 0)
    for (uint32_t j = n > C::kStages ? n - C::kStages : 0; j < n; ++j)
      bounded_drain(bars + kFull + j % C::kStages, (j / C::kStages) & 1, kWaitNs / 4);
  __syncwarp();
}

// ------------------------------------------------------------------ MMAs
template <bool MN>
__device__ __forceinline__ uint64_t operand(uint32_t addr) {
  return MN ? ptx::smem_desc_sw128(addr, kSlab, 1024) : ptx::smem_desc_sw128(addr, 16, 1024);
}
// the operand 16 values further along the summed axis
template <bool MN>
__device__ __forceinline__ uint64_t step(uint64_t desc, int k) {
  return ptx::smem_desc_at(desc, k * (MN ? 16 * 128 : 32));
}

template <bool AMN, bool BMN, int N>
__device__ __forceinline__ void block_mma(uint32_t acc, uint32_t s, bool fresh) {
  const uint32_t idesc = ptx::idesc_bf16_f32(2 * kTile, N, AMN, BMN);
  const uint64_t da = operand<AMN>(s), db = operand<BMN>(s + 2 * kSlab);
#pragma unroll
  for (int k = 0; k < kBK / 16; ++k) ptx::umma_pair<false>(acc, step<AMN>(da, k), step<BMN>(db, k), idesc, !fresh || k > 0);
}

template <DenseOp OP>
__device__ void issue(const DenseArgs& a, uint8_t* sm, uint64_t* bars, uint32_t tmem, volatile int* abort_flag) {
  using C = Cfg<OP>;
  const uint32_t s0 = ptx::smem_u32(sm);
  const bool el = ptx::elect_one();
  constexpr uint32_t rank = 0;  // the first CTA issues for both
  uint32_t n = 0, it = 0;
  for (Units<C::kTileN, DenseArgs> units(a, rank); units.left(); units.next(), ++it) {
    const Unit u = units.get();
    const uint32_t buf = it & 1, round = (it >> 1) & 1;
    if (!bounded_wait_warp(bars + kAccEmpty + buf, round ^ 1, abort_flag, a.status, kWaitNs)) goto out;
    ptx::tc_fence_after();
    if (OP == DenseOp::kDglu) {
      for (int kb = 0; kb < a.kblocks; ++kb, ++n) {
        const int st = n % C::kStages;
        if (!bounded_wait_warp(bars + kFull + st, (n / C::kStages) & 1, abort_flag, a.status, kWaitNs)) goto out;
        ptx::tc_fence_after();
        if (el) {
          block_mma<false, true, kBN / 2>(tmem + kBN + buf * (kBN / 2), s0 + st * C::kStage, kb == 0);
          ptx::umma_commit_pair(bars + kEmpty + st);
        }
        __syncwarp();
      }
      if (!bounded_wait_warp(bars + kGuEmpty, (it & 1) ^ 1, abort_flag, a.status, kWaitNs)) goto out;
      ptx::tc_fence_after();
    }
    const uint32_t acc = OP == DenseOp::kDglu ? tmem : tmem + buf * kBN;
    for (int kb = u.kb0; kb < u.kb1; ++kb, ++n) {
      const int st = n % C::kStages;
      if (!bounded_wait_warp(bars + kFull + st, (n / C::kStages) & 1, abort_flag, a.status, kWaitNs)) goto out;
      ptx::tc_fence_after();
      if (el) {
        block_mma<C::kAMn, C::kBMn, kBN>(acc, s0 + st * C::kStage, kb == u.kb0);
        ptx::umma_commit_pair(bars + kEmpty + st);
      }
      __syncwarp();
    }
    if (el) ptx::umma_commit_pair(bars + kAccFull + buf);
    __syncwarp();
  }
out:
  if (el) {
    ptx::umma_commit_pair(bars + kDone);
    bounded_drain(bars + kDone, 0, kWaitNs / 4);
  }
  __syncwarp();
}

// ------------------------------------------------------------------ epilogues
template <DenseOp OP, int ACT>
__device__ void finish(const DenseArgs& a, uint64_t* bars, uint32_t tmem, volatile int* abort_flag, uint32_t rank, int warp,
                       int lane) {
  using C = Cfg<OP>;
  const int quad = warp & 3, part = (warp - 4) >> 2;
  constexpr int kCols = C::kTileN * 4 / C::kEpiWarps;  // of the result, a warp's share
  constexpr int kStep = C::kPair ? 16 : 32;
  const uint32_t empty = ptx::first_of_pair(bars + kAccEmpty), gu_empty = ptx::first_of_pair(bars + kGuEmpty);
  uint32_t it = 0;
  for (Units<C::kTileN, DenseArgs> units(a, rank); units.left(); units.next(), ++it) {
    const Unit u = units.get();
    const uint32_t buf = it & 1, round = (it >> 1) & 1;
    if (!bounded_wait_warp(bars + kAccFull + buf, round, abort_flag, a.status, kWaitNs)) return;
    ptx::tc_fence_after();
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16) + part * kCols;
    long long row = u.m0 + quad * 32 + lane;
    if (OP == DenseOp::kDw && a.pad && row >= a.cut) row = row < a.cut + a.pad ? a.M : row - a.pad;  // (between: none)
    const auto give_back = [&](uint32_t bar) {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_pair(bar);
    };
    if constexpr (OP == DenseOp::kDglu) {
      // g and u of all of the warp's columns leave their only buffer at once, so that the next tile's can be
      // summed into it; dh, which has two, is read 16 columns at a time.
      uint32_t gu[64];
      ptx::tmem_ld2x32(lanes, lanes + kBN / 2, gu);
      give_back(gu_empty);
#pragma unroll
      for (int c = 0; c < kCols; c += 16) {
        uint32_t d[16], wg[8], wu[8], wh[8];
        ptx::tmem_ld16(lanes + kBN + buf * (kBN / 2) + c, d);
        if (c + 16 >= kCols) give_back(empty + 8 * buf);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const f32x2 dh = pair_of_bits(d[2 * e], d[2 * e + 1]), up = pair_of_bits(gu[32 + c + 2 * e], gu[33 + c + 2 * e]);
          f32x2 slope;
          const f32x2 act = act_both<ACT>(pair_of_bits(gu[c + 2 * e], gu[c + 2 * e + 1]), slope);
          wg[e] = pack_bf16(mul_pairs(mul_pairs(dh, up), slope));
          wu[e] = pack_bf16(mul_pairs(dh, act));
          wh[e] = pack_bf16(mul_pairs(act, up));
        }
        const int col = u.n0 + part * kCols + c, left = a.N - col;
        if (row < a.M && left > 0) {
          const int ld = a.N + a.pad;
          __nv_bfloat16* p = static_cast<__nv_bfloat16*>(a.out) + row * 2 * ld + col;
          store_bf16(p, wg, left, a.wide);
          store_bf16(p + ld, wu, left, a.wide);
          store_bf16(static_cast<__nv_bfloat16*>(a.out2) + row * ld + col, wh, left, a.wide);
        }
      }
      continue;
    }
#pragma unroll 1
    for (int c = 0; c < kCols; c += kStep) {
      const int col = u.n0 + part * kCols + c, left = a.N - col;
      const bool in = row < a.M && left > 0;
      if constexpr (OP == DenseOp::kGlu) {
        uint32_t gu[32], w[8];
        ptx::tmem_ld2x16(lanes + buf * kBN + c, lanes + buf * kBN + kBN / 2 + c, gu);
        if (c + kStep >= kCols) give_back(empty + 8 * buf);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          w[e] = pack_bf16(mul_pairs(act_value<ACT>(pair_of_bits(gu[2 * e], gu[2 * e + 1])),
                                     pair_of_bits(gu[16 + 2 * e], gu[17 + 2 * e])));
        if (in) store_bf16(static_cast<__nv_bfloat16*>(a.out) + row * (a.N + a.pad) + col, w, left, a.wide);
      } else {
        uint32_t r[32];
        ptx::tmem_ld32(lanes + buf * kBN + c, r);
        if (c + kStep >= kCols) give_back(empty + 8 * buf);
        if (a.splits > 1) {
          if (in) {
            float4* dst = reinterpret_cast<float4*>(a.part + ((long long)u.split * a.M + row) * a.N + col);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (4 * e < left)
                dst[e] = make_float4(__uint_as_float(r[4 * e]), __uint_as_float(r[4 * e + 1]),
                                     __uint_as_float(r[4 * e + 2]), __uint_as_float(r[4 * e + 3]));
          }
        } else {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = pack_bf16(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
          if (in) store_bf16(static_cast<__nv_bfloat16*>(a.out) + row * a.N + col, w, left, a.wide);
        }
      }
    }
  }
}

template <DenseOp OP, int ACT>
__global__ void __maxnreg__((Cfg<OP>::kRegs))
    k_dense(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
            const __grid_constant__ CUtensorMap ma2, const __grid_constant__ CUtensorMap mb2, const DenseArgs a) {
  using C = Cfg<OP>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kBars];
  __shared__ int s_abort;
  __shared__ uint32_t tmem_slot;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  volatile int* abort_flag = &s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      ptx::mbar_init(bars + kFull + i, 1);
      ptx::mbar_init(bars + kEmpty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bars + kAccFull + i, 1);
      ptx::mbar_init(bars + kAccEmpty + i, 2 * C::kEpiWarps);
    }
    ptx::mbar_init(bars + kGuEmpty, 2 * C::kEpiWarps);
    ptx::mbar_init(bars + kDone, 1);
    s_abort = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 1) ptx::tmem_alloc_pair(&tmem_slot, C::kTmem);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();  // both CTAs' barriers are there
  ptx::tc_fence_after();
  const uint32_t rank = ptx::cluster_rank();
  ptx::successor_may_start();
  if (a.follows) ptx::predecessor_done();
  const uint32_t tmem = tmem_slot;
  if (warp < 4) {
    if (C::kSplitRegs) ptx::fewer_registers<C::kFewRegs>();
    if (warp == 0) produce<OP>(a, &ma, &mb, &ma2, &mb2, sm, bars, abort_flag, rank, lane);
    else if (warp == 1 && rank == 0) issue<OP>(a, sm, bars, tmem, abort_flag);
  } else {
    if (C::kSplitRegs) ptx::more_registers<C::kSumRegs>();
    finish<OP, ACT>(a, bars, tmem, abort_flag, rank, warp, lane);
  }
  ptx::tc_fence_before();
  __syncthreads();
  // nothing of one CTA's reaches into the other any more, the last commit too
  if (warp == 1 && rank == 1 && lane == 0) bounded_drain(bars + kDone, 0, kWaitNs / 4);
  __syncwarp();
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, C::kTmem);
  }
}

// The parts' sums, in their order.
template <bool BF16>
__global__ void k_dense_sum(const float* part, void* out, long long n, int splits) {
  const long long i = ((long long)blockIdx.x * blockDim.x + threadIdx.x) * 4;
  ptx::successor_may_start();
  ptx::predecessor_done();
  if (i >= n) return;
  float4 s = *reinterpret_cast<const float4*>(part + i);
  for (int k = 1; k < splits; ++k) {
    const float4 v = *reinterpret_cast<const float4*>(part + k * n + i);
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  }
  if (BF16) reinterpret_cast<uint2*>(out)[i / 4] = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
  else reinterpret_cast<float4*>(out)[i / 4] = s;
}

template <DenseOp OP, int ACT>
cudaError_t run(const CUtensorMap (&m)[4], DenseArgs a, int num_sms, cudaStream_t st) {
  using C = Cfg<OP>;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(done, (const void*)k_dense<OP, ACT>, C::kDynamic);
  if (e != cudaSuccess) return e;
  static std::atomic<int> regs{0};
  if (C::kSplitRegs && !launched_with(regs, (const void*)k_dense<OP, ACT>, C::kRegs)) return cudaErrorInvalidConfiguration;
  a.tiles_m = (a.M + (OP == DenseOp::kDw ? a.pad : 0) + C::kTileM - 1) / C::kTileM;
  a.tiles_n = (a.N + C::kTileN - 1) / C::kTileN;
  const long long units = (long long)a.tiles_m * a.tiles_n * a.splits;
  const int places = num_sms / 2;
  return launch_pairs(2, a.follows != 0, k_dense<OP, ACT>, (int)(units < places ? units : places) * 2,
                      C::kThreads, C::kDynamic, st, m[0], m[1], m[2], m[3], a);
}

}  // namespace

bool encode_dense(CUtensorMap* m, const void* base, long long rows, long long cols, bool mn_major, long long ld) {
  return encode_map(m, base, rows, cols, mn_major ? 64 : kTile, ld);
}

// Asked once per device (the first call may be captured: the question belongs to no stream).
int* dense_status() {
  static std::atomic<int*> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return nullptr;
  if (dev < 64)
    if (int* w = known[dev].load(std::memory_order_relaxed)) return w;
  const OutsideCapture now;
  void* p = nullptr;
  if (cudaGetSymbolAddress(&p, g_dense_status) != cudaSuccess) return nullptr;
  if (dev < 64) known[dev].store(static_cast<int*>(p), std::memory_order_relaxed);
  return static_cast<int*>(p);
}

// The parts that take the least time: rounds of the pairs of SMs times a part's blocks, and the parts' sums
// written and read.
int dense_splits(int M, int N, int kblocks, double block_us, int num_sms) {
  const long long tiles = (long long)((M + 255) / 256) * ((N + 255) / 256), places = num_sms / 2;
  int best = 1;
  double least = 1e300;
  for (int s = 1; s <= 64 && s <= kblocks; ++s) {
    const long long rounds = (tiles * s + places - 1) / places;
    const double us = rounds * (block_us * ((kblocks + s - 1) / s) + 1) + (s > 1 ? s * 8e-6 / 5 * M * N + 3 : 0);
    if (us < least) {
      least = us;
      best = s;
    }
  }
  return best;
}

cudaError_t launch_dense_sum(const float* part, void* out, long long n, int splits, int dtype, cudaStream_t st) {
  const unsigned blocks = (unsigned)((n / 4 + 255) / 256);
  return launch_pairs(1, true, dtype == REC_ATTN_BF16 ? k_dense_sum<true> : k_dense_sum<false>, (int)blocks, 256, 0, st, part,
                      out, n, splits);
}

cudaError_t launch_dense(DenseOp op, const CUtensorMap (&m)[4], DenseArgs a, int num_sms, cudaStream_t st) {
  switch (op) {
    case DenseOp::kGlu:
      return a.act == REC_ATTN_SILU ? run<DenseOp::kGlu, REC_ATTN_SILU>(m, a, num_sms, st)
                                    : run<DenseOp::kGlu, REC_ATTN_GELU>(m, a, num_sms, st);
    case DenseOp::kDglu:
      return a.act == REC_ATTN_SILU ? run<DenseOp::kDglu, REC_ATTN_SILU>(m, a, num_sms, st)
                                    : run<DenseOp::kDglu, REC_ATTN_GELU>(m, a, num_sms, st);
    case DenseOp::kOut: return run<DenseOp::kOut, 0>(m, a, num_sms, st);
    case DenseOp::kDx: return run<DenseOp::kDx, 0>(m, a, num_sms, st);
    case DenseOp::kDw: return run<DenseOp::kDw, 0>(m, a, num_sms, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace recattn
