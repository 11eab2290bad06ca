// attn_bwd_tc.cu -- backward pass of the masked time-RoPE attention on the sm_103a
// tensor cores (bf16 inputs and gradients, fp32 accumulation, head_dim 64 or 128).
//
// Gradients of O = Softmax(QK^T/sqrt(d) + M) V (TM20K review page, section 2.1;
// LazFormer review page, Eq. 19-21) through the time-RoPE (CADET review page, time
// encoding).  With P rebuilt from the forward's log-sum-exp, P_ij = exp(s_ij - lse_i)
// on visible pairs, D_i = <dO_i, O_i> and dS_ij = P_ij (dP_ij - D_i):
//   mode DQ:   dQ'_i = scale sum_j dS_ij K'_j
//   mode DKV:  dV_j = sum_i P_ij dO_i,  dK'_j = scale sum_i dS_ij Q'_i
// and dQ = R(t_i)^T dQ', dK = R(t_j)^T dK' (the rotation is orthogonal).
//
// Both modes share one persistent kernel shape: one CTA per SM with all 512 TMEM columns and 19
// warps.  Warp 0 loads with TMA; warps 1 and 2 issue the MMAs; sixteen compute warps (four
// warpgroups) hold one tile row per thread (its TMEM lane) and 32 of a step's 128 columns each.
// The producer claims the planner's (tile, head) items from a global counter and publishes each
// item's descriptor in shared memory for the other roles; mode DKV visits key tiles in the mirrored
// order of the query tiles, so under causal masks both modes start with their heaviest items.  Per
// item the resident operand pair stays in shared memory (DQ: Q', dO; DKV: K', V) and the streamed
// pair (DQ: K', V of the query tile's non-SKIP key tiles; DKV: Q', dO of the query tiles whose class
// against the key tile is not SKIP) runs through two rings; at head_dim 64 there is room for two
// resident pairs, and the next item's loads while this one runs (1% on items of a few tiles).  A step
// is a whole streamed tile:
//   DQ   S = Q' K'^T - lse / scale, dP = dO V^T - D; the compute warps write dS (bf16) over the
//        first half of the 32 columns of S that each has read; dQ += dS K' with dS read from TMEM.
//   DKV  S^T = K' Q'^T - lse / scale, dP^T = V dO^T - D; P^T over the first half of S's columns,
//        dS^T over the second; dV += P^T dO, dK += dS^T Q'.  (head_dim 128: dS^T over dP^T.)
// The queries' constants enter as one more K step of 16 (constants x ones in DQ, ones x constants in
// DKV), each split into three bf16 that add up to its 24 bits: the compute warps then take P =
// exp2(scale log2(e) S) and dS = P dP from the products as they are.  In DKV, where the queries are
// the columns, reading the constants from shared memory instead cost more of its bandwidth than the
// scores' operands.
// TMEM columns:  head_dim 64   S[0] 0..127 | S[1] 128..255 | dP 256..383 | dQ or dV 384.. | dK 448..
//                head_dim 128  S[0] 0..127 | dP 128..255 | dQ or dV 256.. | DQ: S[1], DKV: dK 384..
// With two buffers of S the next step's scores are issued during this step's compute: S when the
// accumulation of the step before last has read its operands, dP when the compute warps have loaded
// this step's; and warp 1 issues the scores while warp 2 issues the accumulation (one warp for both
// spent 700 of a step's 2400 cycles in waits for what was already there).  With one buffer (DKV at
// head_dim 128) warp 1 issues everything in turns: S behind dV, dP behind dK, each pair running under
// the compute of the other.
// What bounds it: a step's products take 1370 (DKV) and 1010 (DQ) tensor cycles at head_dim 64, 2200
// and 1680 at 128, its exponentials 512 of the special-function unit; a step takes 1980, 1610, 3500
// and 2750, the difference being the chain score - exponential - operand - sum between barriers, of
// which one step (two with two S) is under way.  Sixteen ragged requests of 603 to 1850 tokens,
// head_dim 128, 8 query and 2 key/value heads: dQ 133 us, dK/dV 174 us (two 64-column steps at a time
// with two compute warpgroups: 170 and 231); two causal ones of 8192 and 7000 tokens, head_dim 64, 8
// and 1 heads: 164 and 213 us (two such CTAs per SM: 470 in all).  Also slower there: 64-column steps
// of two groups of eight warps in turn (307 and 385).
// The accumulators stay in TMEM across an item's tiles; the epilogue scales, undoes the rotation and
// writes bf16 rows.  The rest a compute thread needs comes through shared memory with the tiles: the
// planner's record of the item's tile and the masks.  FULL tiles take no mask.  PARTIAL pairs
// with a slot in the plan's mask table read its rows (DQ) or columns (DKV; transposed once per plan by
// k_bwd_colmask), bulk-copied with the streamed tile; others the forward's per-row visibility bits
// (row_mask.cuh), built from the key tile's record, in DKV by threads that act as rows of the
// query tile, whose warps transpose the bits into per-key columns with shuffles.  The MMAs of one
// thread run in issue order, so an MMA that overwrites TMEM columns an earlier MMA of it reads needs
// no wait.  Every mbarrier wait is bounded (REC_ATTN_ERR_TIMEOUT in the status word).
//
// Rounded to bf16 on the way, as the products' operands: Q' and K' (rope.cu), P and dS; and D_i takes O as
// the forward wrote it (an fp32 copy of O would be another 4 H d bytes a token, written and read).
// dQ, dK and dV are off by 2.5e-3 to 3.1e-3 (relative, against 64 bits), where their last rounding alone
// gives 1.7e-3.  Sums, P before its rounding and the rows' constants are fp32.
#include <cuda_bf16.h>

#include "attn_common.cuh"
#include "launchers.cuh"
#include "ptx_sm103.cuh"
#include "row_mask.cuh"
#include "wait.cuh"

namespace recattn {

namespace {

constexpr int kSlab = kTile * 128;          // 128 rows x 64 bf16 columns, 128-byte swizzled
// Per head dimension: a [128][D] bf16 tile is D / 64 slabs.
template <int D>
struct BCfg {
  static constexpr int kTileBytes = kTile * D * 2;
  // stages of the streamed rings (first and second operand)
  template <bool DKV>
  static constexpr int kNS0 = D == 64 ? 3 : DKV ? 2 : 3;
  template <bool DKV>
  static constexpr int kNS1 = D == 64 ? 3 : DKV ? 2 : 1;
  // resident pairs in shared memory: at head_dim 64 the next item's loads while this one runs
  static constexpr int kRB = D == 64 ? 2 : 1;
  static constexpr int kWG = 4;                   // compute warpgroups, 32 of a step's 128 columns each
  static constexpr int kRoles = 3;                // producer, one or two issuers
  static constexpr int kThreads = 32 * kRoles + 128 * kWG;
  // TMEM columns of S (step parity b), dP and the accumulators
  template <bool DKV>
  __host__ __device__ static constexpr uint32_t s_col(uint32_t b) {
    return D == 64 ? b * 128 : (DKV ? 0u : b * 384);
  }
  static constexpr uint32_t kDP = D == 64 ? 256 : 128;
  static constexpr uint32_t kDQ = D == 64 ? 384 : 256, kDV = kDQ, kDK = kDV + D;
  // whether S has two buffers (head_dim 128 leaves DKV none)
  template <bool DKV>
  static constexpr bool kTwoS = D == 64 || !DKV;
};
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kChunkCols = 32;         // a step's bf16 operand: each warpgroup's 16 columns of packed pairs
                                            // (two K steps) over the first half of the 32 columns it has read
constexpr uint32_t kDsCols = 16;            // DKV with two S: dS^T stands over the second half, beside P^T
constexpr int kRecB = (int)sizeof(KeyTileRec);
constexpr int kMaskB = kTile * 16;  // a PARTIAL pair's 128 rows (or columns) of the mask table
constexpr int kStageRecB = kMaskB > kRecB ? kMaskB : kRecB;  // per streamed stage: one or the other
constexpr uint64_t kWaitNsB = 2000000000ull;  // 2 s
constexpr float kLog2e = 1.4426950408889634f;

// mbarriers (steps are counted over the CTA's life; [2]: by step parity)
enum : int {
  kResFull = 0,                 // [kRB]
  kResEmpty = kResFull + 2,     // [kRB]
  kStr0Full = kResEmpty + 2,    // [4] the streamed tile of the scores S (DQ: K', DKV: Q'), with the record
  kStr0Empty = kStr0Full + 4,   // [4] and the row constants
  kStr1Full = kStr0Empty + 4,   // [4] the streamed tile of dP (DQ: V, DKV: dO)
  kStr1Empty = kStr1Full + 4,   // [4]
  kSFull = kStr1Empty + 4,      // [2] S completed
  kDpFull = kSFull + 2,         // dP completed
  kDpFree,                      // DQ: the compute warps loaded dP
  kPReady,                      // [2] DQ: the compute warps wrote dS; DKV: P^T (the next step's may be
                                // written before the issuer looks for this one's)
  kDsReady = kPReady + 2,       // DKV, one S: the compute warps wrote dS^T
  kSFree,                       // [2] two S: the accumulation read the step's operand in S's columns
  kAccFull = kSFree + 2,        // the item's last accumulating MMA completed
  kAccEmpty,                    // the compute warps read the accumulators
  kGroup,                       // DKV: barrier of the compute threads
  kItemFull,                    // [2] the producer published an item descriptor
  kItemEmpty = kItemFull + 2,   // [2] the MMA issuer and the compute warps copied it
  kMmaDone = kItemEmpty + 2,    // [2] an issuing warp's MMAs are done, at the end
  kNumBars = kMmaDone + 2
};
// wait parity of step `step` on a barrier of its own and on one of two
__host__ __device__ constexpr uint32_t par1(uint32_t step) { return step & 1u; }
__host__ __device__ constexpr uint32_t par2(uint32_t step) { return (step >> 1) & 1u; }

// Byte offsets from the 1024-aligned base of dynamic shared memory.
constexpr int kRowX = kTile * 16;    // a tile's rows of the constants' operand, 8 bf16 each
constexpr int kAugB = 2 * kRowX;     // an operand of 16 columns: two 8-column halves, the second zero
template <int D>
struct BL {
  static constexpr int kRB = BCfg<D>::kRB;
  static constexpr int kTiles = D == 64 ? 6 : 4;             // streamed tiles: kNS0 + kNS1 of both modes
  static constexpr int kRecs = 3;                            // at least kNS0 of both modes,
  static constexpr int kAugs = BCfg<D>::template kNS0<true>; // of DKV (and at least kRB)
  static constexpr int kTileBytes = BCfg<D>::kTileBytes;
  static constexpr int kOnes = 0;                            // [2 (S, dP)] ones that pick the constants
  static constexpr int kAug = kOnes + 2 * kAugB;              // constants of the query tiles (DKV: [kNS0]; DQ: [kRB])
  static constexpr int kRes = kAug + kAugs * kAugB;           // [kRB][2] resident tiles
  static constexpr int kStr = kRes + kRB * 2 * kTileBytes;         // the streamed tiles, [kNS0] first operands, then [kNS1]
  static constexpr int kSRec = kStr + kTiles * kTileBytes;  // [kNS0] records of the streamed tiles
  static constexpr int kRRec = kSRec + kRecs * kStageRecB;   // [kRB] record of the item's tile
  static constexpr int kCol = kRRec + kRB * kRecB;                 // DKV: [2][128 keys] 128 query bits
  static constexpr int kItems = kCol + 2 * kTile * 16;       // [2] published item descriptors
  static constexpr int kBarsOff = kItems + 2 * 64;
  static constexpr int kTotal = kBarsOff + kNumBars * 8 + 16;  // + abort flag and TMEM slot
  static constexpr int kDynamic = kTotal + 1024;               // slack to align the base
};
template <int D>
constexpr bool layout_ok() {
  using L = BL<D>;
  return L::kAugs >= L::kRB && L::kRes % 1024 == 0 && L::kStr % 1024 == 0 && L::kSRec % 16 == 0 && L::kRRec % 16 == 0 &&
         L::kCol % 16 == 0 && L::kBarsOff % 8 == 0 && L::kDynamic <= 227 * 1024 &&
         BCfg<D>::template kNS0<true> + BCfg<D>::template kNS1<true> <= L::kTiles && BCfg<D>::template kNS0<true> <= L::kRecs &&
         BCfg<D>::template kNS0<false> + BCfg<D>::template kNS1<false> <= L::kTiles && BCfg<D>::template kNS0<false> <= L::kRecs;
}
static_assert(layout_ok<64>() && layout_ok<128>(), "shared memory layout");

__device__ __forceinline__ bool bw_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  return bounded_wait(bar, parity, abort_flag, status, kWaitNsB);
}
__device__ __forceinline__ bool bw_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                             int* status) {
  return bounded_wait_warp(bar, parity, abort_flag, status, kWaitNsB);
}
// The compute warps' barriers by their shared-memory address (32 bits: a step has few instructions).
struct WarpBars {
  uint32_t base;
  uint64_t* bars;
  volatile int* abort_flag;
  int* status;
  __device__ __forceinline__ bool wait(int bar, uint32_t parity) const {
    const bool ok = ptx::mbar_try_wait_at(base + 8 * bar, parity);
    if (__all_sync(0xffffffffu, ok)) return true;
    return bw_wait_warp(bars + bar, parity, abort_flag, status);
  }
  __device__ __forceinline__ void arrive(int bar) const {  // one arrival for the warp
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive_at(base + 8 * bar);
  }
};
__device__ __forceinline__ void bw_drain(uint64_t* bar, uint32_t parity) {
  bounded_drain(bar, parity, kWaitNsB / 4);
}

// A published item: its descriptor (as three 16-byte words) and the end flag.
struct ItemSlot {
  uint4 d[3];
  int end;
  int pad[3];
};
static_assert(sizeof(ItemSlot) == 64, "");

__device__ __forceinline__ BwdItemDesc unpack_desc(const uint4 (&nx)[3]) {
  BwdItemDesc d;
  d.tok_start = (long long)(((unsigned long long)nx[0].y << 32) | nx[0].x);
  d.t_ref = (long long)(((unsigned long long)nx[0].w << 32) | nx[0].z);
  d.list = (long long)(((unsigned long long)nx[1].y << 32) | nx[1].x);
  d.len = (int)nx[1].z;
  d.tile = (int)nx[1].w;
  d.tile_start = (int)nx[2].x;
  d.h = (int)nx[2].y;
  d.n = (int)nx[2].z;
  d.pad = 0;
  return d;
}

// Consumer side of the item slots (whole warps): the next item's descriptor, or false at the end
// (or after an abort).
template <int D>
__device__ __forceinline__ bool next_item(uint8_t* sm, uint64_t* bars, uint32_t& it_cnt, BwdItemDesc& d,
                                          volatile int* abort_flag, int* status) {
  const int slot = (int)(it_cnt & 1);
  const uint32_t ph = (it_cnt >> 1) & 1;
  ++it_cnt;
  if (!bw_wait_warp(bars + kItemFull + slot, ph, abort_flag, status)) return false;
  const ItemSlot* is = reinterpret_cast<const ItemSlot*>(sm + BL<D>::kItems) + slot;
  const uint4 nx[3] = {is->d[0], is->d[1], is->d[2]};
  const int end = is->end;
  __syncwarp();
  if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(bars + kItemEmpty + slot);
  if (end) return false;
  d = unpack_desc(nx);
  return true;
}

// The streamed tiles of an item, in order: request-local tile index, class and
// mask-table slot (-1: none).  DKV visits each listed query tile once for every query
// head of the item's part of the group (`reps` times in a row), so dK and dV sum over those
// heads in TMEM.
template <bool DKV>
struct Cursor {
  long long at;
  int rep, reps;
  __device__ __forceinline__ void init(const BwdItemDesc& d, int n_rep) {
    at = d.list;
    rep = 0;
    reps = n_rep;
  }
  // The entry as loaded, so that a caller may fetch it ahead without waiting for it.
  struct Entry {
    uint32_t e;
    int slot;
    __device__ __forceinline__ int tile() const { return (int)(e & 0xffffffu); }
    __device__ __forceinline__ int cls() const { return (int)(e >> 24); }
  };
  __device__ __forceinline__ Entry next(const BwdArgs& a) {
    Entry x;
    x.e = (DKV ? a.qlist : a.klist)[at];
    x.slot = (DKV ? a.qslot : a.kslot)[at];
    if (!DKV || ++rep == reps) {
      rep = 0;
      ++at;
    }
    return x;
  }
};

// The same for the compute warps, which need to know little of most tiles: lane i holds the i-th of 32
// entries, and one bit of each says whether the tile is FULL.  (One entry loaded ahead for every
// step cost 185 cycles of a step of 2100: address arithmetic and a queue for the load.)
template <bool DKV>
struct WarpCursor {
  long long at;
  uint32_t e, full;
  int slot, r, rep, left;
  __device__ __forceinline__ void load(const BwdArgs& a) {
    const int lane = threadIdx.x & 31;
    const bool in = lane < left;
    e = in ? (DKV ? a.qlist : a.klist)[at + lane] : 0u;  // (class 0 is not FULL)
    slot = in ? (DKV ? a.qslot : a.kslot)[at + lane] : -1;
    at += 32;
    left -= 32;
    r = 0;
  }
  __device__ __forceinline__ void vote() {
    full = __ballot_sync(0xffffffffu, (e >> 24) == (uint32_t)REC_ATTN_TILE_FULL);
  }
  // init starts the first loads; vote() once, before the first step
  __device__ __forceinline__ void init(const BwdArgs& a, const BwdItemDesc& d, int entries) {
    at = d.list;
    left = entries;
    rep = 0;
    load(a);
  }
  __device__ __forceinline__ bool is_full() const { return (full >> r) & 1u; }
  __device__ __forceinline__ int tile() const { return (int)(__shfl_sync(0xffffffffu, e, r) & 0xffffffu); }
  __device__ __forceinline__ int table_slot() const { return __shfl_sync(0xffffffffu, slot, r); }
  __device__ __forceinline__ void next(const BwdArgs& a, int reps) {
    if (DKV && ++rep < reps) return;
    rep = 0;
    if (++r == 32 && left > 0) {
      load(a);
      vote();
    }
  }
};

// ------------------------------------------------------------------ producer
// maps: resident pair res[0], res[1]; streamed pair str[0], str[1].
//   DQ:  resident Q', dO + the query tile's record and row constants; streamed K' (+ the key
//        tile's record or mask rows when the tile is PARTIAL) and V.
//   DKV: resident K', V + the key tile's record; streamed Q' + the query tile's record and its
//        constants' operand, and dO.
// The two streamed tiles have rings of their own: the second is free again as soon as dP (DQ) or
// dV (DKV) has read it, the first after dQ or dK, the step's last MMA.
template <int D, bool DKV>
__device__ void bwd_producer(const BwdArgs& a, const void* const (&res)[2], const void* const (&str)[2],
                             uint8_t* sm, uint64_t* bars, volatile int* abort_flag) {
  using L = BL<D>;
  constexpr int kTileBytes = L::kTileBytes, kNS0 = BCfg<D>::template kNS0<DKV>, kNS1 = BCfg<D>::template kNS1<DKV>;
  uint32_t it_n = 0, s_it = 0, it_cnt = 0;
  uint32_t n0 = 0, n1 = 0;  // steps whose first, second operand was loaded
  const uint4* descs = reinterpret_cast<const uint4*>(a.desc + (DKV ? a.n_items : 0));
  ItemSlot* slots = reinterpret_cast<ItemSlot*>(sm + L::kItems);
  int* counter = a.counters + (DKV ? 5 : 3);
  const long long n_items = DKV ? a.n_kv_items : a.n_items;
  for (;;) {
    const long long w = atomicAdd(counter, 1);
    const int slot = (int)(it_cnt & 1);
    if (!bw_wait(bars + kItemEmpty + slot, ((it_cnt >> 1) & 1) ^ 1, abort_flag, a.status)) goto drain;
    ++it_cnt;
    if (w >= n_items) {
      slots[slot].end = 1;
      ptx::mbar_arrive(bars + kItemFull + slot);
      break;
    }
    uint4 nx[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) nx[k] = descs[3 * w + k];
#pragma unroll
    for (int k = 0; k < 3; ++k) slots[slot].d[k] = nx[k];
    slots[slot].end = 0;
    ptx::mbar_arrive(bars + kItemFull + slot);  // release: the slot's contents reach the waiters
    const BwdItemDesc d = unpack_desc(nx);
    if (d.n <= 0) continue;

    const int rb = (int)(it_n % L::kRB);
    if (!bw_wait(bars + kResEmpty + rb, ((it_n / L::kRB) & 1) ^ 1, abort_flag, a.status)) goto drain;
    {
      uint64_t* const res_full = bars + kResFull + rb;
      uint8_t* const res_at = sm + L::kRes + rb * 2 * kTileBytes;
      const int x = (DKV ? d.h / a.parts : d.h) * D;
      const long long g = (long long)d.tile_start + d.tile;
      ptx::mbar_arrive_expect_tx(res_full, 2 * kTileBytes + kRecB + (DKV ? 0 : kRowX));
      const int y = (int)(d.tok_start + (long long)d.tile * kTile);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        ptx::tma_load_2d(res_at + c * kSlab, res[0], x + 64 * c, y, res_full);
        ptx::tma_load_2d(res_at + kTileBytes + c * kSlab, res[1], x + 64 * c, y, res_full);
      }
      ptx::bulk_load(sm + L::kRRec + rb * kRecB, a.krec + g, kRecB, res_full);
      if (!DKV)
        ptx::bulk_load(sm + L::kAug + rb * kAugB, a.rowx + ((long long)d.h * a.n_tiles + g) * kTile, kRowX, res_full);
      ++it_n;
      Cursor<DKV> cur;
      const int reps = DKV ? a.group / a.parts : 1;
      cur.init(d, reps);
      const int kvx = (d.h / a.group) * D;  // DQ: the columns of the head's key/value head
      for (int j = 0; j < d.n; ++j, ++s_it) {
        // DKV: the query head of this visit, its columns and its row constants
        const int hq = d.h * reps + cur.rep;
        const int xs = DKV ? hq * D : kvx;
        const auto x_at = cur.next(a);
        const int tile = x_at.tile(), cls = x_at.cls(), tslot = x_at.slot;
        const int st = (int)(s_it % kNS0), st1 = (int)(s_it % kNS1);
        const long long gs = (long long)d.tile_start + tile;
        const int ys = (int)(d.tok_start + (long long)tile * kTile);
        auto load1 = [&]() -> bool {
          if (!bw_wait(bars + kStr1Empty + st1, ((s_it / kNS1) & 1) ^ 1, abort_flag, a.status)) return false;
          ptx::mbar_arrive_expect_tx(bars + kStr1Full + st1, kTileBytes);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            ptx::tma_load_2d(sm + L::kStr + (kNS0 + st1) * kTileBytes + c * kSlab, str[1], xs + 64 * c, ys,
                             bars + kStr1Full + st1);
          ++n1;
          return true;
        };
        // the operand whose place is free earlier goes first
        constexpr bool kSecondFirst = kNS1 >= kNS0;
        if (kSecondFirst && !load1()) goto drain;
        if (!bw_wait(bars + kStr0Empty + st, ((s_it / kNS0) & 1) ^ 1, abort_flag, a.status)) goto drain;
        // PARTIAL tiles with a mask-table slot: the tile's rows (DQ) or columns (DKV) of the
        // table; otherwise the key (DQ) or query (DKV) tile's record
        const bool part = cls != REC_ATTN_TILE_FULL, tab = part && tslot >= 0, rec = part && !tab;
        ptx::mbar_arrive_expect_tx(bars + kStr0Full + st,
                                   kTileBytes + (tab ? kMaskB : rec ? kRecB : 0) + (DKV ? kRowX : 0));
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          ptx::tma_load_2d(sm + L::kStr + st * kTileBytes + c * kSlab, str[0], xs + 64 * c, ys,
                           bars + kStr0Full + st);
        if (tab)
          ptx::bulk_load(sm + L::kSRec + st * kStageRecB, (DKV ? a.ctab : a.mtab) + (long long)tslot * (kMaskB / 4),
                         kMaskB, bars + kStr0Full + st);
        else if (rec)
          ptx::bulk_load(sm + L::kSRec + st * kStageRecB, a.krec + gs, kRecB, bars + kStr0Full + st);
        if (DKV)
          ptx::bulk_load(sm + L::kAug + st * kAugB, a.rowx + ((long long)hq * a.n_tiles + gs) * kTile, kRowX,
                         bars + kStr0Full + st);
        ++n0;
        if (!kSecondFirst && !load1()) goto drain;
      }
    }
  }
drain:
  // every copy issued must land before the CTA exits (only waits after an abort): the rings' last ones
  for (uint32_t u = it_n > L::kRB ? it_n - L::kRB : 0; u < it_n; ++u)
    bw_drain(bars + kResFull + u % L::kRB, (u / L::kRB) & 1);
  for (uint32_t u = n0 > kNS0 ? n0 - kNS0 : 0; u < n0; ++u) bw_drain(bars + kStr0Full + u % kNS0, (u / kNS0) & 1);
  for (uint32_t u = n1 > kNS1 ? n1 - kNS1 : 0; u < n1; ++u) bw_drain(bars + kStr1Full + u % kNS1, (u / kNS1) & 1);
}

// ------------------------------------------------------------------ MMA issuer
__device__ __forceinline__ uint64_t kdesc(uint32_t addr) { return ptx::smem_desc_sw128(addr, 16, 1024); }
// MN-major operand: 64-column blocks of N one slab apart
__device__ __forceinline__ uint64_t mndesc(uint32_t addr) { return ptx::smem_desc_sw128(addr, kSlab, 1024); }

// Scores of a whole tile over K = D (both operands K-major, the K steps of 16 columns four per slab).
template <int D>
__device__ __forceinline__ void mma_scores(uint32_t d, uint32_t a_addr, uint32_t b_addr) {
  constexpr uint32_t id = ptx::idesc_bf16_f32(kTile, kTile, false, false);
  const uint64_t da = kdesc(a_addr), db = kdesc(b_addr);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = (kk >> 2) * kSlab + (kk & 3) * 32;
    ptx::umma_f16(d, ptx::smem_desc_at(da, off), ptx::smem_desc_at(db, off), id, kk > 0);
  }
}
// The constants of the queries added to scores, one more K step: ones x constants (DKV: the queries are
// the columns) or constants x ones (DQ: the rows).
__device__ __forceinline__ void mma_consts(uint32_t d, uint32_t a_addr, uint32_t b_addr) {
  constexpr uint32_t id = ptx::idesc_bf16_f32(kTile, kTile, false, false);
  ptx::umma_f16(d, ptx::smem_desc_plain(a_addr, kRowX, 128), ptx::smem_desc_plain(b_addr, kRowX, 128), id, 1u);
}
// D (+)= A B with A (128 x 128, bf16) in TMEM and the tile's 128 rows as the K dimension
// (MN-major: the tile's D columns are N).
template <int D>
__device__ __forceinline__ void mma_acc(uint32_t d, uint32_t a_tmem, uint32_t b_rows, bool accumulate) {
  constexpr uint32_t id = ptx::idesc_bf16_f32(kTile, D, false, true);
  const uint64_t db = mndesc(b_rows);
#pragma unroll
  for (int kk = 0; kk < kTile / 16; ++kk)
    ptx::umma_f16_ts(d, a_tmem + (kk >> 1) * kChunkCols + (kk & 1) * 8, ptx::smem_desc_at(db, kk * 16 * 128), id,
                     (accumulate || kk > 0) ? 1u : 0u);
}

// What the issuing warps share: addresses, the barriers they wait for, and the MMAs of a step.
template <int D, bool DKV>
struct Issuer {
  using L = BL<D>;
  using C = BCfg<D>;
  static constexpr int kNS0 = C::template kNS0<DKV>, kNS1 = C::template kNS1<DKV>;
  uint8_t* sm;
  uint64_t* bars;
  volatile int* abort_flag;
  int* status;
  uint32_t res0, str0, str1, aug, ones, tmem;
  uint32_t rb = 0;  // the item's resident buffer
  bool el;  // this lane issues for the warp
  __device__ __forceinline__ Issuer(const BwdArgs& a, uint8_t* smem, uint64_t* b, uint32_t tmem_base, volatile int* ab)
      : sm(smem), bars(b), abort_flag(ab), status(a.status), res0(ptx::smem_u32(smem + L::kRes)),
        str0(ptx::smem_u32(smem + L::kStr)), str1(str0 + kNS0 * L::kTileBytes), aug(ptx::smem_u32(smem + L::kAug)),
        ones(ptx::smem_u32(smem + L::kOnes)), tmem(__shfl_sync(0xffffffffu, tmem_base, 0)), el(ptx::elect_one()) {}
  __device__ __forceinline__ bool ready(int bar, uint32_t parity) const {
    if (!bw_wait_warp(bars + bar, parity, abort_flag, status)) return false;
    ptx::tc_fence_after();
    return true;
  }
  // the it-th item's resident pair
  __device__ __forceinline__ bool resident(uint32_t it) {
    rb = __shfl_sync(0xffffffffu, it % L::kRB, 0);
    return ready(kResFull + (int)rb, (it / L::kRB) & 1);
  }
  __device__ __forceinline__ uint32_t res_at() const { return res0 + rb * 2 * L::kTileBytes; }
  // step s's operands are there, and its S and dP
  __device__ __forceinline__ bool full0(uint32_t s) const { return ready(kStr0Full + (int)(s % kNS0), (s / kNS0) & 1); }
  __device__ __forceinline__ bool full1(uint32_t s) const { return ready(kStr1Full + (int)(s % kNS1), (s / kNS1) & 1); }
  __device__ __forceinline__ uint32_t op0(uint32_t s) const { return str0 + (s % kNS0) * L::kTileBytes; }
  __device__ __forceinline__ uint32_t op1(uint32_t s) const { return str1 + (s % kNS1) * L::kTileBytes; }
  __device__ __forceinline__ uint32_t s_at(uint32_t s) const { return tmem + C::template s_col<DKV>(s & 1); }
  __device__ __forceinline__ void scores_s(uint32_t s) const {
    if (el) {
      mma_scores<D>(s_at(s), res_at(), op0(s));
      if constexpr (DKV) mma_consts(s_at(s), ones, aug + (s % kNS0) * kAugB);
      else mma_consts(s_at(s), aug + rb * kAugB, ones);
      ptx::umma_commit(bars + kSFull + (s & 1));
    }
    __syncwarp();
  }
  __device__ __forceinline__ void scores_dp(uint32_t s, bool last) const {
    if (el) {
      mma_scores<D>(tmem + C::kDP, res_at() + L::kTileBytes, op1(s));
      if constexpr (DKV) mma_consts(tmem + C::kDP, ones + kAugB, aug + (s % kNS0) * kAugB);
      else mma_consts(tmem + C::kDP, aug + rb * kAugB, ones + kAugB);
      ptx::umma_commit(bars + kDpFull);
      if constexpr (!DKV) ptx::umma_commit(bars + kStr1Empty + s % kNS1);
      if (last) ptx::umma_commit(bars + kResEmpty + rb);  // the resident pair read for the last time
    }
    __syncwarp();
  }
  // all MMAs this warp issued must complete before TMEM is released
  __device__ __forceinline__ void finish(int bar) const {
    if (el) ptx::umma_commit(bars + bar);
    __syncwarp();
    bw_drain(bars + bar, 0);
  }
};

// Two S buffers: one warp issues the scores and another the accumulation, so that neither's waits
// (over 100 cycles each, even for what is there: the MMAs' operands take the shared memory) leave the
// tensor core idle.
template <int D, bool DKV>
__device__ void bwd_issue_scores(const BwdArgs& a, uint8_t* sm, uint64_t* bars, uint32_t tmem_base,
                                 volatile int* abort_flag) {
  Issuer<D, DKV> q(a, sm, bars, tmem_base, abort_flag);
  uint32_t it_n = 0, step = 0, it_cnt = 0;
  BwdItemDesc it;
  while (next_item<D>(sm, bars, it_cnt, it, abort_flag, a.status)) {
    const int n = __shfl_sync(0xffffffffu, it.n, 0);
    if (n <= 0) continue;
    if (!q.resident(it_n++)) goto out;
    for (int j = 0; j < n; ++j, ++step) {
      const uint32_t s = __shfl_sync(0xffffffffu, step, 0);
      // S's buffer: free when the accumulation of the step before last has read it
      if (s >= 2 && !q.ready(kSFree + (int)(s & 1), par2(s - 2))) goto out;
      if (!q.full0(s)) goto out;
      q.scores_s(s);
      if (s >= 1 && !q.ready(kDpFree, par1(s - 1))) goto out;
      if (!q.full1(s)) goto out;
      q.scores_dp(s, j == n - 1);
    }
  }
out:
  q.finish(kMmaDone);
}
template <int D, bool DKV>
__device__ void bwd_issue_acc(const BwdArgs& a, uint8_t* sm, uint64_t* bars, uint32_t tmem_base, volatile int* abort_flag) {
  using C = BCfg<D>;
  const Issuer<D, DKV> q(a, sm, bars, tmem_base, abort_flag);
  uint32_t it_n = 0, step = 0, it_cnt = 0;
  BwdItemDesc it;
  while (next_item<D>(sm, bars, it_cnt, it, abort_flag, a.status)) {
    const int n = __shfl_sync(0xffffffffu, it.n, 0);
    if (n <= 0) continue;
    for (int j = 0; j < n; ++j, ++step) {
      const uint32_t s = __shfl_sync(0xffffffffu, step, 0);
      if (!q.ready(kPReady + (int)(s & 1), par2(s))) goto out;
      // the item's first MMA overwrites the accumulators: the compute warps must have read the last item's
      if (j == 0 && it_n > 0 && !q.ready(kAccEmpty, (it_n - 1) & 1)) goto out;
      if (q.el) {
        // (the step's scores are complete too: the compute warps have read them)
        if constexpr (DKV) {
          mma_acc<D>(q.tmem + C::kDV, q.s_at(s), q.op1(s), j > 0);  // dV += P^T dO
          ptx::umma_commit(bars + kStr1Empty + s % q.kNS1);
          mma_acc<D>(q.tmem + C::kDK, q.s_at(s) + kDsCols, q.op0(s), j > 0);  // dK += dS^T Q'
        } else {
          mma_acc<D>(q.tmem + C::kDQ, q.s_at(s), q.op0(s), j > 0);  // dQ += dS K'
        }
        ptx::umma_commit(bars + kSFree + (s & 1));
        ptx::umma_commit(bars + kStr0Empty + s % q.kNS0);
        if (j == n - 1) ptx::umma_commit(bars + kAccFull);
      }
      __syncwarp();
    }
    ++it_n;
  }
out:
  q.finish(kMmaDone + 1);
}

// One buffer of S and dP each (DKV at head_dim 128): one warp issues everything in order.  S goes out
// behind dV, which reads P^T in its columns, and dP behind dK, which reads dS^T; each pair runs under
// the compute of the other.
template <int D>
__device__ void bwd_issue_dkv(const BwdArgs& a, uint8_t* sm, uint64_t* bars, uint32_t tmem_base, volatile int* abort_flag) {
  using C = BCfg<D>;
  Issuer<D, true> q(a, sm, bars, tmem_base, abort_flag);
  uint32_t it_n = 0, step = 0, it_cnt = 0;
  BwdItemDesc it;
  while (next_item<D>(sm, bars, it_cnt, it, abort_flag, a.status)) {
    const int n = __shfl_sync(0xffffffffu, it.n, 0);
    if (n <= 0) continue;
    if (!q.resident(it_n)) goto out;
    {
      const uint32_t s0 = __shfl_sync(0xffffffffu, step, 0);
      if (!q.full0(s0)) goto out;
      q.scores_s(s0);
      if (!q.full1(s0)) goto out;
      q.scores_dp(s0, n == 1);
      for (int j = 0; j < n; ++j) {
        const uint32_t s = s0 + (uint32_t)j;
        const bool more = j + 1 < n;
        if (!q.ready(kPReady + (int)(s & 1), par2(s))) goto out;
        if (j == 0 && it_n > 0 && !q.ready(kAccEmpty, (it_n - 1) & 1)) goto out;
        if (q.el) {
          mma_acc<D>(q.tmem + C::kDV, q.s_at(s), q.op1(s), j > 0);
          ptx::umma_commit(bars + kStr1Empty + s % q.kNS1);
        }
        __syncwarp();
        if (more) {
          if (!q.full0(s + 1)) goto out;
          q.scores_s(s + 1);
        }
        if (!q.ready(kDsReady, par1(s))) goto out;
        if (q.el) {
          mma_acc<D>(q.tmem + C::kDK, q.tmem + C::kDP, q.op0(s), j > 0);
          ptx::umma_commit(bars + kStr0Empty + s % q.kNS0);
          if (!more) ptx::umma_commit(bars + kAccFull);
        }
        __syncwarp();
        if (more) {
          if (!q.full1(s + 1)) goto out;
          q.scores_dp(s + 1, j + 2 == n);
        }
      }
      step += (uint32_t)n;
      ++it_n;
    }
  }
out:
  q.finish(kMmaDone);
}

// ------------------------------------------------------------------ compute warps
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// fp32 pairs for the f32x2 instructions (one instruction for two columns)
__device__ __forceinline__ unsigned long long f2pack(float lo, float hi) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f2unpack(unsigned long long v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ unsigned long long f2mul(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 32 columns of a gradient row, scaled and (rotate) turned back by dt, to global memory in bf16:
// 32-byte stores when the gradient buffers are 32-byte aligned (each store then fills whole
// sectors; the rows of a warp lie H * d * 2 bytes apart), else 16-byte stores.
__device__ __forceinline__ void store_cols(__nv_bfloat16* dst, const uint32_t (&acc)[32], float scale, bool rotate,
                                          float dt, const float* omega, bool wide) {
  uint32_t w[16];
#pragma unroll
  for (int p = 0; p < 16; ++p) {
    float u = __uint_as_float(acc[2 * p]) * scale, v = __uint_as_float(acc[2 * p + 1]) * scale;
    if (rotate) {
      float sn, cs;
      __sincosf(dt * omega[p], &sn, &cs);
      const float u2 = u * cs + v * sn;
      v = -u * sn + v * cs;
      u = u2;
    }
    w[p] = bf16x2(u, v);
  }
  if (wide) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
      ptx::st_global_v8(reinterpret_cast<char*>(dst) + 32 * c, w[8 * c], w[8 * c + 1], w[8 * c + 2], w[8 * c + 3],
                        w[8 * c + 4], w[8 * c + 5], w[8 * c + 6], w[8 * c + 7]);
  } else {
    uint4* d4 = reinterpret_cast<uint4*>(dst);
#pragma unroll
    for (int c = 0; c < 4; ++c) d4[c] = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  }
}

template <int D>
__device__ __forceinline__ void zero_row(__nv_bfloat16* dst) {
  uint4* d4 = reinterpret_cast<uint4*>(dst);
#pragma unroll
  for (int c = 0; c < D / 8; ++c) d4[c] = make_uint4(0, 0, 0, 0);
}

// A row's time and type from a tile record (type -1 past the request end).
__device__ __forceinline__ void rec_row(const KeyTileRec* rec, int row, long long& t, int& ty) {
  t = rec->t[row];
  ty = -1;
#pragma unroll
  for (int c = 0; c < kTypes; ++c)
    if ((rec->typebits[c][row >> 5] >> (row & 31)) & 1u) ty = c;
}

// A query row's visibility bits over a key tile without a slot in the mask table.  Not inlined: rare,
// and its registers would be taken from the scores.
__device__ __noinline__ uint4 built_mask(const MaskP& mask, bool live, int pi, long long ti, int tyi,
                                         const KeyTileRec* rec, int key0) {
  const uint32_t f = live ? ~0u : 0u;
  uint32_t vm[4] = {f, f, f, f};
  RowMask rm;
  row_mask_setup(mask, live, pi, ti, tyi, rm);
  build_mask(rm, rec, key0, vm);
  return make_uint4(vm[0], vm[1], vm[2], vm[3]);
}

// DQ: thread = query row of the item's tile and 32 of its keys.
template <int D>
__device__ void bwd_compute_dq(const BwdArgs& a, uint8_t* sm, uint64_t* bars, uint32_t tmem,
                               volatile int* abort_flag) {
  using BL = recattn::BL<D>;
  using C = BCfg<D>;
  constexpr int kNS0 = C::template kNS0<false>;
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3, row = quad * 32 + lane;
  const int wg = (int)((threadIdx.x - 32 * C::kRoles) >> 7);  // this thread's warpgroup
  const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16);
  const float sl2 = a.scale * kLog2e;
  const unsigned long long sl2x2 = f2pack(sl2, sl2);
  const WarpBars wb{ptx::smem_u32(bars), bars, abort_flag, a.status};
  uint32_t it_n = 0, step = 0, it_cnt = 0;
  BwdItemDesc it;
  while (next_item<D>(sm, bars, it_cnt, it, abort_flag, a.status)) {
    const int pi = it.tile * kTile + row;
    const bool row_ok = pi < it.len;
    auto dst = [&]() {
      return static_cast<__nv_bfloat16*>(a.dq) + ((it.tok_start + pi) * a.heads + it.h) * D;
    };
    if (it.n <= 0) {  // no visible key tile
      if (row_ok && wg == 0) zero_row<D>(dst());
      continue;
    }
    WarpCursor<false> cur;
    cur.init(a, it, it.n);
    // the row's time, loaded with Q'
    const int rb = (int)(it_n % BL::kRB);
    if (!wb.wait(kResFull + rb, (it_n / BL::kRB) & 1)) return;
    const float dt = (float)(reinterpret_cast<const KeyTileRec*>(sm + BL::kRRec + rb * kRecB)->t[row] - it.t_ref);
    wb.arrive(kResEmpty + rb);
    cur.vote();
    for (int j = 0; j < it.n; ++j, ++step) {
      // this thread's 32 keys (FULL: the constants of rows past the request's end and of rows that see
      // no key make P zero)
      uint32_t bits = ~0u;
      const bool full = cur.is_full();
      if (!full) {
        const int st = (int)(step % kNS0);
        if (!wb.wait(kStr0Full + st, (step / kNS0) & 1)) return;
        const int tslot = cur.table_slot(), tile = cur.tile();
        const uint8_t* rec = sm + BL::kSRec + st * kStageRecB;  // (read before the step's operand is ready)
        if (tslot >= 0) {  // the row's words of the mask table
          bits = reinterpret_cast<const uint32_t*>(rec)[4 * row + wg];
        } else {
          const long long tok = it.tok_start + (row_ok ? pi : 0);
          const uint4 vm = built_mask(a.mask, row_ok, pi, a.t[tok], a.ty[tok], reinterpret_cast<const KeyTileRec*>(rec),
                                      tile * kTile);
          bits = wg == 0 ? vm.x : wg == 1 ? vm.y : wg == 2 ? vm.z : vm.w;
        }
        __syncwarp();
      }
      cur.next(a, 1);
      if (!wb.wait(kSFull + (step & 1), par2(step))) return;
      ptx::tc_fence_after();
      const uint32_t sb = tl + C::template s_col<false>(step & 1) + 32 * wg, db = tl + C::kDP + 32 * wg;
      uint32_t p[32];
      ptx::tmem_ld32(sb, p);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float y0, y1;
        f2unpack(f2mul(f2pack(__uint_as_float(p[2 * e]), __uint_as_float(p[2 * e + 1])), sl2x2), y0, y1);
        p[2 * e] = __float_as_uint(ex2(y0));
        p[2 * e + 1] = __float_as_uint(ex2(y1));
      }
      if (!full) {
#pragma unroll
        for (int e = 0; e < 32; ++e) p[e] = ((bits >> e) & 1u) ? p[e] : 0u;
      }
      if (!wb.wait(kDpFull, par1(step))) return;
      ptx::tc_fence_after();
      uint32_t d[32], pk[16];
      ptx::tmem_ld32(db, d);
      ptx::tc_fence_before();  // dP's columns go back to the MMA issuer
      wb.arrive(kDpFree);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float g0, g1;
        f2unpack(f2mul(f2pack(__uint_as_float(p[2 * e]), __uint_as_float(p[2 * e + 1])),
                       f2pack(__uint_as_float(d[2 * e]), __uint_as_float(d[2 * e + 1]))), g0, g1);
        pk[e] = bf16x2(g0, g1);
      }
      ptx::tmem_st16_async(sb, pk);  // dS over S columns already read
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      wb.arrive(kPReady + (step & 1));
    }
    if (!wb.wait(kAccFull, it_n & 1)) return;
    ++it_n;
    ptx::tc_fence_after();
    // 32 columns a warpgroup (at head_dim 64 the first two)
    const int c0 = 32 * wg;
    if (c0 < D) {
      uint32_t acc[32];
      ptx::tmem_ld32(tl + C::kDQ + c0, acc);
      ptx::tc_fence_before();
      wb.arrive(kAccEmpty);
      if (row_ok)
        store_cols(dst() + c0, acc, a.scale, a.rotate != 0, dt, a.omega + c0 / 2,
                   (reinterpret_cast<uintptr_t>(a.dq) & 31) == 0);
    } else if (lane == 0) {
      ptx::mbar_arrive(bars + kAccEmpty);
    }
    __syncwarp();
  }
}

// Transpose of the 32 x 32 bit matrix held one row per lane: afterwards lane b holds
// bit l = bit b of lane l's input.  Five rounds swap the off-diagonal blocks of width
// 16, 8, 4, 2 and 1 between lanes l and l ^ j.
__device__ __forceinline__ uint32_t transpose32(uint32_t x, int lane) {
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) {
    const uint32_t m = j == 16 ? 0x0000ffffu : j == 8 ? 0x00ff00ffu : j == 4 ? 0x0f0f0f0fu : j == 2 ? 0x33333333u : 0x55555555u;
    const uint32_t p = __shfl_xor_sync(0xffffffffu, x, j);
    x = (lane & j) ? ((x & ~m) | ((p & ~m) >> j)) : ((x & m) | ((p & m) << j));
  }
  return x;
}

// The compute threads meet (bounded); `n` counts the uses of the barrier.
__device__ __forceinline__ bool group_sync(uint64_t* bar, uint32_t& n, volatile int* abort_flag, int* status) {
  ptx::mbar_arrive(bar);
  return bw_wait_warp(bar, (n++) & 1, abort_flag, status);
}

// DKV: thread = key row of the item's tile and 32 queries of the step (and, while the first
// warpgroup builds a mask, a row of the query tile).
template <int D>
__device__ void bwd_compute_dkv(const BwdArgs& a, uint8_t* sm, uint64_t* bars, uint32_t tmem,
                                volatile int* abort_flag) {
  using BL = recattn::BL<D>;
  using C = BCfg<D>;
  constexpr int kNS0 = C::template kNS0<true>;
  constexpr bool kTwoS = C::template kTwoS<true>;
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3, row = quad * 32 + lane;
  const int wg = (int)((threadIdx.x - 32 * C::kRoles) >> 7);  // this thread's warpgroup
  const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16);
  const float sl2 = a.scale * kLog2e;
  const unsigned long long sl2x2 = f2pack(sl2, sl2);
  const long long T = a.rows / a.heads;
  const int reps = a.group / a.parts;
  const WarpBars wb{ptx::smem_u32(bars), bars, abort_flag, a.status};
  uint32_t it_n = 0, step = 0, grp = 0, it_cnt = 0;
  BwdItemDesc it;
  while (next_item<D>(sm, bars, it_cnt, it, abort_flag, a.status)) {
    const int pj = it.tile * kTile + row;
    const bool key_ok = pj < it.len;
    // where the key's row of dK (at column 0) stands in the gradients, or in the parts
    auto at = [&]() {
      return a.kv_part ? ((long long)it.h * T + it.tok_start + pj) * D
                       : ((it.tok_start + pj) * (a.heads / a.group) + it.h / a.parts) * D;
    };
    auto part_dv = [&]() { return (long long)(a.heads / a.group) * a.parts * T * D; };
    if (it.n <= 0) {  // no query sees this key tile
      if (wg != 0) continue;
      if (key_ok && a.kv_part) {
        float* part = a.kv_part + at();
        const long long n_part = part_dv();
        for (int e = 0; e < D; e += 4)
          *reinterpret_cast<float4*>(part + e) = *reinterpret_cast<float4*>(part + n_part + e) = make_float4(0, 0, 0, 0);
      } else if (key_ok) {
        zero_row<D>(static_cast<__nv_bfloat16*>(a.dk) + at());
        zero_row<D>(static_cast<__nv_bfloat16*>(a.dv) + at());
      }
      continue;
    }
    WarpCursor<true> cur;
    cur.init(a, it, it.n / reps);
    const int rb = (int)(it_n % BL::kRB);
    if (!wb.wait(kResFull + rb, (it_n / BL::kRB) & 1)) return;  // the key tile's record
    const float dt = (float)(reinterpret_cast<const KeyTileRec*>(sm + BL::kRRec + rb * kRecB)->t[row] - it.t_ref);
    cur.vote();
    for (int j = 0; j < it.n; ++j, ++step) {
      // The key's bits for this thread's 32 queries: its word of the mask table's columns when the
      // pair has a slot; otherwise the first warpgroup's threads, as rows of the query tile, build
      // their rows' bits over the key tile and its warps transpose them into per-key words.  Two
      // buffers in turn: a thread reads one before it meets the others for the next.
      uint32_t bits = ~0u;  // (FULL: the constants of queries past the request's end make P zero)
      const bool full = cur.is_full();
      if (!full) {
        const int st = (int)(step % kNS0);
        if (!wb.wait(kStr0Full + st, (step / kNS0) & 1)) return;
        const int tslot = cur.table_slot(), tile = cur.tile();
        const uint8_t* rec = sm + BL::kSRec + st * kStageRecB;  // (read before the step's operands are ready)
        if (tslot >= 0) {
          bits = reinterpret_cast<const uint32_t*>(rec)[4 * row + wg];
        } else {
          uint32_t* col = reinterpret_cast<uint32_t*>(sm + BL::kCol) + (grp & 1) * (kTile * 4);
          if (wg == 0) {
            const int qi = tile * kTile + row;
            long long tq;
            int tyq;
            rec_row(reinterpret_cast<const KeyTileRec*>(rec), row, tq, tyq);
            const uint4 vm = built_mask(a.mask, qi < it.len, qi, tq, tyq,
                                        reinterpret_cast<const KeyTileRec*>(sm + BL::kRRec + rb * kRecB), it.tile * kTile);
            const uint32_t w[4] = {vm.x, vm.y, vm.z, vm.w};
#pragma unroll
            for (int wd = 0; wd < 4; ++wd) col[(32 * wd + lane) * 4 + quad] = transpose32(w[wd], lane);
          }
          if (!group_sync(bars + kGroup, grp, abort_flag, a.status)) return;
          bits = col[4 * row + wg];
        }
        __syncwarp();
      }
      if (j == it.n - 1) {  // the key tile's record was read for the last time
        wb.arrive(kResEmpty + rb);
      }
      cur.next(a, reps);
      // P^T over the columns of S^T already read
      if (!wb.wait(kSFull + (step & 1), par2(step))) return;
      ptx::tc_fence_after();
      const uint32_t sb = tl + C::template s_col<true>(step & 1) + 32 * wg, db = tl + C::kDP + 32 * wg;
      uint32_t p[32], pk[16];
      ptx::tmem_ld32(sb, p);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float y0, y1;
        f2unpack(f2mul(f2pack(__uint_as_float(p[2 * e]), __uint_as_float(p[2 * e + 1])), sl2x2), y0, y1);
        p[2 * e] = __float_as_uint(ex2(y0));
        p[2 * e + 1] = __float_as_uint(ex2(y1));
      }
      if (!full) {
#pragma unroll
        for (int e = 0; e < 32; ++e) p[e] = ((bits >> e) & 1u) ? p[e] : 0u;
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) pk[e] = bf16x2(__uint_as_float(p[2 * e]), __uint_as_float(p[2 * e + 1]));
      ptx::tmem_st16_async(sb, pk);
      if constexpr (!kTwoS) {
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        wb.arrive(kPReady + (step & 1));
      }
      // dS^T beside P^T, or over the columns of dP^T
      if (!wb.wait(kDpFull, par1(step))) return;
      ptx::tc_fence_after();
      uint32_t d[32];
      ptx::tmem_ld32(db, d);
      if constexpr (kTwoS) {
        ptx::tc_fence_before();  // dP's columns go back to the MMA issuer
        wb.arrive(kDpFree);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float g0, g1;
        f2unpack(f2mul(f2pack(__uint_as_float(p[2 * e]), __uint_as_float(p[2 * e + 1])),
                       f2pack(__uint_as_float(d[2 * e]), __uint_as_float(d[2 * e + 1]))), g0, g1);
        pk[e] = bf16x2(g0, g1);
      }
      ptx::tmem_st16_async(kTwoS ? sb + kDsCols : db, pk);
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      wb.arrive(kTwoS ? kPReady + (int)(step & 1) : (int)kDsReady);
    }
    if (!wb.wait(kAccFull, it_n & 1)) return;
    ++it_n;
    ptx::tc_fence_after();
    // dV and dK behind it, 32 columns at a time, the warpgroups in turn
#pragma unroll 1
    for (int c0 = 32 * wg; c0 < 2 * D; c0 += 32 * C::kWG) {
      uint32_t acc[32];
      ptx::tmem_ld32(tl + C::kDV + c0, acc);
      if (c0 + 32 * C::kWG >= 2 * D) {
        ptx::tc_fence_before();
        wb.arrive(kAccEmpty);
      }
      const bool is_v = c0 < D;
      const int col = is_v ? c0 : c0 - D;
      const bool wide = ((reinterpret_cast<uintptr_t>(a.dk) | reinterpret_cast<uintptr_t>(a.dv)) & 31) == 0;
      if (!key_ok) {
        // nothing to store
      } else if (a.kv_part) {  // the part's sums as they are: k_bwd_kv_sum adds the parts of the group
        float* dst = a.kv_part + at() + (is_v ? part_dv() : 0) + col;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          ptx::st_global_v8(dst + 8 * c, acc[8 * c], acc[8 * c + 1], acc[8 * c + 2], acc[8 * c + 3], acc[8 * c + 4],
                            acc[8 * c + 5], acc[8 * c + 6], acc[8 * c + 7]);
      } else if (is_v) {
        store_cols(static_cast<__nv_bfloat16*>(a.dv) + at() + col, acc, 1.f, false, 0.f, a.omega, wide);
      } else {  // scaled and rotated back
        store_cols(static_cast<__nv_bfloat16*>(a.dk) + at() + col, acc, a.scale, a.rotate != 0, dt, a.omega + col / 2, wide);
      }
      __syncwarp();
    }
  }
}

// ------------------------------------------------------------------ row constants
// Block = (tile g, head h, half): D_i = <dO_i, O_i> for 64 rows of the tile, 16 bytes of dO and O a
// thread, every row's loads in flight at once (row by row the kernel took 23 us where it takes 18: 16 ragged requests,
// head_dim 128).  The row's constants as an operand row of the scores'
// extra K step: -lse / scale (in the scores' unit) and -D, each as three bf16 that add up to it, and
// -1e38 in place of the first for rows that see no key, rows past the request's end and pruned
// rows, so that their every P is exp2(-1e38) = 0 whatever mask bits they have.
template <int D>
__global__ void __launch_bounds__(256) k_bwd_rowc(BwdArgs a) {
  constexpr int kLanes = D / 8;  // 16-byte chunks of a row, one per thread
  constexpr int kRows = kTile / 2;  // per block
  const int H = a.heads, h = (int)((blockIdx.x >> 1) % H);
  const long long g = (blockIdx.x >> 1) / H;
  const int b = a.qreq[g];
  const ReqMeta m = a.meta[b];
  const int tile = (int)(g - m.tile_start);
  const int sub = threadIdx.x & (kLanes - 1);
  const int keep = a.qkeep[b];
#pragma unroll
  for (int r0 = 0; r0 < kRows; r0 += 256 / kLanes) {
    const int r = (int)(blockIdx.x & 1) * kRows + r0 + (int)threadIdx.x / kLanes;
    const int p = tile * kTile + r;
    const bool in = p < m.len;
    const long long tok = m.tok_start + (in ? p : 0), row = tok * H + h;
    const uint4 x = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.dout) + row * D)[sub];
    const uint4 y = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.out) + row * D)[sub];
    const float lse = a.lse[row];
    // a pruned query (a query-pruned plan) has no output, so no gradient flows from it;
    // its forward lse and O were never written
    const bool ok = in && query_kept(a.ty[tok], p, keep);
    float acc = 0.f;
    if (ok) {
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 fx = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&xs[i]));
        const float2 fy = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&ys[i]));
        acc = fmaf(fx.x, fy.x, fmaf(fx.y, fy.y, acc));
      }
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (sub == 0) {
      const float l = ok ? lse : INFINITY;
      const float c[2] = {isinf(l) ? -1e38f : -l / a.scale, -acc};
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // three bf16 that add up to it: 24 bits
        const float hi = __bfloat162float(__float2bfloat16(c[i])), mid = __bfloat162float(__float2bfloat16(c[i] - hi));
        w[2 * i] = bf16x2(hi, mid);
        w[2 * i + 1] = bf16x2(c[i] - hi - mid, 0.f);
      }
      a.rowx[((long long)h * a.n_tiles + g) * kTile + r] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// ------------------------------------------------------------------ schedule
// reps > 1: dK/dV items are (tile, part of reps query heads) pairs, one block compacting the
// planner's order of (tile, query head) items to each part's first head, in order.
__global__ void __launch_bounds__(1024) k_bwd_kv_items(BwdSchedArgs s) {
  __shared__ int s_warp[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, Hp = s.heads / s.reps;
  long long base = 0;
  for (long long i0 = 0; i0 < s.n_items; i0 += 1024) {
    const long long i = i0 + threadIdx.x;
    const int e = i < s.n_items ? s.items[i] : 0;
    const int h = e % s.heads;
    const bool take = i < s.n_items && h % s.reps == 0;
    const unsigned bal = __ballot_sync(0xffffffffu, take);
    if (lane == 0) s_warp[warp] = __popc(bal);
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < 32; ++w) {
      before += w < warp ? s_warp[w] : 0;
      total += s_warp[w];
    }
    const long long at = base + before + __popc(bal & ((1u << lane) - 1u));
    if (take && at < s.n_kv_items) s.kv_items[at] = (e / s.heads) * Hp + h / s.reps;
    base += total;
    __syncthreads();
  }
}

// Warps [0, n_tiles): the transposed tile lists -- for key tile g, the query tiles
// of its request whose class against it is not SKIP, in order.  Warps
// [n_tiles, n_tiles + n_items): the descriptors of item w for both modes (DKV: the
// mirrored key tile of the item's query tile, for the first n_kv_items warps).  Lanes take 32 tiles of
// a column of the class matrix at a time (a thread each took 32 us at 64 tiles, 6 now).
__global__ void __launch_bounds__(128) k_bwd_schedule(BwdSchedArgs s) {
  const int lane = threadIdx.x & 31;
  const long long i = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (i < s.n_tiles) {
    const ReqMeta m = s.meta[s.qreq[i]];
    const int kt = (int)(i - m.tile_start);
    uint32_t* out = s.qlist + m.cls_start + (long long)kt * m.ntiles;
    int* out_slot = s.qslot + m.cls_start + (long long)kt * m.ntiles;
    int n = 0;
    for (int q0 = 0; q0 < m.ntiles; q0 += 32) {
      const int qt = q0 + lane;
      const long long pair = m.cls_start + (long long)qt * m.ntiles + kt;
      const int c = qt < m.ntiles ? s.cls[pair] : REC_ATTN_TILE_SKIP;
      const unsigned bal = __ballot_sync(0xffffffffu, c != REC_ATTN_TILE_SKIP);
      if (c != REC_ATTN_TILE_SKIP) {
        const int at = n + __popc(bal & ((1u << lane) - 1u));
        out[at] = (uint32_t)qt | ((uint32_t)c << 24);
        const int p = c == REC_ATTN_TILE_PARTIAL ? s.pslot[pair] : -1;
        out_slot[at] = (p >= 0 && p < s.mcap) ? p : -1;  // a slot always indexes the table
      }
      n += __popc(bal);
    }
    return;
  }
  const long long w = i - s.n_tiles;
  if (w >= s.n_items) return;
  const long long e = s.items[w];
  const long long g = e / s.heads;
  ReqMeta m = s.meta[s.qreq[g]];
  const int qt = (int)(g - m.tile_start);
  int kt = m.ntiles - 1 - qt;
  BwdItemDesc d;
  d.tok_start = m.tok_start;
  d.t_ref = s.t[m.tok_start];
  d.len = m.len;
  d.tile_start = (int)m.tile_start;
  d.h = (int)(e % s.heads);
  d.pad = 0;
  d.list = m.cls_start + (long long)qt * m.ntiles;
  d.tile = qt;
  d.n = max(s.kcount[g], 0);
  if (lane == 0) s.desc[w] = d;
  if (w >= s.n_kv_items) return;
  if (s.reps > 1) {  // dK/dV item w has a tile and heads of its own
    const int Hp = s.heads / s.reps;
    const long long ek = s.kv_items[w], gk = ek / Hp;
    m = s.meta[s.qreq[gk]];
    kt = m.ntiles - 1 - (int)(gk - m.tile_start);
    d.tok_start = m.tok_start;
    d.t_ref = s.t[m.tok_start];
    d.len = m.len;
    d.tile_start = (int)m.tile_start;
    d.h = (int)(ek % Hp);
  }
  const uint8_t* col = s.cls + m.cls_start + kt;
  int n = 0;
  for (int r0 = 0; r0 < m.ntiles; r0 += 32) {
    const int r = r0 + lane;
    n += __popc(__ballot_sync(0xffffffffu, r < m.ntiles && col[(long long)r * m.ntiles] != REC_ATTN_TILE_SKIP));
  }
  d.list = m.cls_start + (long long)kt * m.ntiles;
  d.tile = kt;
  d.n = n * s.reps;
  if (lane == 0) s.desc[s.n_items + w] = d;
}

// The mask table's columns (once per plan): per slot, each warp transposes its 32 query
// rows' words into per-key words, so key j of the tile finds the 128 query bits of its
// column as four words.
__global__ void __launch_bounds__(kTile) k_bwd_colmask(BwdSchedArgs s) {
  const int used = min(__ldcg(s.counters + 7), s.mcap);
  const int r = threadIdx.x, lane = r & 31, quad = r >> 5;
  for (int slot = blockIdx.x; slot < used; slot += gridDim.x) {
    const uint4 w = reinterpret_cast<const uint4*>(s.mtab)[(long long)slot * kTile + r];
    const uint32_t vm[4] = {w.x, w.y, w.z, w.w};
    uint32_t* out = s.ctab + (long long)slot * kTile * 4;
#pragma unroll
    for (int wd = 0; wd < 4; ++wd) out[(32 * wd + lane) * 4 + quad] = transpose32(vm[wd], lane);
  }
}

// ------------------------------------------------------------------ sum of the parts
// Block = (part of tile g, key/value head): dK and dV of its rows as the sums of the group's
// parts, in order; dK is scaled and rotated back; both rounded once.  Eight columns of one row
// a thread.
template <int D>
__global__ void __launch_bounds__(256) k_bwd_kv_sum(BwdArgs a) {
  constexpr int kLanes = D / 8;
  constexpr int kBlocks = kTile * kLanes / 256;  // blocks per tile
  const long long g = blockIdx.x / kBlocks;
  const int hk = blockIdx.y, Hk = a.heads / a.group;
  const ReqMeta m = a.meta[a.qreq[g]];
  const int tile = (int)(g - m.tile_start), c = threadIdx.x & (kLanes - 1);
  const long long T = a.rows / a.heads, n_part = (long long)Hk * a.parts * T * D;
  const long long t_ref = a.t[m.tok_start];
  const int p = tile * kTile + (int)(blockIdx.x % kBlocks) * (256 / kLanes) + threadIdx.x / kLanes;
  if (p < m.len) {
    const long long tok = m.tok_start + p;
    const float* src = a.kv_part + ((long long)hk * a.parts * T + tok) * D + 8 * c;
    float k[8], v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) k[e] = v[e] = 0.f;
#pragma unroll 4
    for (int i = 0; i < a.parts; ++i) {
      const float4* pk = reinterpret_cast<const float4*>(src + (long long)i * T * D);
      const float4* pv = reinterpret_cast<const float4*>(src + (long long)i * T * D + n_part);
      const float4 k0 = __ldcs(pk), k1 = __ldcs(pk + 1), v0 = __ldcs(pv), v1 = __ldcs(pv + 1);
      k[0] += k0.x; k[1] += k0.y; k[2] += k0.z; k[3] += k0.w;
      k[4] += k1.x; k[5] += k1.y; k[6] += k1.z; k[7] += k1.w;
      v[0] += v0.x; v[1] += v0.y; v[2] += v0.z; v[3] += v0.w;
      v[4] += v1.x; v[5] += v1.y; v[6] += v1.z; v[7] += v1.w;
    }
    uint32_t wk[4], wv[4];
    const float dt = (float)(a.t[tok] - t_ref);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float x = k[2 * e] * a.scale, y = k[2 * e + 1] * a.scale;
      if (a.rotate) {
        float sn, cs;
        __sincosf(dt * a.omega[4 * c + e], &sn, &cs);
        const float x2 = x * cs + y * sn;
        y = -x * sn + y * cs;
        x = x2;
      }
      wk[e] = bf16x2(x, y);
      wv[e] = bf16x2(v[2 * e], v[2 * e + 1]);
    }
    const long long at = (tok * Hk + hk) * D + 8 * c;
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.dk) + at) = make_uint4(wk[0], wk[1], wk[2], wk[3]);
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.dv) + at) = make_uint4(wv[0], wv[1], wv[2], wv[3]);
  }
}

// ------------------------------------------------------------------ kernel
// maps: Q', K', V, dO as bf16 views [T][heads * d] (K', V: key/value heads), 64 x 128 boxes.
template <int D, bool DKV>
__global__ void __launch_bounds__(BCfg<D>::kThreads, 1)
    k_bwd_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
             const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do, const BwdArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  using BL = recattn::BL<D>;
  constexpr uint32_t kCW = 4 * BCfg<D>::kWG;  // compute warps
  constexpr bool kTwoS = BCfg<D>::template kTwoS<DKV>;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + BL::kBarsOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + kNumBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kNumBars) + 1;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < BL::kRB; ++i) {
      ptx::mbar_init(bars + kResFull + i, 1);
      ptx::mbar_init(bars + kResEmpty + i, 1 + kCW);  // MMAs done + the compute warps read the record
    }
    for (int i = 0; i < 4; ++i) {
      ptx::mbar_init(bars + kStr0Full + i, 1);
      ptx::mbar_init(bars + kStr0Empty + i, 1);  // the step's last MMA done (the record was read before it)
      ptx::mbar_init(bars + kStr1Full + i, 1);
      ptx::mbar_init(bars + kStr1Empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bars + kSFull + i, 1);
      ptx::mbar_init(bars + kPReady + i, kCW);
    }
    ptx::mbar_init(bars + kDpFull, 1);
    ptx::mbar_init(bars + kDpFree, kCW);
    ptx::mbar_init(bars + kDsReady, kCW);
    ptx::mbar_init(bars + kAccFull, 1);
    ptx::mbar_init(bars + kAccEmpty, kCW);
    ptx::mbar_init(bars + kGroup, 32 * kCW);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bars + kItemFull + i, 1);
      ptx::mbar_init(bars + kItemEmpty + i, (kTwoS ? 2 : 1) + kCW);  // the issuers and the compute warps
      ptx::mbar_init(bars + kSFree + i, 1);
      ptx::mbar_init(bars + kMmaDone + i, 1);
    }
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  {
    // ones over the first three values of a row's constants (S) or the next three (dP); the second
    // halves of the operands are zero
    for (int i = threadIdx.x; i < 2 * kAugB / 16; i += BCfg<D>::kThreads) {
      const int half = i / kTile;  // S ones, zero, dP ones, zero
      reinterpret_cast<uint4*>(sm + BL::kOnes)[i] = make_uint4(half == 0 ? 0x3f803f80u : 0u, half == 0 ? 0x3f80u : 0u,
                                                               half == 2 ? 0x3f803f80u : 0u, half == 2 ? 0x3f80u : 0u);
    }
    for (int i = threadIdx.x; i < BL::kAugs * kAugB / 16; i += BCfg<D>::kThreads)
      reinterpret_cast<uint4*>(sm + BL::kAug)[i] = make_uint4(0u, 0u, 0u, 0u);
    ptx::fence_proxy_async_smem();
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_slot, kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (warp == 0) {
    if ((threadIdx.x & 31) == 0) {
      const void* const res[2] = {DKV ? (const void*)&tm_k : (const void*)&tm_q,
                                  DKV ? (const void*)&tm_v : (const void*)&tm_do};
      const void* const str[2] = {DKV ? (const void*)&tm_q : (const void*)&tm_k,
                                  DKV ? (const void*)&tm_do : (const void*)&tm_v};
      bwd_producer<D, DKV>(a, res, str, sm, bars, abort_flag);
    }
  } else if (warp == 1) {
    if constexpr (kTwoS) bwd_issue_scores<D, DKV>(a, sm, bars, tmem, abort_flag);
    else bwd_issue_dkv<D>(a, sm, bars, tmem, abort_flag);
  } else if (warp == 2) {
    if constexpr (kTwoS) bwd_issue_acc<D, DKV>(a, sm, bars, tmem, abort_flag);
  } else {
    if constexpr (DKV) bwd_compute_dkv<D>(a, sm, bars, tmem, abort_flag);
    else bwd_compute_dq<D>(a, sm, bars, tmem, abort_flag);
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
  // the last CTA to leave resets the item counter for the next launch
  if (threadIdx.x == 0) {
    int* counter = a.counters + (DKV ? 5 : 3);
    __threadfence();
    if (atomicAdd(counter + 1, 1) == (int)gridDim.x - 1) {
      atomicExch(counter, 0);
      atomicExch(counter + 1, 0);
    }
  }
}

template <int D, bool DKV>
cudaError_t launch_mode(const CUtensorMap (&maps)[4], const BwdArgs& a, int grid, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(done, (const void*)k_bwd_tc<D, DKV>, BL<D>::kDynamic);
  if (e != cudaSuccess) return e;
  k_bwd_tc<D, DKV><<<grid, BCfg<D>::kThreads, BL<D>::kDynamic, st>>>(maps[0], maps[1], maps[2], maps[3], a);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_bwd_d(const BwdArgs& a, const CUtensorMap (&maps)[4], int num_sms, cudaStream_t st) {
  k_bwd_rowc<D><<<(unsigned)(2 * a.n_tiles * a.heads), 256, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const long long cap = num_sms;
  e = launch_mode<D, false>(maps, a, (int)(a.n_items < cap ? a.n_items : cap), st);
  if (e != cudaSuccess) return e;
  e = launch_mode<D, true>(maps, a, (int)(a.n_kv_items < cap ? a.n_kv_items : cap), st);
  if (e != cudaSuccess || a.parts == 1) return e;
  const dim3 grid((unsigned)(a.n_tiles * (kTile * D / 8 / 256)), (unsigned)(a.heads / a.group));
  k_bwd_kv_sum<D><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

int bwd_kv_parts(long long n_tiles, int kv_heads, int group, long long least) {
  int parts = 1;
  while (parts < group && n_tiles * kv_heads * parts < least) {
    ++parts;
    while (group % parts) ++parts;
  }
  return parts;
}

cudaError_t launch_bwd_schedule(const BwdSchedArgs& s, int num_sms, cudaStream_t st) {
  const long long n = s.n_tiles + s.n_items;
  if (n <= 0) return cudaSuccess;
  if (s.reps > 1) {
    k_bwd_kv_items<<<1, 1024, 0, st>>>(s);
    const cudaError_t ek = cudaGetLastError();
    if (ek != cudaSuccess) return ek;
  }
  k_bwd_schedule<<<(unsigned)((n + 3) / 4), 128, 0, st>>>(s);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || s.mcap <= 0) return e;
  k_bwd_colmask<<<s.mcap < 8 * num_sms ? s.mcap : 8 * num_sms, kTile, 0, st>>>(s);
  return cudaGetLastError();
}

cudaError_t launch_attn_bwd_tc(const BwdArgs& a, const CUtensorMap (&maps)[4], int head_dim, int num_sms,
                               cudaStream_t st) {
  if (a.n_items <= 0) return cudaSuccess;
  switch (head_dim) {
    case 64: return launch_bwd_d<64>(a, maps, num_sms, st);
    case 128: return launch_bwd_d<128>(a, maps, num_sms, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace recattn
