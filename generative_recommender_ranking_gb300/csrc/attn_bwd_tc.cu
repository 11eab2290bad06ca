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
// Both modes share one persistent kernel shape: at head_dim 64 two CTAs per SM (256
// TMEM columns each), at 128 one (512 columns: the accumulators are twice as wide), and
// six warps -- warp 0 loads with TMA, one thread of warp 1 issues every MMA,
// warps 2 on are the compute warps (one TMEM lane, i.e. one tile row, per
// thread).  The producer claims the planner's (tile, head) items from a global counter
// and publishes each item's descriptor in shared memory for the other roles; mode DKV
// visits key tiles in the mirrored order of the query tiles, so under causal masks
// both modes start with their heaviest items.  Per item the resident operand pair
// stays in shared memory (DQ: Q', dO; DKV: K', V) and the streamed pair (DQ: K', V of
// the query tile's non-SKIP key tiles; DKV: Q', dO of the query tiles whose class
// against the key tile is not SKIP) runs through a two-stage ring.  A streamed tile
// is two 64-wide steps:
//   DQ   S = Q' K'_h^T and dP = dO V_h^T (N = 64); the compute warps write dS (bf16)
//        over the first columns of S; dQ += dS K'_h with dS read from TMEM.  S is
//        double-buffered, so the next step's S runs during this step's compute.
//   DKV  S^T = K' Q'_h^T and dP^T = V dO_h^T; the compute warps write P^T and dS^T
//        (bf16) over them; dV += P^T dO_h and dK += dS^T Q'_h.
// TMEM columns:  DQ   S[0] 0..63 | S[1] 64..127 | dP 128..191 | dQ 192..192+d
//                DKV  S^T 0..63 | dP^T 64..127 | dV 128..128+d | dK 128+d..128+2d
// At head_dim 128, where one CTA has the SM and all 512 columns to itself, the other scores have
// buffers too (DQ: dP[1] 320..383; DKV: S^T[1] 384..447 | dP^T[1] 448..511), so the next step's
// scores always run under this step's compute, and there are two compute warpgroups: each
// takes 32 of a step's 64 columns and half of the epilogue's (with one warpgroup and one buffer
// the SM had four compute warps, all of them waiting for the step's MMAs in turn: 16 ragged
// requests of 603 to 1850 tokens, 8 query and 2 key/value heads, dQ 228 and dK/dV 383 us).
// The accumulators stay in TMEM across an item's tiles; the epilogue scales, undoes
// the rotation and writes bf16 rows.  Everything a compute thread needs besides TMEM
// comes through shared memory with the tiles: the planner's records of the item's tile
// and the streamed tiles (times, type bitmaps) and the rows' constants -lse * log2(e)
// and -D, stored for row pairs as {-lse2(2k), -lse2(2k+1), -D(2k), -D(2k+1)} so that a
// pair of query columns takes one f32x2 operation (k_bwd_rowc, tile-padded so that a
// bulk copy moves a tile's 128 rows), and the item descriptors (k_bwd_schedule, once
// per plan) come from the producer.  PARTIAL tiles take the forward's per-row
// visibility bits (row_mask.cuh), built from the key tile's planner record; in DKV
// each thread first acts as a row of the query tile, builds that row's bits against
// the item's key tile, and the warps transpose the bits into per-key columns with
// shuffles.  PARTIAL pairs with a slot in the plan's mask table skip both: DQ reads the
// table's rows, DKV its columns (transposed once per plan by k_bwd_colmask), bulk-copied
// with the streamed tile.  FULL tiles skip the mask.  The MMAs of one thread run in issue order, so
// an MMA that overwrites TMEM columns an earlier MMA reads needs no wait.  Every
// mbarrier wait is bounded (REC_ATTN_ERR_TIMEOUT in the status word).
#include <cuda_bf16.h>

#include "attn_common.cuh"
#include "launchers.cuh"
#include "ptx_sm103.cuh"
#include "row_mask.cuh"
#include "wait.cuh"

namespace recattn {

namespace {

constexpr int kStep = 64;                   // keys (DQ) or queries (DKV) per MMA step
constexpr int kSlab = kTile * 128;          // 128 rows x 64 bf16 columns, 128-byte swizzled
constexpr int kNS = 2;                      // stages of the streamed ring
// Per head dimension: a [128][D] bf16 tile is D / 64 slabs; TMEM columns of the
// accumulators (DQ: S[0] 0..63 | S[1] 64..127 | dP 128..191 | dQ 192..; DKV: S^T 0..63 |
// dP^T 64..127 | dV 128.. | dK 128 + D..); d = 64 runs two CTAs per SM, d = 128 one.
template <int D>
struct BCfg {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr uint32_t kCols = D == 64 ? 256 : 512;
  static constexpr int kBlocksPerSM = D == 64 ? 2 : 1;
  static constexpr uint32_t kDQ = 192, kDV = 128, kDK = 128 + D;
  static constexpr int kWG = 2;                   // compute warpgroups, 32 of a step's 64 columns each
  static constexpr int kSub = D == 64 ? 16 : 32;  // columns a thread holds at a time
  static constexpr bool kDB = D == 128;           // every score buffer twice
  static constexpr int kThreads = 64 + 128 * kWG;
  // the bf16 operand of a step: each warpgroup's 16 columns of packed pairs (two K steps) over the
  // first half of the 32 score columns that it has read
  static constexpr uint32_t kChunkCols = 32;
  // score buffers of step parity b
  __host__ __device__ static constexpr uint32_t dq_s(uint32_t b) { return b * 64; }
  __host__ __device__ static constexpr uint32_t dq_dp(uint32_t b) { return kDB && b ? 320u : 128u; }
  __host__ __device__ static constexpr uint32_t dkv_s(uint32_t b) { return kDB && b ? 384u : 0u; }
};
constexpr int kRecB = (int)sizeof(KeyTileRec);
constexpr int kMaskB = kTile * 16;  // a PARTIAL pair's 128 rows (or columns) of the mask table
constexpr int kStageRecB = kMaskB > kRecB ? kMaskB : kRecB;  // per streamed stage: one or the other
constexpr uint64_t kWaitNsB = 2000000000ull;  // 2 s
constexpr float kLog2e = 1.4426950408889634f;

// mbarriers
enum : int {
  kResFull = 0,
  kResEmpty,
  kStrFull,
  kStrEmpty = kStrFull + kNS,
  kSyFull = kStrEmpty + kNS,  // [2] the step's two score MMAs completed (by step parity where the
                              // scores have two buffers, else the first only)
  kXReady = kSyFull + 2,      // [2, by step parity] the compute warps wrote the step's bf16 operands
                              // (in mode DQ the next step's scores go out before this step's
                              // operands are consumed, so the compute warps may finish a whole step
                              // ahead of the issuer's wait; with one barrier per parity a barrier
                              // cannot complete twice before its wait)
  kDpFree = kXReady + 2,      // DQ: the compute warps loaded the step's dP
  kAccFull,                   // the item's last accumulating MMA completed
  kAccEmpty,                  // the compute warps read the accumulators
  kGroup,                     // DKV: barrier of the compute threads
  kItemFull,                  // [2] the producer published an item descriptor
  kItemEmpty = kItemFull + 2, // [2] the MMA issuer and the compute warps copied it
  kMmaDone = kItemEmpty + 2,
  kNumBars
};

// The ready barrier of step `step` (a stream-wide step count) and its wait parity.
__host__ __device__ constexpr int xready(uint32_t step) { return kXReady + (int)(step & 1u); }
__host__ __device__ constexpr uint32_t xready_parity(uint32_t step) { return (step >> 1) & 1u; }

// The scores' barrier of a step and its wait parity.
template <int D>
__host__ __device__ constexpr int syfull(uint32_t step) { return kSyFull + (BCfg<D>::kDB ? (int)(step & 1u) : 0); }
template <int D>
__host__ __device__ constexpr uint32_t syfull_parity(uint32_t step) { return BCfg<D>::kDB ? (step >> 1) & 1u : step & 1u; }

// Byte offsets from the 1024-aligned base of dynamic shared memory.
constexpr int kRowB = kTile * 8;  // {-lse2, -D} of a tile's rows, paired (row_neg_lse2 / row_neg_d)
template <int D>
struct BL {
  static constexpr int kTileBytes = BCfg<D>::kTileBytes;
  static constexpr int kRes = 0;                             // [2] resident tiles
  static constexpr int kStr = kRes + 2 * kTileBytes;         // [kNS][2] streamed tiles
  static constexpr int kSRec = kStr + 2 * kNS * kTileBytes;  // [kNS] records of the streamed tiles
  static constexpr int kSRow = kSRec + kNS * kStageRecB;     // DKV: [kNS] row constants of the query tiles
  static constexpr int kRRec = kSRow + kNS * kRowB;          // record of the item's tile
  static constexpr int kRRow = kRRec + kRecB;                // DQ: row constants of the query tile
  static constexpr int kCol = kRRow + kRowB;                 // DKV: [2][128 keys] 128 query bits
  static constexpr int kItems = kCol + 2 * kTile * 16;       // [2] published item descriptors
  static constexpr int kBarsOff = kItems + 2 * 64;
  static constexpr int kTotal = kBarsOff + kNumBars * 8 + 16;  // + abort flag and TMEM slot
  static constexpr int kDynamic = kTotal + 1024;               // slack to align the base
};
static_assert(BL<64>::kSRec % 16 == 0 && BL<64>::kSRow % 16 == 0 && BL<64>::kRRec % 16 == 0 &&
                  BL<64>::kRRow % 16 == 0 && BL<64>::kCol % 16 == 0 && BL<128>::kSRec % 16 == 0 &&
                  BL<128>::kSRow % 16 == 0 && BL<128>::kRRec % 16 == 0 && BL<128>::kRRow % 16 == 0 &&
                  BL<128>::kCol % 16 == 0,
              "bulk-copy alignment");
static_assert(BL<64>::kBarsOff % 8 == 0 && BL<128>::kBarsOff % 8 == 0, "mbarrier alignment");
static_assert(2 * (BL<64>::kDynamic + 1024) <= 228 * 1024, "two CTAs per SM at d = 64");
static_assert(BL<128>::kDynamic <= 227 * 1024, "one CTA per SM at d = 128");

__device__ __forceinline__ bool bw_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  return bounded_wait(bar, parity, abort_flag, status, kWaitNsB);
}
__device__ __forceinline__ bool bw_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                             int* status) {
  const bool ok = bw_wait(bar, parity, abort_flag, status);
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void bw_drain(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = ptx::globaltimer();
  while (!ptx::mbar_try_wait(bar, parity))
    if (ptx::globaltimer() - t0 > kWaitNsB / 4) return;
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
struct Cursor {
  const uint32_t* list;
  const int* slots;
  int r, rep, reps;
  __device__ __forceinline__ void init(const uint32_t* base, const int* slot_base, const BwdItemDesc& d, int n_rep) {
    list = base + d.list;
    slots = slot_base + d.list;
    r = 0;
    rep = 0;
    reps = n_rep;
  }
  __device__ __forceinline__ void next(int& tile, int& cls, int& slot) {
    const uint32_t e = list[r];
    slot = slots[r];
    if (++rep == reps) {
      rep = 0;
      ++r;
    }
    tile = (int)(e & 0xffffffu);
    cls = (int)(e >> 24);
  }
};

// ------------------------------------------------------------------ producer
// maps: resident pair res[0], res[1]; streamed pair str[0], str[1].
//   DQ:  resident Q', dO + the query tile's record and row constants; streamed K', V
//        (+ the key tile's record when the tile is PARTIAL).
//   DKV: resident K', V + the key tile's record; streamed Q', dO + the query tile's
//        record and row constants.
template <int D, bool DKV>
__device__ void bwd_producer(const BwdArgs& a, const void* const (&res)[2], const void* const (&str)[2],
                             uint8_t* sm, uint64_t* bars, volatile int* abort_flag) {
  const uint32_t* lists = DKV ? a.qlist : a.klist;
  uint32_t it_n = 0, s_it = 0, it_cnt = 0;
  bool res_used = false, str_used[kNS];
  uint32_t res_ph = 0, str_ph[kNS];
  for (int i = 0; i < kNS; ++i) { str_used[i] = false; str_ph[i] = 0; }
  const uint4* descs = reinterpret_cast<const uint4*>(a.desc + (DKV ? a.n_items : 0));
  using L = BL<D>;
  constexpr int kTileBytes = L::kTileBytes;
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

    if (!bw_wait(bars + kResEmpty, (it_n & 1) ^ 1, abort_flag, a.status)) goto drain;
    {
      const int x = (DKV ? d.h / a.parts : d.h) * D;
      const long long g = (long long)d.tile_start + d.tile;
      const float2* rows_h = a.rowc + (long long)d.h * a.n_tiles * kTile;  // DQ: head h's row constants
      ptx::mbar_arrive_expect_tx(bars + kResFull, 2 * kTileBytes + kRecB + (DKV ? 0 : kRowB));
      const int y = (int)(d.tok_start + (long long)d.tile * kTile);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        ptx::tma_load_2d(sm + L::kRes + c * kSlab, res[0], x + 64 * c, y, bars + kResFull);
        ptx::tma_load_2d(sm + L::kRes + kTileBytes + c * kSlab, res[1], x + 64 * c, y, bars + kResFull);
      }
      ptx::bulk_load(sm + L::kRRec, a.krec + g, kRecB, bars + kResFull);
      if (!DKV) ptx::bulk_load(sm + L::kRRow, rows_h + g * kTile, kRowB, bars + kResFull);
      res_used = true;
      res_ph = it_n & 1;
      ++it_n;
      Cursor cur;
      const int reps = DKV ? a.group / a.parts : 1;
      cur.init(lists, DKV ? a.qslot : a.kslot, d, reps);
      const int kvx = (d.h / a.group) * D;  // DQ: the columns of the head's key/value head
      for (int j = 0; j < d.n; ++j) {
        int tile, cls, tslot;
        // DKV: the query head of this visit, its columns and its row constants
        const int hq = d.h * reps + cur.rep;
        const int xs = DKV ? hq * D : kvx;
        cur.next(tile, cls, tslot);
        const int st = (int)(s_it % kNS);
        const uint32_t ph = (s_it / kNS) & 1;
        if (!bw_wait(bars + kStrEmpty + st, ph ^ 1, abort_flag, a.status)) goto drain;
        const long long gs = (long long)d.tile_start + tile;
        // PARTIAL tiles with a mask-table slot: the tile's rows (DQ) or columns (DKV) of the
        // table; otherwise DQ reads the key record on PARTIAL tiles, DKV the query record
        const bool tab = cls != REC_ATTN_TILE_FULL && tslot >= 0;
        const bool rec = !tab && (DKV || cls != REC_ATTN_TILE_FULL);
        const int ys = (int)(d.tok_start + (long long)tile * kTile);
        ptx::mbar_arrive_expect_tx(bars + kStrFull + st,
                                   2 * kTileBytes + (tab ? kMaskB : rec ? kRecB : 0) + (DKV ? kRowB : 0));
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          ptx::tma_load_2d(sm + L::kStr + (2 * st) * kTileBytes + c * kSlab, str[0], xs + 64 * c, ys,
                           bars + kStrFull + st);
          ptx::tma_load_2d(sm + L::kStr + (2 * st + 1) * kTileBytes + c * kSlab, str[1], xs + 64 * c, ys,
                           bars + kStrFull + st);
        }
        if (tab)
          ptx::bulk_load(sm + L::kSRec + st * kStageRecB, (DKV ? a.ctab : a.mtab) + (long long)tslot * (kMaskB / 4),
                         kMaskB, bars + kStrFull + st);
        else if (rec)
          ptx::bulk_load(sm + L::kSRec + st * kStageRecB, a.krec + gs, kRecB, bars + kStrFull + st);
        if (DKV)
          ptx::bulk_load(sm + L::kSRow + st * kRowB, a.rowc + ((long long)hq * a.n_tiles + gs) * kTile, kRowB,
                         bars + kStrFull + st);
        str_used[st] = true;
        str_ph[st] = ph;
        ++s_it;
      }
    }
  }
drain:
  // every copy issued must land before the CTA exits (only waits after an abort)
  if (res_used) bw_drain(bars + kResFull, res_ph);
  for (int i = 0; i < kNS; ++i)
    if (str_used[i]) bw_drain(bars + kStrFull + i, str_ph[i]);
}

// ------------------------------------------------------------------ MMA issuer
__device__ __forceinline__ uint64_t kdesc(uint32_t addr) { return ptx::smem_desc_sw128(addr, 16, 1024); }
// MN-major operand: 64-column blocks of N one slab apart
__device__ __forceinline__ uint64_t mndesc(uint32_t addr) { return ptx::smem_desc_sw128(addr, kSlab, 1024); }

// Scores over K = D (both operands K-major, the K steps of 16 columns four per slab;
// B = 64 rows of a tile): N = 64.
template <int D>
__device__ __forceinline__ void mma_scores(uint32_t d, uint32_t a_addr, uint32_t b_addr) {
  constexpr uint32_t id = ptx::idesc_bf16_f32(kTile, kStep, false, false);
  const uint64_t da = kdesc(a_addr), db = kdesc(b_addr);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = (kk >> 2) * kSlab + (kk & 3) * 32;
    ptx::umma_f16(d, ptx::smem_desc_at(da, off), ptx::smem_desc_at(db, off), id, kk > 0);
  }
}
// D (+)= A B with A (128 x 64, bf16) in TMEM and B = 64 rows of a tile as the K
// dimension (MN-major: the tile's D columns are N).
template <int D>
__device__ __forceinline__ void mma_acc(uint32_t d, uint32_t a_tmem, uint32_t b_rows, bool accumulate) {
  constexpr uint32_t id = ptx::idesc_bf16_f32(kTile, D, false, true);
  const uint64_t db = mndesc(b_rows);
#pragma unroll
  for (int kk = 0; kk < kStep / 16; ++kk)
    ptx::umma_f16_ts(d, a_tmem + (kk >> 1) * BCfg<D>::kChunkCols + (kk & 1) * 8, ptx::smem_desc_at(db, kk * 16 * 128), id,
                     (accumulate || kk > 0) ? 1u : 0u);
}

template <int D, bool DKV>
__device__ void bwd_mma(const BwdArgs& a, uint8_t* sm, uint64_t* bars, uint32_t tmem_base, volatile int* abort_flag) {
  using L = BL<D>;
  using C = BCfg<D>;
  constexpr int kTileBytes = L::kTileBytes;
  const uint32_t res0 = ptx::smem_u32(sm + L::kRes), res1 = res0 + kTileBytes;
  const uint32_t str = ptx::smem_u32(sm + L::kStr);
  constexpr uint32_t kHalfBytes = kStep * 128;  // 64 rows of a tile
  uint32_t it_n = 0, s_it = 0, step = 0, it_cnt = 0;
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0);
  const bool el = ptx::elect_one();  // issues for the warp
  BwdItemDesc it;
  while (next_item<D>(sm, bars, it_cnt, it, abort_flag, a.status)) {
    const int n = __shfl_sync(0xffffffffu, it.n, 0);
    if (n <= 0) continue;
    if (!bw_wait_warp(bars + kResFull, it_n & 1, abort_flag, a.status)) goto out;
    ptx::tc_fence_after();
    {
      const uint32_t ii = it_n++;
      const int nsteps = 2 * n;
      const uint32_t step0 = step;
      // the streamed stage of local step ls; waits for it on the tile's first step
      auto stage_of = [&](int ls, bool wait_full, int& st) -> bool {
        const uint32_t sj = s_it + (uint32_t)(ls >> 1);
        st = (int)(sj % kNS);
        if (wait_full && (ls & 1) == 0) {
          if (!bw_wait_warp(bars + kStrFull + st, (sj / kNS) & 1, abort_flag, a.status)) return false;
          ptx::tc_fence_after();
        }
        return true;
      };
      // the first accumulating MMA of an item overwrites the accumulators: the compute
      // warps must have read the previous item's
      auto acc_free = [&]() -> bool {
        if (ii == 0) return true;
        if (!bw_wait_warp(bars + kAccEmpty, (ii - 1) & 1, abort_flag, a.status)) return false;
        ptx::tc_fence_after();
        return true;
      };
      if constexpr (C::kDB) {
        // two buffers of every score: the scores of step ls + 1 go out before this step's operands are
        // waited for.  Their buffer was last read by the accumulation of step ls - 1, issued before
        // them, and by the compute warps, whose operands of that step were waited for.
        auto issue_scores = [&](int ls) -> bool {
          int st;
          if (!stage_of(ls, true, st)) return false;
          const uint32_t b = (step0 + ls) & 1, half = (uint32_t)(ls & 1) * kHalfBytes;
          const uint32_t s0 = tmem + (DKV ? C::dkv_s(b) : C::dq_s(b)), s1 = DKV ? s0 + 64 : tmem + C::dq_dp(b);
          if (el) {
            mma_scores<D>(s0, res0, str + (2 * st) * kTileBytes + half);
            mma_scores<D>(s1, res1, str + (2 * st + 1) * kTileBytes + half);
            ptx::umma_commit(bars + syfull<D>(step0 + ls));
            if (ls == nsteps - 1) ptx::umma_commit(bars + kResEmpty);  // the resident pair read for the last time
          }
          __syncwarp();
          return true;
        };
        if (!issue_scores(0)) goto out;
        for (int ls = 0; ls < nsteps; ++ls) {
          int st;
          stage_of(ls, false, st);
          if (ls + 1 < nsteps && !issue_scores(ls + 1)) goto out;
          if (!bw_wait_warp(bars + xready(step0 + ls), xready_parity(step0 + ls), abort_flag, a.status)) goto out;
          ptx::tc_fence_after();
          if (ls == 0 && !acc_free()) goto out;
          const uint32_t b = (step0 + ls) & 1, half = (uint32_t)(ls & 1) * kHalfBytes;
          const uint32_t r0 = str + (2 * st) * kTileBytes + half, r1 = str + (2 * st + 1) * kTileBytes + half;
          if (el) {
            if constexpr (DKV) {
              mma_acc<D>(tmem + C::kDV, tmem + C::dkv_s(b), r1, ls > 0);       // dV += P^T dO_h
              mma_acc<D>(tmem + C::kDK, tmem + C::dkv_s(b) + 64, r0, ls > 0);  // dK += dS^T Q'_h
            } else {
              mma_acc<D>(tmem + C::kDQ, tmem + C::dq_s(b), r0, ls > 0);  // dQ += dS K'_h
          }
          if (ls & 1) ptx::umma_commit(bars + kStrEmpty + st);
          }
          __syncwarp();
        }
      } else if constexpr (!DKV) {
        // S(ls) = Q' K'_h^T into S buffer (step0 + ls) % 2, dP(ls) = dO V_h^T.  dP(ls + 1)
        // goes out as soon as the compute warps have loaded dP(ls), so both scores of
        // the next step are ready when this step's compute ends.
        auto issue_scores = [&](int ls) -> bool {
          int st;
          if (!stage_of(ls, true, st)) return false;
          const uint32_t half = (uint32_t)(ls & 1) * kHalfBytes;
          if (el) {
            mma_scores<D>(tmem + ((step0 + ls) & 1) * kStep, res0, str + (2 * st) * kTileBytes + half);
            mma_scores<D>(tmem + 128, res1, str + (2 * st + 1) * kTileBytes + half);
            ptx::umma_commit(bars + kSyFull);
            if (ls == nsteps - 1) ptx::umma_commit(bars + kResEmpty);  // Q' and dO read for the last time
          }
          __syncwarp();
          return true;
        };
        if (!issue_scores(0)) goto out;
        for (int ls = 0; ls < nsteps; ++ls) {
          int st;
          stage_of(ls, false, st);
          if (ls + 1 < nsteps) {
            if (!bw_wait_warp(bars + kDpFree, (step0 + ls) & 1, abort_flag, a.status)) goto out;
            ptx::tc_fence_after();
            if (!issue_scores(ls + 1)) goto out;
          }
          if (!bw_wait_warp(bars + xready(step0 + ls), xready_parity(step0 + ls), abort_flag, a.status)) goto out;
          ptx::tc_fence_after();
          if (ls == 0 && !acc_free()) goto out;
          const uint32_t kb = str + (2 * st) * kTileBytes + (ls & 1) * kHalfBytes;
          if (el) {
            mma_acc<D>(tmem + C::kDQ, tmem + ((step0 + ls) & 1) * kStep, kb, ls > 0);  // dQ += dS K'_h
            if (ls & 1) ptx::umma_commit(bars + kStrEmpty + st);
          }
          __syncwarp();
        }
      } else {
        // S^T = K' Q'_h^T and dP^T = V dO_h^T
        auto issue_scores = [&](int ls) -> bool {
          int st;
          if (!stage_of(ls, true, st)) return false;
          if (el) {
            mma_scores<D>(tmem + 0, res0, str + (2 * st) * kTileBytes + (ls & 1) * kHalfBytes);
            mma_scores<D>(tmem + 64, res1, str + (2 * st + 1) * kTileBytes + (ls & 1) * kHalfBytes);
            ptx::umma_commit(bars + kSyFull);
            if (ls == nsteps - 1) ptx::umma_commit(bars + kResEmpty);  // K' and V read for the last time
          }
          __syncwarp();
          return true;
        };
        if (!issue_scores(0)) goto out;
        for (int ls = 0; ls < nsteps; ++ls) {
          int st;
          stage_of(ls, false, st);
          if (!bw_wait_warp(bars + xready(step0 + ls), xready_parity(step0 + ls), abort_flag, a.status)) goto out;
          ptx::tc_fence_after();
          if (ls == 0 && !acc_free()) goto out;
          const uint32_t qb = str + (2 * st) * kTileBytes + (ls & 1) * kHalfBytes;
          const uint32_t ob = str + (2 * st + 1) * kTileBytes + (ls & 1) * kHalfBytes;
          if (el) {
            mma_acc<D>(tmem + C::kDV, tmem + 0, ob, ls > 0);   // dV += P^T dO_h
            mma_acc<D>(tmem + C::kDK, tmem + 64, qb, ls > 0);  // dK += dS^T Q'_h
            if (ls & 1) ptx::umma_commit(bars + kStrEmpty + st);
          }
          __syncwarp();
          if (ls + 1 < nsteps && !issue_scores(ls + 1)) goto out;
        }
      }
      step += (uint32_t)nsteps;
      s_it += (uint32_t)n;
      if (el) ptx::umma_commit(bars + kAccFull);
      __syncwarp();
    }
  }
out:
  // all issued MMAs must complete before TMEM is released
  if (el) ptx::umma_commit(bars + kMmaDone);
  __syncwarp();
  bw_drain(bars + kMmaDone, 0);
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
__device__ __forceinline__ unsigned long long f2fma(unsigned long long a, unsigned long long b,
                                                    unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ unsigned long long f2add(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long f2mul(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The row-constant table of one tile (128 rows): rows 2k and 2k+1 share 16 bytes,
// {-lse2(2k), -lse2(2k+1), -D(2k), -D(2k+1)}, with lse2 = lse * log2(e).
__device__ __forceinline__ float row_neg_lse2(const float* tab, int r) { return tab[(r >> 1) * 4 + (r & 1)]; }
__device__ __forceinline__ float row_neg_d(const float* tab, int r) { return tab[(r >> 1) * 4 + 2 + (r & 1)]; }

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

// DQ: thread = query row of the item's tile.
template <int D>
__device__ void bwd_compute_dq(const BwdArgs& a, uint8_t* sm, uint64_t* bars, uint32_t tmem,
                               volatile int* abort_flag) {
  using BL = recattn::BL<D>;
  using C = BCfg<D>;
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3, row = quad * 32 + lane;
  const int wg = (int)((threadIdx.x - 64) >> 7);  // this thread's warpgroup
  const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16);
  const float sl2 = a.scale * kLog2e;
  const uint8_t* sstage = sm + BL::kSRec;  // per stage: key record or mask-table rows
  const KeyTileRec* rrec = reinterpret_cast<const KeyTileRec*>(sm + BL::kRRec);
  const float* rrow = reinterpret_cast<const float*>(sm + BL::kRRow);
  const int H = a.heads;
  const unsigned long long sl2x2 = f2pack(sl2, sl2);
  const bool wide = (reinterpret_cast<uintptr_t>(a.dq) & 31) == 0;  // row pieces 32-byte aligned
  uint32_t it_n = 0, s_it = 0, step = 0, it_cnt = 0;
  BwdItemDesc it;
  while (next_item<D>(sm, bars, it_cnt, it, abort_flag, a.status)) {
    const int pi = it.tile * kTile + row;
    const bool row_ok = pi < it.len;
    const long long tok = it.tok_start + pi, grow = tok * H + it.h;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.dq) + grow * D;
    if (it.n <= 0) {  // no visible key tile
      if (row_ok && wg == 0) zero_row<D>(dst);
      continue;
    }
    // the row's time, type and constants, loaded with Q'
    if (!bw_wait_warp(bars + kResFull, it_n & 1, abort_flag, a.status)) return;
    long long ti;
    int tyi;
    rec_row(rrec, row, ti, tyi);
    const float nl = row_neg_lse2(rrow, row), nd = row_neg_d(rrow, row);
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bars + kResEmpty);
    // a row that sees no key contributes nothing: its P is exp2(s - inf) = 0, so FULL
    // tiles need no mask for it
    const bool live = row_ok && nl != INFINITY;
    const unsigned long long nl2 = f2pack(live ? nl : -INFINITY, live ? nl : -INFINITY), nd2 = f2pack(nd, nd);
    RowMask rm;
    row_mask_setup(a.mask, live, pi, ti, tyi, rm);
    Cursor cur;
    cur.init(a.klist, a.kslot, it, 1);
    for (int j = 0; j < it.n; ++j) {
      int kt, cls, tslot;
      cur.next(kt, cls, tslot);
      const int st = (int)(s_it % kNS);
      const uint32_t ph = (s_it / kNS) & 1;
      ++s_it;
      const uint32_t f = live ? ~0u : 0u;
      uint32_t vm[4] = {f, f, f, f};
      if (cls != REC_ATTN_TILE_FULL) {
        if (!bw_wait_warp(bars + kStrFull + st, ph, abort_flag, a.status)) return;
        if (tslot >= 0) {  // the row's words of the mask table (zero for rows that see no key)
          const uint4 w = reinterpret_cast<const uint4*>(sstage + st * kStageRecB)[row];
          vm[0] = w.x; vm[1] = w.y; vm[2] = w.z; vm[3] = w.w;
        } else {
          build_mask(rm, reinterpret_cast<const KeyTileRec*>(sstage + st * kStageRecB), kt * kTile, vm);
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bars + kStrEmpty + st);  // the stage's record was read
#pragma unroll 1
      for (int hh = 0; hh < 2; ++hh, ++step) {
        if (!bw_wait_warp(bars + syfull<D>(step), syfull_parity<D>(step), abort_flag, a.status)) return;
        ptx::tc_fence_after();
        const uint32_t sb = tl + C::dq_s(step & 1), db = tl + C::dq_dp(step & 1);
        const uint32_t wb[2] = {hh ? vm[2] : vm[0], hh ? vm[3] : vm[1]};  // this step's 64 keys
        constexpr int SUB = C::kSub;
        const uint32_t bits = wg ? wb[1] : wb[0];  // this warpgroup's 32 keys
        uint32_t d[32], sr[SUB], pk[SUB / 2];
        ptx::tmem_ld32_async(db + 32 * wg, d);
        if constexpr (SUB == 32) ptx::tmem_ld32_async(sb + 32 * wg, sr);
        ptx::tmem_wait_ld32(d);
        if constexpr (SUB == 32) ptx::tmem_wait_ld32(sr);
        if constexpr (!C::kDB) {  // dP's columns go back to the MMA issuer
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bars + kDpFree);
        }
#pragma unroll
        for (int u = 0; u < 32 / SUB; ++u) {
          if constexpr (SUB == 16) ptx::tmem_ld16(sb + 32 * wg + 16 * u, sr);
#pragma unroll
          for (int e = 0; e < SUB / 2; ++e) {
            float y0, y1;
            f2unpack(f2fma(f2pack(__uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1])), sl2x2, nl2), y0, y1);
            float p0 = ex2(y0), p1 = ex2(y1);
            if (cls != REC_ATTN_TILE_FULL) {
              p0 = ((bits >> (SUB * u + 2 * e)) & 1u) ? p0 : 0.f;
              p1 = ((bits >> (SUB * u + 2 * e + 1)) & 1u) ? p1 : 0.f;
            }
            float g0, g1;
            f2unpack(f2mul(f2pack(p0, p1), f2add(f2pack(__uint_as_float(d[SUB * u + 2 * e]),
                                                        __uint_as_float(d[SUB * u + 2 * e + 1])), nd2)), g0, g1);
            pk[e] = bf16x2(g0, g1);
          }
          // dS over S columns already read
          if constexpr (SUB == 16) ptx::tmem_st8_async(sb + 32 * wg + 8 * u, pk);
          else ptx::tmem_st16_async(sb + 32 * wg, pk);
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bars + xready(step));
      }
    }
    if (!bw_wait_warp(bars + kAccFull, it_n & 1, abort_flag, a.status)) return;
    ++it_n;
    ptx::tc_fence_after();
    // each warpgroup half of the columns, 32 at a time
#pragma unroll 1
    for (int c0 = wg * (D / 2); c0 < (wg + 1) * (D / 2); c0 += 32) {
      uint32_t acc[32];
      ptx::tmem_ld32(tl + C::kDQ + c0, acc);
      if (c0 + 32 >= (wg + 1) * (D / 2)) {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bars + kAccEmpty);
      }
      if (row_ok)
        store_cols(dst + c0, acc, a.scale, a.rotate != 0, (float)(ti - it.t_ref), a.omega + c0 / 2, wide);
      __syncwarp();
    }
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

// DKV: thread = key row of the item's tile (and, while the masks are built, a row of
// the query tile).  The column bits of the next query tile are built while the tensor
// core runs the second half of the current one (two buffers of column bits).
template <int D>
__device__ void bwd_compute_dkv(const BwdArgs& a, uint8_t* sm, uint64_t* bars, uint32_t tmem,
                                volatile int* abort_flag) {
  using BL = recattn::BL<D>;
  using C = BCfg<D>;
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3, row = quad * 32 + lane;
  const int wg = (int)((threadIdx.x - 64) >> 7);  // this thread's warpgroup
  const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16);
  const float sl2 = a.scale * kLog2e;
  const KeyTileRec* rrec = reinterpret_cast<const KeyTileRec*>(sm + BL::kRRec);
  const uint8_t* sstage = sm + BL::kSRec;  // per stage: query record or mask-table columns
  const float* srow = reinterpret_cast<const float*>(sm + BL::kSRow);
  const unsigned long long sl2x2 = f2pack(sl2, sl2);
  const bool wide = ((reinterpret_cast<uintptr_t>(a.dk) | reinterpret_cast<uintptr_t>(a.dv)) & 31) == 0;
  uint32_t* colS = reinterpret_cast<uint32_t*>(sm + BL::kCol);
  const int Hk = a.heads / a.group;
  uint32_t it_n = 0, s_it = 0, step = 0, grp = 0, cbuf = 0, it_cnt = 0;
  BwdItemDesc it;
  while (next_item<D>(sm, bars, it_cnt, it, abort_flag, a.status)) {
    const int pj = it.tile * kTile + row;
    const bool key_ok = pj < it.len;
    const long long growk = (it.tok_start + pj) * Hk + it.h / a.parts;
    const long long n_part = (long long)Hk * a.parts * (a.rows / a.heads) * D;  // one gradient's parts
    float* part = a.kv_part ? a.kv_part + ((long long)it.h * (a.rows / a.heads) + it.tok_start + pj) * D : nullptr;
    __nv_bfloat16* dkr = static_cast<__nv_bfloat16*>(a.dk) + growk * D;
    __nv_bfloat16* dvr = static_cast<__nv_bfloat16*>(a.dv) + growk * D;
    if (it.n <= 0) {  // no query sees this key tile
      if (wg != 0) continue;
      if (key_ok && part) {
        for (int e = 0; e < D; e += 4)
          *reinterpret_cast<float4*>(part + e) = *reinterpret_cast<float4*>(part + n_part + e) = make_float4(0, 0, 0, 0);
      } else if (key_ok) {
        zero_row<D>(dkr);
        zero_row<D>(dvr);
      }
      continue;
    }
    if (!bw_wait_warp(bars + kResFull, it_n & 1, abort_flag, a.status)) return;  // the key tile's record
    const long long tj = rrec->t[row];
    Cursor cur;
    cur.init(a.qlist, a.qslot, it, a.group / a.parts);
    // Column bits of the item's j-th query tile (stage st) into buffer `buf`: the key's
    // words of the mask table's columns when the pair has a slot; otherwise, as query
    // row `row` of the tile, this thread builds the row's bits over the key tile and
    // each warp transposes its 32 rows into per-key words.
    auto prepare = [&](int j, int qt, int cls, int tslot, int st, uint32_t ph, uint32_t buf) -> bool {
      if (!bw_wait_warp(bars + kStrFull + st, ph, abort_flag, a.status)) return false;
      // after the item's last read of the key tile's record, its buffer may be refilled
      auto release_rec = [&]() {
        if (j == it.n - 1) {
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bars + kResEmpty);
        }
      };
      if (cls == REC_ATTN_TILE_FULL || wg != 0) {  // the steps of a FULL tile apply no mask
        release_rec();                             // (and one warpgroup builds the others' bits)
        return true;
      }
      if (tslot >= 0) {
        reinterpret_cast<uint4*>(colS + buf * (kTile * 4))[row] =
            reinterpret_cast<const uint4*>(sstage + st * kStageRecB)[row];
        release_rec();
        return true;
      }
      const int qi = qt * kTile + row;
      long long tq;
      int tyq;
      rec_row(reinterpret_cast<const KeyTileRec*>(sstage + st * kStageRecB), row, tq, tyq);
      const bool live = qi < it.len && row_neg_lse2(srow + st * 2 * kTile, row) != INFINITY;
      const uint32_t f = live ? ~0u : 0u;
      uint32_t vm[4] = {f, f, f, f};
      RowMask rm;
      row_mask_setup(a.mask, live, qi, tq, tyq, rm);
      build_mask(rm, rrec, it.tile * kTile, vm);
      release_rec();
#pragma unroll
      for (int wd = 0; wd < 4; ++wd) colS[buf * (kTile * 4) + (32 * wd + lane) * 4 + quad] = transpose32(vm[wd], lane);
      return true;
    };
    int qt, cls, tslot;
    cur.next(qt, cls, tslot);
    int scls = cls;  // the class of the query tile the steps run on
    int st = (int)(s_it % kNS);
    if (!prepare(0, qt, cls, tslot, st, (s_it / kNS) & 1, cbuf)) return;
    ++s_it;
    for (int j = 0; j < it.n; ++j) {
      // a masked tile's words, written by the first warpgroup, are read by both.  The other buffer,
      // which prepare() overwrites next, was read at the start of the last tile by every thread:
      // prepare() comes after this tile's first scores, and those went out after the last tile's
      // first operands were ready.
      uint4 cm = make_uint4(0, 0, 0, 0);
      if (scls != REC_ATTN_TILE_FULL) {
        if (!group_sync(bars + kGroup, grp, abort_flag, a.status)) return;
        cm = reinterpret_cast<const uint4*>(colS)[cbuf * kTile + row];
      }
      const float* rows = srow + st * 2 * kTile;
      int nqt = 0, ncls = 0, nslot = -1, nst = 0;
      uint32_t nph = 0;
      if (j + 1 < it.n) {
        cur.next(nqt, ncls, nslot);
        nst = (int)(s_it % kNS);
        nph = (s_it / kNS) & 1;
        ++s_it;
      }
      // one 64-query step: P^T and dS^T over the scores' TMEM columns
      auto do_step = [&](int hh) -> bool {
        if (!bw_wait_warp(bars + syfull<D>(step), syfull_parity<D>(step), abort_flag, a.status)) return false;
        const uint32_t sb = tl + C::dkv_s(step & 1);
        ++step;
        ptx::tc_fence_after();
        const uint32_t wb[2] = {hh ? cm.z : cm.x, hh ? cm.w : cm.y};  // this step's 64 queries
        constexpr int SUB = C::kSub;
        const uint32_t bits = wg ? wb[1] : wb[0];  // this warpgroup's 32 queries
        // {-lse2, -D} of the 32 queries, a pair per 16-byte load (broadcast; one load for P^T and
        // dS^T: the scores' MMAs take most of the shared memory's bandwidth, loads wait behind them)
        const float4* q4 = reinterpret_cast<const float4*>(rows + (hh * kStep + 32 * wg) * 2);
#pragma unroll
        for (int u = 0; u < 32 / SUB; ++u) {
          uint32_t r[2 * SUB], pk[SUB / 2], pd[SUB / 2];  // S^T, then dP^T
          if constexpr (SUB == 16) {
            ptx::tmem_ld16x2(sb + 32 * wg + 16 * u, sb + 64 + 32 * wg + 16 * u, r);
          } else {
            ptx::tmem_ld32x2_async(sb + 32 * wg, sb + 64 + 32 * wg, r);
            ptx::tmem_wait_ld(r);
          }
#pragma unroll
          for (int g = 0; g < SUB / 2; ++g) {
            const float4 k2 = q4[SUB / 2 * u + g];
            float x0, x1;
            f2unpack(f2fma(f2pack(__uint_as_float(r[2 * g]), __uint_as_float(r[2 * g + 1])), sl2x2,
                           f2pack(k2.x, k2.y)), x0, x1);
            x0 = ex2(x0);
            x1 = ex2(x1);
            if (scls != REC_ATTN_TILE_FULL) {  // FULL: queries past the request end have -lse2 = -inf
              x0 = ((bits >> (SUB * u + 2 * g)) & 1u) ? x0 : 0.f;
              x1 = ((bits >> (SUB * u + 2 * g + 1)) & 1u) ? x1 : 0.f;
            }
            pk[g] = bf16x2(x0, x1);
            float g0, g1;
            f2unpack(f2mul(f2pack(x0, x1),
                           f2add(f2pack(__uint_as_float(r[SUB + 2 * g]), __uint_as_float(r[SUB + 2 * g + 1])),
                                 f2pack(k2.z, k2.w))), g0, g1);
            pd[g] = bf16x2(g0, g1);
          }
          // P^T and dS^T over the columns already read
          if constexpr (SUB == 16) {
            ptx::tmem_st8_async(sb + 32 * wg + 8 * u, pk);
            ptx::tmem_st8_async(sb + 64 + 32 * wg + 8 * u, pd);
          } else {
            ptx::tmem_st16_async(sb + 32 * wg, pk);
            ptx::tmem_st16_async(sb + 64 + 32 * wg, pd);
          }
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bars + xready(step - 1));  // step was counted on at the wait
        return true;
      };
      if (!do_step(0)) return;
      if (j + 1 < it.n && !prepare(j + 1, nqt, ncls, nslot, nst, nph, cbuf ^ 1u)) return;
      if (!do_step(1)) return;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bars + kStrEmpty + st);  // the stage's record and constants were read
      st = nst;
      scls = ncls;
      cbuf ^= 1u;
    }
    if (!bw_wait_warp(bars + kAccFull, it_n & 1, abort_flag, a.status)) return;
    ++it_n;
    ptx::tc_fence_after();
    // dV and dK behind it, 32 columns at a time, the warpgroups in turn
#pragma unroll 1
    for (int c0 = 32 * wg; c0 < 2 * D; c0 += 64) {
      uint32_t acc[32];
      ptx::tmem_ld32(tl + C::kDV + c0, acc);
      if (c0 + 64 >= 2 * D) {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bars + kAccEmpty);
      }
      const bool is_v = c0 < D;
      const int col = is_v ? c0 : c0 - D;
      if (!key_ok) {
        // nothing to store
      } else if (part) {  // the part's sums as they are: k_bwd_kv_sum adds the parts of the group
        float* dst = part + (is_v ? n_part : 0) + col;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          ptx::st_global_v8(dst + 8 * c, acc[8 * c], acc[8 * c + 1], acc[8 * c + 2], acc[8 * c + 3], acc[8 * c + 4],
                            acc[8 * c + 5], acc[8 * c + 6], acc[8 * c + 7]);
      } else if (is_v) {
        store_cols(dvr + col, acc, 1.f, false, 0.f, a.omega, wide);
      } else {  // scaled and rotated back
        store_cols(dkr + col, acc, a.scale, a.rotate != 0, (float)(tj - it.t_ref), a.omega + col / 2, wide);
      }
      __syncwarp();
    }
  }
}

// ------------------------------------------------------------------ row constants
// Block = (tile g, head h): D_i = <dO_i, O_i> for the tile's 128 rows, eight threads per
// row (16 bytes of dO and O each, coalesced), written negated with -lse * log2(e) into
// the tile-padded table, rows paired (row_neg_lse2 / row_neg_d).  lse2 is -inf for rows
// that see no key and +inf for rows past the request end and pruned rows, so that
// every P of the latter is exp2(s - inf) = 0 whatever mask bits they have.
template <int D>
__global__ void __launch_bounds__(256) k_bwd_rowc(BwdArgs a) {
  constexpr int kLanes = D / 8;  // 16-byte chunks of a row, one per thread
  const long long g = blockIdx.x;
  const int h = blockIdx.y, H = a.heads;
  const int b = a.qreq[g];
  const ReqMeta m = a.meta[b];
  const int tile = (int)(g - m.tile_start);
  const int sub = threadIdx.x & (kLanes - 1);
  float* out = reinterpret_cast<float*>(a.rowc + ((long long)h * a.n_tiles + g) * kTile);
  const int keep = a.qkeep[b];
#pragma unroll 1
  for (int r = threadIdx.x / kLanes; r < kTile; r += 256 / kLanes) {
    const int p = tile * kTile + r;
    const bool in = p < m.len;
    // a pruned query (a query-pruned plan) has no output, so no gradient flows from it;
    // its forward lse and O were never written
    const bool ok = in && query_kept(a.ty[m.tok_start + p], p, keep);
    const long long row = (m.tok_start + p) * H + h;
    float acc = 0.f;
    if (ok) {
      const uint4 x = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.dout) + row * D)[sub];
      const uint4 y = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.out) + row * D)[sub];
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
      const float l = ok ? a.lse[row] : INFINITY;
      out[(r >> 1) * 4 + (r & 1)] = -(l == -INFINITY ? -INFINITY : l * kLog2e);
      out[(r >> 1) * 4 + 2 + (r & 1)] = -acc;
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

// Threads [0, n_tiles): the transposed tile lists -- for key tile g, the query tiles
// of its request whose class against it is not SKIP, in order.  Threads
// [n_tiles, n_tiles + n_items): the descriptors of item w for both modes (DKV: the
// mirrored key tile of the item's query tile, for the first n_kv_items threads).
__global__ void __launch_bounds__(128) k_bwd_schedule(BwdSchedArgs s) {
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i < s.n_tiles) {
    const ReqMeta m = s.meta[s.qreq[i]];
    const int kt = (int)(i - m.tile_start);
    uint32_t* out = s.qlist + m.cls_start + (long long)kt * m.ntiles;
    int* out_slot = s.qslot + m.cls_start + (long long)kt * m.ntiles;
    int n = 0;
    for (int qt = 0; qt < m.ntiles; ++qt) {
      const long long pair = m.cls_start + (long long)qt * m.ntiles + kt;
      const int c = s.cls[pair];
      if (c == REC_ATTN_TILE_SKIP) continue;
      out[n] = (uint32_t)qt | ((uint32_t)c << 24);
      const int p = c == REC_ATTN_TILE_PARTIAL ? s.pslot[pair] : -1;
      out_slot[n] = (p >= 0 && p < s.mcap) ? p : -1;  // a slot always indexes the table
      ++n;
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
  s.desc[w] = d;
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
  for (int r = 0; r < m.ntiles; ++r) n += col[(long long)r * m.ntiles] != REC_ATTN_TILE_SKIP;
  d.list = m.cls_start + (long long)kt * m.ntiles;
  d.tile = kt;
  d.n = n * s.reps;
  s.desc[s.n_items + w] = d;
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
__global__ void __launch_bounds__(BCfg<D>::kThreads, BCfg<D>::kBlocksPerSM)
    k_bwd_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
             const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do, const BwdArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  using BL = recattn::BL<D>;
  constexpr uint32_t kCols = BCfg<D>::kCols;
  constexpr uint32_t kCW = 4 * BCfg<D>::kWG;  // compute warps
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + BL::kBarsOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + kNumBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kNumBars) + 1;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    ptx::mbar_init(bars + kResFull, 1);
    ptx::mbar_init(bars + kResEmpty, 1 + kCW);  // MMAs done + the compute warps read the record
    for (int i = 0; i < kNS; ++i) {
      ptx::mbar_init(bars + kStrFull + i, 1);
      ptx::mbar_init(bars + kStrEmpty + i, 1 + kCW);  // MMAs done + the compute warps read the record
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bars + kSyFull + i, 1);
      ptx::mbar_init(bars + kXReady + i, kCW);
    }
    ptx::mbar_init(bars + kDpFree, kCW);
    ptx::mbar_init(bars + kAccFull, 1);
    ptx::mbar_init(bars + kAccEmpty, kCW);
    ptx::mbar_init(bars + kGroup, 32 * kCW);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bars + kItemFull + i, 1);
      ptx::mbar_init(bars + kItemEmpty + i, 1 + kCW);  // the MMA issuer and the compute warps
    }
    ptx::mbar_init(bars + kMmaDone, 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_slot, kCols);
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
    bwd_mma<D, DKV>(a, sm, bars, tmem, abort_flag);
  } else {
    if constexpr (DKV) bwd_compute_dkv<D>(a, sm, bars, tmem, abort_flag);
    else bwd_compute_dq<D>(a, sm, bars, tmem, abort_flag);
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kCols);
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
  k_bwd_rowc<D><<<dim3((unsigned)a.n_tiles, (unsigned)a.heads), 256, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const long long cap = (long long)BCfg<D>::kBlocksPerSM * num_sms;
  e = launch_mode<D, false>(maps, a, (int)(a.n_items < cap ? a.n_items : cap), st);
  if (e != cudaSuccess) return e;
  e = launch_mode<D, true>(maps, a, (int)(a.n_kv_items < cap ? a.n_kv_items : cap), st);
  if (e != cudaSuccess || a.parts == 1) return e;
  const dim3 grid((unsigned)(a.n_tiles * (kTile * D / 8 / 256)), (unsigned)(a.heads / a.group));
  k_bwd_kv_sum<D><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

int bwd_kv_parts(long long n_tiles, int kv_heads, int group, int head_dim, int num_sms) {
  const long long slots = (long long)(head_dim == 64 ? BCfg<64>::kBlocksPerSM : BCfg<128>::kBlocksPerSM) * num_sms;
  int parts = 1;
  while (parts < group && n_tiles * kv_heads * parts < 3 * slots) {
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
  k_bwd_schedule<<<(unsigned)((n + 127) / 128), 128, 0, st>>>(s);
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
