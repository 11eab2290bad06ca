// score.cu -- candidates scored against a cached history that all of them share, with
// query heads in groups of G per key/value head (M-FALCON, HSTU notes on the blog index
// page: the history's keys and values are computed once and every candidate reads them;
// CADET review page, hundreds of candidates per request).
//
// For request b and key/value head hk the rows are (candidate c, head of the group g), all
// reading the same keys: r = c G + g.  Row r gets
//   O = (sum_j vis(r, j) 2^(s_rj - m) V_j + 2^(s_self - m) v_c) / (sum of the weights),
// s = scale log2(e) <Q'_r, K'_j> over the history, s_self = scale log2(e) <q_r, k_c> (both
// rotated by the same angle, so not rotated at all).  The only masks of a candidate row are
// in time: real-time events need t_j < t_c, the delay rule t_j <= t_c - delta, so key j is
// visible exactly when t_c >= need_j, and need_j is computed once when the cache is made.
//
// k_score_rows (few rows): bound by HBM, the history's keys and values being read once.  A
// block takes M groups of 8 rows, one key/value head and a run of key tiles; a producer warp
// keeps three 32 KB stages of K' and V tiles in flight with TMA, four warps each take a
// quarter of every tile's keys with their own running maximum and sum, so they meet only at
// the end.  The scores' and outputs' matrix products are m16n8k16 with 8 rows in the 16: the
// upper 8 hold the operand rounded to bf16 and the lower 8 what the rounding left, so Q' and P
// enter with 16 bits of mantissa at no cost (a thread holds row g and row g + 8 of every
// product).  The blocks of a thread-block cluster share one item's key tiles and join their parts
// through distributed shared memory; where clusters of eight would leave most SMs idle (few rows,
// long histories) blocks leave their maximum, sum and unnormalised output in a workspace, which
// k_score_combine joins.  Both orders are fixed.  64 requests of 4100 to 8192 keys, a candidate each,
// head_dim 128, 8 query and 2 key/value heads: 72 us, 5.6 TB/s of the cache (84% of a copy's rate); one
// request of 1023 keys: 7 us.
//
// Many rows (score_many in api.cu has both kernels' measured cost): k_score_pack lays Q' out in row
// order, rounded to bf16, and k_attn_tc's CAND instantiation takes items of 128 rows, P rounded too (the
// output is off by 3.0e-3, relative, against 2.1e-3 to 2.3e-3 with few rows, 1.6e-3 being its own rounding).  16 requests of 3500 to 4096
// keys, 420 to 500 candidates, head_dim 64: 8 + 107 us (540 TFLOP/s); bound by the softmax of its 1.6
// items a stream.
#include <climits>

#include <cuda_bf16.h>

#include "launchers.cuh"
#include "ptx_sm103.cuh"
#include "wait.cuh"

namespace recattn {

namespace {

constexpr uint64_t kScoreWaitNs = 2000000000ull;  // 2 s
constexpr int kScoreStages = 3;
constexpr int kScoreWarps = 4;                          // consumer warps; one more loads
constexpr int kScoreThreads = 32 * (kScoreWarps + 1);
constexpr int kOperand = 16384;                         // bytes of a stage's K' (or V) tile

template <int D>
struct SCfg {
  static constexpr int kKeys = D == 64 ? 128 : 64;      // keys per stage
  static constexpr int kWarpKeys = kKeys / kScoreWarps; // 32 or 16
  static constexpr int kNT = kWarpKeys / 8;             // 8-key score tiles per warp
  static constexpr int kSlab = kKeys * 128;             // 64 columns, 128-byte swizzled rows
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
// The bf16 pair nearest to (lo, hi), and the pair of what that rounding left.
__device__ __forceinline__ void split_pair(float lo, float hi, uint32_t& top, uint32_t& rest) {
  top = bf16_pair(lo, hi);
  rest = bf16_pair(lo - __uint_as_float(top << 16), hi - __uint_as_float(top & 0xffff0000u));
}
__device__ __forceinline__ float2 bf16x2_float(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Block-uniform place of a work item: request, row group, key/value head, run of key tiles.
struct ScoreItem {
  int b, rows, rb, hk, split, nsplit;
  long long cand0;  // first candidate of the request
};
__device__ __forceinline__ int upper_index(const int* starts, int n, int x) {  // last i with starts[i] <= x
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}
__device__ __forceinline__ int n_splits(const ScoreArgs& a, int tiles) {
  const int n = (tiles + a.chunk_tiles - 1) / a.chunk_tiles;
  return n > 0 ? n : 1;
}
__device__ __forceinline__ int request_tiles(const ScoreArgs& a, int b) {
  return (a.hist_len[b] + a.tile_keys - 1) / a.tile_keys;
}

// A row's parts (maximum, sum, this lane's DL output columns) joined with the candidate's own
// key, and written: the row's output in bf16 and its log-sum-exp.
template <int D>
__device__ __forceinline__ void finish_row(const ScoreArgs& a, long long cand, int h, int lane, float m, float l,
                                           float (&o)[D / 32]) {
  constexpr int DL = D / 32;
  const int G = a.heads / a.kv_heads;
  const long long qrow = (cand * a.heads + h) * D + lane * DL;
  const long long krow = (cand * a.kv_heads + h / G) * D + lane * DL;
  float dot = 0.f, v[DL];
#pragma unroll
  for (int e = 0; e < DL; e += 2) {
    const float2 q2 = bf16x2_float(*reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.q) + qrow + e));
    const float2 k2 = bf16x2_float(*reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.k) + krow + e));
    const float2 v2 = bf16x2_float(*reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.v) + krow + e));
    dot = fmaf(q2.x, k2.x, fmaf(q2.y, k2.y, dot));
    v[e] = v2.x;
    v[e + 1] = v2.y;
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, x);
  const float s = dot * a.scale_log2;
  const float top = fmaxf(m, s);
  const float wp = exp2_fast(m - top), ws = exp2_fast(s - top);
  const float sum = l * wp + ws, inv = 1.f / sum;
#pragma unroll
  for (int e = 0; e < DL; e += 2)
    *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + qrow + e) =
        bf16_pair((o[e] * wp + v[e] * ws) * inv, (o[e + 1] * wp + v[e + 1] * ws) * inv);
  if (a.lse && lane == 0) a.lse[cand * a.heads + h] = (top + log2f(sum)) * 0.6931471805599453f;
}

// Joins the parts of one row into (m, l, this lane's columns of the output): lane i brings part
// i's maximum and sum (-inf and 0 past the last), cols(i, x) reads its columns.
template <int D, typename Cols>
__device__ __forceinline__ void join_parts(float2 part, int n, const Cols& cols, float& m, float& l,
                                           float (&out)[D / 32]) {
  constexpr int DL = D / 32;
  float top = part.x;
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  const float m_new = fmaxf(m, top);
  const float wo = m == -INFINITY ? 0.f : exp2_fast(m - m_new);
  const float w = part.x == -INFINITY ? 0.f : exp2_fast(part.x - m_new);  // 0: nothing visible in the part
  float sum = part.y * w;
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
  l = l * wo + sum;
#pragma unroll
  for (int e = 0; e < DL; ++e) out[e] *= wo;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float wi = __shfl_sync(0xffffffffu, w, i);
    float x[DL];
    cols(i, x);
#pragma unroll
    for (int e = 0; e < DL; ++e) out[e] = fmaf(wi, x[e], out[e]);
  }
  m = m_new;
}
template <int DL>
__device__ __forceinline__ void read_cols(const float* p, float (&x)[DL]) {
#pragma unroll
  for (int e = 0; e < DL; e += 2) {
    const float2 v = *reinterpret_cast<const float2*>(p + e);
    x[e] = v.x;
    x[e + 1] = v.y;
  }
}

// Shared memory of the cluster's block `rank`: the address of the same object there, and loads.
__device__ __forceinline__ uint32_t at_rank(const void* p, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(ptx::smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ float2 remote_float2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}

// M groups of 8 rows.
template <int D, int M>
__global__ void __launch_bounds__(kScoreThreads, 2)
    k_score_rows(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const __grid_constant__ ScoreArgs a) {
  using C = SCfg<D>;
  constexpr int kRows = 8 * M;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t s_full[kScoreStages], s_empty[kScoreStages];
  __shared__ int s_abort;
  __shared__ float2 s_ml[kScoreWarps][kRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &s_abort;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kScoreStages; ++i) {
      ptx::mbar_init(s_full + i, 1);
      ptx::mbar_init(s_empty + i, kScoreWarps);
    }
    s_abort = 0;
    ptx::fence_barrier_init();
  }
  __syncthreads();

  ScoreItem it;
  {
    const int x = a.cluster > 0 ? blockIdx.x / a.cluster : blockIdx.x, i = upper_index(a.item_start, a.n_req, x);
    it.b = a.req0 + i;
    it.cand0 = a.cand_start[i];
    const int G = a.heads / a.kv_heads;
    it.nsplit = a.cluster > 0 ? 1 : n_splits(a, request_tiles(a, it.b));
    const int local = x - a.item_start[i];
    it.split = local % it.nsplit;
    it.hk = local / it.nsplit % a.kv_heads;
    it.rb = local / it.nsplit / a.kv_heads;
    it.rows = min(kRows, (a.cand_start[i + 1] - a.cand_start[i]) * G - it.rb * kRows);
  }
  const long long hist0 = a.hist_off[it.b];
  const int hist_len = a.hist_len[it.b];
  const int tiles = request_tiles(a, it.b);
  // the block's run of key tiles: an item of its own, or its share of the cluster's
  const int rank = a.cluster > 0 ? blockIdx.x % a.cluster : 0;
  const int tile0 = a.cluster > 0 ? tiles * rank / a.cluster : it.split * a.chunk_tiles;
  const int tile1 = a.cluster > 0 ? tiles * (rank + 1) / a.cluster : min(tiles, tile0 + a.chunk_tiles);
  const int G = a.heads / a.kv_heads;

  if (warp == kScoreWarps) {
    if (lane == 0) {
      int k = 0;  // tiles loaded
      for (; tile0 + k < tile1; ++k) {
        const int t = tile0 + k, st = k % kScoreStages;
        const uint32_t ph = (k / kScoreStages) & 1;
        if (!bounded_wait(s_empty + st, ph ^ 1, abort_flag, a.status, kScoreWaitNs)) break;
        ptx::mbar_arrive_expect_tx(s_full + st, 2 * kOperand);
        uint8_t* kb = sm + st * 2 * kOperand;
        const int y = (int)(hist0 + (long long)t * C::kKeys);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          ptx::tma_load_2d(kb + c * C::kSlab, &tm_k, it.hk * D + c * 64, y, s_full + st);
          ptx::tma_load_2d(kb + kOperand + c * C::kSlab, &tm_v, it.hk * D + c * 64, y, s_full + st);
        }
      }
      // the last copies land before the stages take the warps' outputs and the block leaves (the
      // consumers may have given up on them)
      for (int j = max(0, k - kScoreStages); j < k; ++j)
        bounded_drain(s_full + j % kScoreStages, (j / kScoreStages) & 1, kScoreWaitNs / 4);
    }
  }

  const int g = lane >> 2, q = lane & 3;
  float o[M][D / 8][4], m_run[M], l_run[M];
  if (warp < kScoreWarps) {
    // rows g of each group of 8: Q' times scale log2(e), the rotation's angle from the request's
    // reference time; upper half of the A operand the bf16 rounding, lower half the rest
    uint32_t qa[M][D / 16][4];
    long long tq[M], t_lo = LLONG_MAX;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int r = it.rb * kRows + m * 8 + g;
      const bool ok = m * 8 + g < it.rows;
      const long long cand = it.cand0 + (ok ? r / G : 0);
      tq[m] = a.tc[cand];
      if (ok) t_lo = min(t_lo, tq[m]);
      const float dt = (float)(tq[m] - a.t_ref[it.b]);
      const __nv_bfloat16* src =
          static_cast<const __nv_bfloat16*>(a.q) + (cand * a.heads + it.hk * G + (ok ? r % G : 0)) * D;
#pragma unroll
      for (int s = 0; s < D / 16; ++s)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int e = 16 * s + 8 * half + 2 * q;
          float2 x = bf16x2_float(*reinterpret_cast<const uint32_t*>(src + e));
          if (a.rotate) {
            float sn, cs;
            sincosf(dt * a.omega[e / 2], &sn, &cs);
            x = make_float2(x.x * cs - x.y * sn, x.x * sn + x.y * cs);
          }
          const float f = ok ? a.scale_log2 : 0.f;
          split_pair(x.x * f, x.y * f, qa[m][s][2 * half], qa[m][s][2 * half + 1]);
        }
      m_run[m] = -INFINITY;
      l_run[m] = 0.f;
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[m][n][e] = 0.f;
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) {
      const long long u = __shfl_xor_sync(0xffffffffu, t_lo, x);
      t_lo = min(t_lo, u);
    }
    const int key0 = warp * C::kWarpKeys;  // this warp's first key of every tile
    for (int t = tile0; t < tile1; ++t) {
      const int kt = t - tile0, st = kt % kScoreStages;
      // the 64-key block of this warp's keys, and whether it needs a mask
      const int pos0 = t * C::kKeys + key0;
      const bool any = pos0 < hist_len;
      const bool masked = any && (pos0 + C::kWarpKeys > hist_len ||
                                  a.block_need[a.block_off[it.b] + pos0 / kNeedBlock] > t_lo);
      if (!bounded_wait_warp(s_full + st, (kt / kScoreStages) & 1, abort_flag, a.status, kScoreWaitNs)) break;
      if (any) {
        const uint32_t kb = ptx::smem_u32(sm + st * 2 * kOperand), vb = kb + kOperand;
        float s[M][C::kNT][4];
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int n = 0; n < C::kNT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[m][n][e] = 0.f;
#pragma unroll
        for (int n = 0; n < C::kNT; ++n) {
          const int row = key0 + n * 8 + (lane & 7);
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {  // 32 dims: four 8 x 8 matrices
            const int chunk = (c & 1) * 4 + (lane >> 3);
            uint32_t b[4];
            ldsm4(kb + (c >> 1) * C::kSlab + row * 128 + ((chunk ^ (row & 7)) << 4), b);
#pragma unroll
            for (int m = 0; m < M; ++m) {
              mma16816(s[m][n], qa[m][2 * c], b[0], b[1]);
              mma16816(s[m][n], qa[m][2 * c + 1], b[2], b[3]);
            }
          }
        }
        uint32_t pa[M][C::kNT / 2][4];  // P as the A operand: 16 keys each
#pragma unroll
        for (int m = 0; m < M; ++m) {
          float x[C::kNT][2], mx = -INFINITY;
#pragma unroll
          for (int n = 0; n < C::kNT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              x[n][e] = s[m][n][e] + s[m][n][e + 2];
              if (masked) {
                const int p = pos0 + n * 8 + 2 * q + e;
                if (p >= hist_len || a.need[hist0 + min(p, hist_len - 1)] > tq[m]) x[n][e] = -INFINITY;
              }
              mx = fmaxf(mx, x[n][e]);
            }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const float m_new = fmaxf(m_run[m], mx);
          const float m_use = m_new == -INFINITY ? 0.f : m_new;
          const float corr = exp2_fast(m_run[m] - m_use);  // 0 while nothing was visible
          m_run[m] = m_new;
          if (__any_sync(0xffffffffu, corr != 1.f)) {
            l_run[m] *= corr;
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[m][n][e] *= corr;
          }
#pragma unroll
          for (int n = 0; n < C::kNT; ++n) {
            const float p0 = exp2_fast(x[n][0] - m_use), p1 = exp2_fast(x[n][1] - m_use);
            l_run[m] += p0 + p1;
            split_pair(p0, p1, pa[m][n >> 1][2 * (n & 1)], pa[m][n >> 1][2 * (n & 1) + 1]);
          }
        }
#pragma unroll
        for (int kk = 0; kk < C::kNT / 2; ++kk) {
          const int row = key0 + kk * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {  // 16 output columns
            const int chunk = (c & 3) * 2 + (lane >> 4);
            uint32_t b[4];
            ldsm4_t(vb + (c >> 2) * C::kSlab + row * 128 + ((chunk ^ (row & 7)) << 4), b);
#pragma unroll
            for (int m = 0; m < M; ++m) {
              mma16816(o[m][2 * c], pa[m][kk], b[0], b[1]);
              mma16816(o[m][2 * c + 1], pa[m][kk], b[2], b[3]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(s_empty + st);
    }
  }
  __syncthreads();  // every tile was read: the stages now hold the warps' outputs
  float* s_o = reinterpret_cast<float*>(sm);  // [warp][row][D]
  if (warp < kScoreWarps) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      float l = l_run[m];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if (q == 0) s_ml[warp][m * 8 + g] = make_float2(m_run[m], l);
      float* dst = s_o + (warp * kRows + m * 8 + g) * D + 2 * q;
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
        *reinterpret_cast<float2*>(dst + n * 8) = make_float2(o[m][n][0] + o[m][n][2], o[m][n][1] + o[m][n][3]);
    }
  }
  __syncthreads();
  for (int r = warp; r < it.rows; r += kScoreWarps + 1) {
    float m = -INFINITY, l = 0.f, out[D / 32] = {};
    join_parts<D>(lane < kScoreWarps ? s_ml[lane][r] : make_float2(-INFINITY, 0.f), kScoreWarps,
                  [&](int i, float (&x)[D / 32]) { read_cols(s_o + (i * kRows + r) * D + lane * (D / 32), x); }, m, l, out);
    const int row = it.rb * kRows + r;
    if (a.cluster > 1) {  // over the row's first part, which this warp alone has read
      __syncwarp();
      if (lane == 0) s_ml[0][r] = make_float2(m, l);
#pragma unroll
      for (int e = 0; e < D / 32; e += 2)
        *reinterpret_cast<float2*>(s_o + r * D + lane * (D / 32) + e) = make_float2(out[e], out[e + 1]);
    } else if (a.part_ml == nullptr) {
      finish_row<D>(a, it.cand0 + row / G, it.hk * G + row % G, lane, m, l, out);
    } else {
      const long long at = (long long)blockIdx.x * kRows + r;
      if (lane == 0) a.part_ml[at] = make_float2(m, l);
#pragma unroll
      for (int e = 0; e < D / 32; ++e) a.part_o[at * D + lane * (D / 32) + e] = out[e];
    }
  }
  if (a.cluster > 1) {  // the cluster's blocks share the rows out and read one another's parts
    cluster_sync();
    for (int r = rank + a.cluster * warp; r < it.rows; r += a.cluster * (kScoreWarps + 1)) {
      float m = -INFINITY, l = 0.f, out[D / 32] = {};
      const float2 part = lane < a.cluster ? remote_float2(at_rank(&s_ml[0][r], lane)) : make_float2(-INFINITY, 0.f);
      join_parts<D>(part, a.cluster,
                    [&](int i, float (&x)[D / 32]) {
                      const uint32_t p = at_rank(s_o + r * D + lane * (D / 32), i);
#pragma unroll
                      for (int e = 0; e < D / 32; e += 2) {
                        const float2 v = remote_float2(p + 4 * e);
                        x[e] = v.x;
                        x[e + 1] = v.y;
                      }
                    },
                    m, l, out);
      const int row = it.rb * kRows + r;
      finish_row<D>(a, it.cand0 + row / G, it.hk * G + row % G, lane, m, l, out);
    }
    cluster_sync();  // no block leaves while another reads its shared memory
  }
}

// The many-row path's prologue.  Block = one work item of k_attn_tc's CAND instantiation: its
// 128 rows of Q' (rotated against the request's reference time, rounded to bf16; rows past
// the request's last are zero) packed in row order, its descriptor, and (block 0) the item
// counters.
// A candidate's angles serve all heads of the group (computed for every row the kernel took 12 us on 476
// items of head_dim 64, 8 now).
constexpr int kPackThreads = 256;
template <int D>
__global__ void __launch_bounds__(kPackThreads) k_score_pack(const __grid_constant__ ScoreArgs a, CandItem* items,
                                                    __nv_bfloat16* qp, int* counters) {
  const int x = blockIdx.x, i = upper_index(a.item_start, a.n_req, x), b = a.req0 + i;
  const int G = a.heads / a.kv_heads, tiles = request_tiles(a, b), nsplit = n_splits(a, tiles);
  const int local = x - a.item_start[i], split = local % nsplit, hk = local / nsplit % a.kv_heads;
  const int row0 = local / nsplit / a.kv_heads * kTile;
  const int rows = min(kTile, (a.cand_start[i + 1] - a.cand_start[i]) * G - row0);
  const long long cand0 = a.cand_start[i], t_ref = a.t_ref[b];
  constexpr int kChunks = D / 8;  // 16-byte pieces of a row, one per thread
  const int c = threadIdx.x % kChunks;
  long long t_lo = LLONG_MAX;
  const int c0 = row0 / G, c1 = rows > 0 ? (row0 + rows - 1) / G + 1 : c0;  // candidates with rows here
  for (int k = c0 + (int)threadIdx.x / kChunks; k < c1; k += kPackThreads / kChunks) {
    const long long cand = cand0 + k, t = a.tc[cand];
    t_lo = min(t_lo, t);
    float sn[4], cs[4];
    if (a.rotate) {
      const float dt = (float)(t - t_ref);
#pragma unroll
      for (int p = 0; p < 4; ++p) sincosf(dt * a.omega[c * 4 + p], &sn[p], &cs[p]);
    }
    for (int g = max(0, row0 - k * G); g < min(G, row0 + rows - k * G); ++g) {
      uint4 w = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                (cand * a.heads + hk * G + g) * D + c * 8);
      if (a.rotate) {
        uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const float2 f = bf16x2_float(ws[p]);
          ws[p] = bf16_pair(f.x * cs[p] - f.y * sn[p], f.x * sn[p] + f.y * cs[p]);
        }
        w = make_uint4(ws[0], ws[1], ws[2], ws[3]);
      }
      *reinterpret_cast<uint4*>(qp + ((long long)x * kTile + k * G + g - row0) * D + c * 8) = w;
    }
  }
  for (int r = rows + (int)threadIdx.x / kChunks; r < kTile; r += kPackThreads / kChunks)
    *reinterpret_cast<uint4*>(qp + ((long long)x * kTile + r) * D + c * 8) = make_uint4(0, 0, 0, 0);
  __shared__ long long s_lo[kPackThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const long long u = __shfl_xor_sync(0xffffffffu, t_lo, o);
    t_lo = min(t_lo, u);
  }
  if ((threadIdx.x & 31) == 0) s_lo[threadIdx.x >> 5] = t_lo;
  __syncthreads();
  if (threadIdx.x == 0) {
    CandItem it;
    it.hist0 = a.hist_off[b];
    it.cand0 = cand0;
    it.t_lo = s_lo[0];
    for (int i = 1; i < kPackThreads / 32; ++i) it.t_lo = min(it.t_lo, s_lo[i]);
    it.len = a.hist_len[b];
    it.row0 = row0;
    it.rows = rows;
    it.hk = hk;
    it.tile0 = split * a.chunk_tiles;
    it.n = min(tiles - it.tile0, a.chunk_tiles);
    it.block0 = a.block_off[b];
    it.pad = 0;
    items[x] = it;
  }
  if (x == 0 && threadIdx.x < 8) counters[threadIdx.x] = 0;
}

// WPR warps per output row (candidate, head), four rows' worth of warps a block: each joins a
// run of the row's parts, in the order of the key tiles, the first then joins the warps' in order.
template <int D, int WPR>
__global__ void __launch_bounds__(128) k_score_combine(const __grid_constant__ ScoreArgs a, int rows_per_item) {
  constexpr int DL = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % WPR;
  const int first = a.cand_start[0];
  const long long w = (long long)blockIdx.x * (4 / WPR) + warp / WPR;
  const bool in = w < (long long)(a.cand_start[a.n_req] - first) * a.heads;
  const int cand = first + (int)(in ? w / a.heads : 0), h = (int)(in ? w % a.heads : 0);
  float m = -INFINITY, l = 0.f, o[DL] = {};
  if (in) {
    const int i = upper_index(a.cand_start, a.n_req, cand);
    const int G = a.heads / a.kv_heads, nsplit = n_splits(a, request_tiles(a, a.req0 + i));
    const int r = (cand - a.cand_start[i]) * G + h % G, rb = r / rows_per_item;
    const long long at = ((long long)a.item_start[i] + (rb * a.kv_heads + h / G) * nsplit) * rows_per_item +
                         r % rows_per_item;
    const int s1 = nsplit * (sub + 1) / WPR;
    for (int s0 = nsplit * sub / WPR; s0 < s1; s0 += 32) {
      const int n = min(32, s1 - s0);
      const long long p = at + (long long)s0 * rows_per_item;
      join_parts<D>(lane < n ? a.part_ml[p + (long long)lane * rows_per_item] : make_float2(-INFINITY, 0.f), n,
                    [&](int k, float (&x)[DL]) {
                      read_cols(a.part_o + (p + (long long)k * rows_per_item) * D + lane * DL, x);
                    },
                    m, l, o);
    }
  }
  if constexpr (WPR > 1) {
    __shared__ float2 s_ml[4];
    __shared__ float s_o[4][D];
    if (lane == 0) s_ml[warp] = make_float2(m, l);
#pragma unroll
    for (int e = 0; e < DL; ++e) s_o[warp][lane * DL + e] = o[e];
    __syncthreads();
    if (sub != 0) return;
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < DL; ++e) o[e] = 0.f;
    join_parts<D>(lane < WPR ? s_ml[warp + lane] : make_float2(-INFINITY, 0.f), WPR,
                  [&](int k, float (&x)[DL]) { read_cols(&s_o[warp + k][lane * DL], x); }, m, l, o);
  }
  if (in) finish_row<D>(a, cand, h, lane, m, l, o);
}

// When key j becomes visible to a candidate, as the least candidate time; per 64-key block of
// a request the largest of them; the request's reference time.  A key whose type is not a user
// side one, or whose time is out of range, is never visible (and reported).
__global__ void __launch_bounds__(kNeedBlock) k_score_need(NeedArgs a) {
  const int b = upper_index(a.block_off, a.batch, blockIdx.x);
  const long long h0 = a.hist_off[b];
  const int len = a.hist_len[b];
  const int p = ((int)blockIdx.x - a.block_off[b]) * kNeedBlock + threadIdx.x;
  long long need = LLONG_MIN;
  if (p < len) {
    const long long t = a.t[h0 + p];
    const int ty = a.ty[h0 + p];
    if (t >= kTimeLimit || t <= -kTimeLimit || (unsigned)ty > 3u) {
      need = LLONG_MAX;
      set_status(a.status, REC_ATTN_ERR_DEVICE_INPUT);
    } else if (ty == REC_ATTN_CAND) {
      need = LLONG_MAX;  // candidates see no other candidate
    } else {
      if (ty == REC_ATTN_RT) need = t + 1;
      if (a.use_delay) need = max(need, t + a.delay);
    }
    a.need[h0 + p] = need;
    if (p == 0) a.t_ref[b] = t;
  }
  __shared__ long long s_max[kNeedBlock];
  s_max[threadIdx.x] = need;
  __syncthreads();
  for (int o = kNeedBlock / 2; o > 0; o >>= 1) {
    if (threadIdx.x < o) s_max[threadIdx.x] = max(s_max[threadIdx.x], s_max[threadIdx.x + o]);
    __syncthreads();
  }
  __syncthreads();
  if (threadIdx.x == 0) a.block_need[blockIdx.x] = s_max[0];
  // keys in order of visibility: a candidate then sees a prefix of the block
  s_max[threadIdx.x] = p < len ? need : LLONG_MAX;
  __syncthreads();
  const int ordered = __syncthreads_and(threadIdx.x == 0 || s_max[threadIdx.x - 1] <= s_max[threadIdx.x]);
  if (threadIdx.x == 0) a.block_ordered[blockIdx.x] = (uint8_t)(ordered != 0);
}

template <int D, int M>
cudaError_t launch_rows_t(const CUtensorMap& k, const CUtensorMap& v, const ScoreArgs& a, int items, cudaStream_t st) {
  const int smem = kScoreStages * 2 * kOperand + 1024;
  static_assert(kScoreWarps * 8 * M * D * 4 <= kScoreStages * 2 * kOperand, "the warps' outputs fit the stages");
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem(done, (const void*)k_score_rows<D, M>, smem);
  if (e != cudaSuccess) return e;
  if (a.cluster <= 1) {
    k_score_rows<D, M><<<items, kScoreThreads, smem, st>>>(k, v, a);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)items * a.cluster);
  cfg.blockDim = dim3(kScoreThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)a.cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_score_rows<D, M>, k, v, a);
}

template <int D>
cudaError_t launch_combine(const ScoreArgs& a, int rows_per_item, cudaStream_t st) {
  const long long rows = (long long)(a.cand_start[a.n_req] - a.cand_start[0]) * a.heads;
  // a warp per row where the rows alone fill the chip, else four (long histories, few rows)
  if (rows >= 4096) k_score_combine<D, 1><<<(unsigned)((rows + 3) / 4), 128, 0, st>>>(a, rows_per_item);
  else k_score_combine<D, 4><<<(unsigned)rows, 128, 0, st>>>(a, rows_per_item);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_score_pack(const ScoreArgs& a, int head_dim, int items, CandItem* desc, void* qp, int* counters,
                              cudaStream_t st) {
  __nv_bfloat16* q = static_cast<__nv_bfloat16*>(qp);
  if (head_dim == 64) k_score_pack<64><<<items, kPackThreads, 0, st>>>(a, desc, q, counters);
  else k_score_pack<128><<<items, kPackThreads, 0, st>>>(a, desc, q, counters);
  return cudaGetLastError();
}

cudaError_t launch_score_combine(const ScoreArgs& a, int head_dim, int rows_per_item, cudaStream_t st) {
  return head_dim == 64 ? launch_combine<64>(a, rows_per_item, st) : launch_combine<128>(a, rows_per_item, st);
}

int score_tile_keys(int head_dim) { return head_dim == 64 ? SCfg<64>::kKeys : SCfg<128>::kKeys; }

// Rows per block: as many groups of 8 as the registers hold without spills.
int score_rows_per_item(int head_dim, int max_rows) {
  const int most = head_dim == 64 ? 16 : 8;
  int r = 8;
  while (r < most && r < max_rows) r *= 2;
  return r;
}

cudaError_t launch_score_need(const NeedArgs& a, int blocks, cudaStream_t st) {
  if (blocks <= 0) return cudaSuccess;
  k_score_need<<<blocks, kNeedBlock, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_score_rows(const CUtensorMap& k, const CUtensorMap& v, const ScoreArgs& a, int head_dim,
                              int rows_per_item, int items, cudaStream_t st) {
  if (items <= 0) return cudaSuccess;
  const int key = head_dim * 100 + rows_per_item;
  switch (key) {
    case 6408: return launch_rows_t<64, 1>(k, v, a, items, st);
    case 6416: return launch_rows_t<64, 2>(k, v, a, items, st);
    case 12808: return launch_rows_t<128, 1>(k, v, a, items, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace recattn
