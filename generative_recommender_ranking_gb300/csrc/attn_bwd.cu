// attn_bwd.cu -- backward pass of the masked time-RoPE softmax attention on the CUDA
// cores (fp32 inputs, head_dim 32 or 64; the bf16 path runs on the tensor cores:
// attn_bwd_tc.cu).
//
// Gradients of O = Softmax(QK^T/sqrt(d) + M) V (TM20K review page, section 2.1;
// LazFormer review page, Eq. 19-21) through the time-RoPE (CADET review page, time
// encoding): with P the forward probabilities, rebuilt from the forward's
// log-sum-exp as P_ij = exp(s_ij - lse_i) on visible pairs,
//   dV_j = sum_i P_ij dO_i,  dP_ij = <dO_i, V_j>,  D_i = <dO_i, O_i>,
//   dS_ij = P_ij (dP_ij - D_i),  dQ'_i = scale sum_j dS_ij K'_j,  dK'_j = scale sum_i dS_ij Q'_i,
// and dQ = R(t_i)^T dQ', dK = R(t_j)^T dK' (the rotation is orthogonal).
//
// Kernels over the planner's tile lists, so SKIP tiles cost nothing here either; the products are of
// 64 x 64 tiles in registers (simt_tile.cuh):
//   k_bwd_delta   D_i per (token, head);
//   k_bwd_dq      a block per (half query tile, head), over the query tile's non-SKIP key tiles;
//   k_bwd_dkv     a block per (half key tile, key/value head or part of its query heads), over the
//                 query tiles whose class against this key tile is not SKIP;
//   k_bwd_kv_add  with parts: their sums, in order.
// FULL tiles skip the mask; PARTIAL tiles take the plan's mask table, or without a slot evaluate it.  Rows with no visible key (lse = -inf)
// contribute nothing.  Bound by the fp32 units and the shared memory that feeds them (k_bwd_dkv at
// head_dim 64: one block per SM).  Forward and backward of 16 causal requests of 400 to 700 tokens,
// 8 query and 2 key/value heads, head_dim 64: 1080 us, dQ 352 and dK/dV 462 of it (a thread per row: 2306);
// of one request of 700 tokens, 8 and 1 heads: 283 us (2742, whose dK/dV had six blocks).
#include "attn_common.cuh"
#include "launchers.cuh"
#include "simt_tile.cuh"

namespace recattn {

namespace {

// The request of global tile g (binary search over the request table).
__device__ __forceinline__ int tile_request(const ReqMeta* meta, int batch, long long g) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (meta[mid].tile_start <= g) lo = mid;
    else hi = mid;
  }
  return lo;
}

// A thread's N = D / 16 gradient columns of one row, turned back by dt (R(t)^T y over adjacent
// pairs, the inverse of the prologue's rotation), to global memory.
template <int D>
__device__ __forceinline__ void store_grad(float* dst, float (&y)[D / 16], bool rotate, float dt, const float* omega) {
#pragma unroll
  for (int p = 0; p < D / 32; ++p) {
    if (rotate) {
      float sn, cs;
      sincosf(dt * omega[p], &sn, &cs);
      const float u = y[2 * p], w = y[2 * p + 1];
      y[2 * p] = u * cs + w * sn;
      y[2 * p + 1] = -u * sn + w * cs;
    }
    *reinterpret_cast<float2*>(dst + 2 * p) = make_float2(y[2 * p], y[2 * p + 1]);
  }
}
template <int N>
__device__ __forceinline__ void row_of(const simt::f2 (&o)[2][N], int i, float (&y)[N]) {
#pragma unroll
  for (int c = 0; c < N; ++c) {
    const float2 v = simt::both(o[i >> 1][c]);
    y[c] = (i & 1) ? v.y : v.x;
  }
}

// 16 bytes of dO and O a thread.
template <int D>
__global__ void __launch_bounds__(256) k_bwd_delta(BwdArgs a) {
  constexpr int kLanes = D / 4;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x, r = i / kLanes;  // (token, head) row
  float acc = 0.f;
  if (r < a.rows) {
    const float4 x = static_cast<const float4*>(a.dout)[i], y = static_cast<const float4*>(a.out)[i];
    acc = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, x.w * y.w)));
  }
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (r < a.rows && i % kLanes == 0) a.delta[r] = acc;
}

template <int D>
struct DqSmem {
  __align__(16) float q[D * simt::kB], go[D * simt::kB];   // transposed; q times the scale
  __align__(16) float k[D * simt::kB], v[D * simt::kB];    // transposed
  __align__(16) float kr[simt::kB * D];
  __align__(16) float ds[simt::kB * simt::kB];
  simt::Tokens tq, tk;
};
template <int D>
struct DkvSmem {
  __align__(16) float k[D * simt::kB], v[D * simt::kB];    // transposed
  __align__(16) float q[D * simt::kB], go[D * simt::kB];   // transposed; q times the scale
  __align__(16) float qr[simt::kB * D], gor[simt::kB * D];
  __align__(16) float p[simt::kB * simt::kB], ds[simt::kB * simt::kB];
  simt::Tokens tq, tk;
  float lse[simt::kB], dlt[simt::kB];
};

// dQ: block = (half of query tile g, head h); thread (ty, tx) has query rows 4 ty ...
template <int D>
__global__ void __launch_bounds__(simt::kThreads) k_bwd_dq(BwdArgs a) {
  using namespace simt;
  constexpr int N = D / 16;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  DqSmem<D>& sm = *reinterpret_cast<DqSmem<D>*>(smem_raw);
  const long long x = gridDim.x - 1 - blockIdx.x;  // (under causal masks the heaviest first)
  const long long g = x / kPerTile;
  const int h = blockIdx.y, H = a.heads, Hk = H / a.group, hk = h / a.group;
  const int b = tile_request(a.meta, a.batch, g);
  const ReqMeta m = a.meta[b];
  const int qt = (int)(g - m.tile_start), pos0 = qt * kTile + (int)(x % kPerTile) * kB;
  if (pos0 >= m.len) return;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const long long tok0 = m.tok_start + pos0, q0 = (tok0 * H + h) * D;
  load_tile<D>(static_cast<const float*>(a.q) + q0, (long long)H * D, m.len - pos0, a.scale, sm.q, nullptr);
  load_tile<D>(static_cast<const float*>(a.dout_attn) + q0, (long long)H * D, m.len - pos0, 1.f, sm.go, nullptr);
  sm.tq.load(a.t, a.ty, tok0, pos0, m.len, a.mask.delay);
  float lse[4], dlt[4];
  bool live[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int pi = pos0 + 4 * ty + i;
    const long long row = (tok0 + 4 * ty + i) * H + h;
    // a pruned query has no output: no gradient
    const bool kept = pi < m.len && query_kept(a.ty[tok0 + 4 * ty + i], pi, a.qkeep[b]);
    lse[i] = kept ? a.lse[row] : -INFINITY;
    dlt[i] = kept ? a.delta[row] : 0.f;
    live[i] = lse[i] != -INFINITY;
  }
  f2 acc[2][N];
#pragma unroll
  for (int c = 0; c < N; ++c) acc[0][c] = acc[1][c] = pair(0.f, 0.f);
  const int n = a.kcount[g];
  const uint32_t* list = a.klist + m.cls_start + (long long)qt * m.ntiles;
  const int* slots = a.kslot + m.cls_start + (long long)qt * m.ntiles;
  // steps of 64 keys; those past the request's end are left out
  const int steps = n * kPerTile;
  auto key_of = [&](int j) { return (int)(list[j / kPerTile] & 0xffffffu) * kTile + j % kPerTile * kB; };
  auto next = [&](int j) {
    while (j < steps && key_of(j) >= m.len) ++j;
    return j;
  };
  Rows<D> nk, nv;
  auto fetch = [&](int j) {
    const int key0 = key_of(j);
    const long long src = ((m.tok_start + key0) * Hk + hk) * D;
    nk.fetch(static_cast<const float*>(a.k) + src, (long long)Hk * D, m.len - key0);
    nv.fetch(static_cast<const float*>(a.v) + src, (long long)Hk * D, m.len - key0);
  };
  int j = next(0);
  if (j < steps) fetch(j);
  while (j < steps) {
    const int key0 = key_of(j);
    const bool full = (int)(list[j / kPerTile] >> 24) == REC_ATTN_TILE_FULL;
    const int slot = full ? -1 : slots[j / kPerTile];  // of the mask table
    __syncthreads();  // the last step's operands were read
    nk.put(1.f, sm.k, sm.kr);
    nv.put(1.f, sm.v, nullptr);
    if (!full && slot < 0) sm.tk.load(a.t, a.ty, m.tok_start + key0, key0, m.len, 0);
    __syncthreads();
    j = next(j + 1);
    if (j < steps) fetch(j);
    f2 s[2][4], dp[2][4];
#pragma unroll
    for (int c = 0; c < 4; ++c) s[0][c] = s[1][c] = dp[0][c] = dp[1][c] = pair(0.f, 0.f);
    scores<D>(sm.q, sm.k, ty, tx, s);
    scores<D>(sm.go, sm.v, ty, tx, dp);
    float x4[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float si[4], di[4];
      row_of<4>(s, i, si);
      row_of<4>(dp, i, di);
      const uint32_t bits = slot >= 0 ? table_bits(a.mtab, slot, pos0 % kTile + 4 * ty + i, (key0 % kTile >> 2) + tx) : 15u;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const bool vis = live[i] && (bits >> c & 1u) &&
                         (full || slot >= 0 || visible(a.mask, sm.tq, 4 * ty + i, sm.tk, 4 * tx + c));
        x4[i][c] = vis ? __expf(si[c] - lse[i]) * (di[c] - dlt[i]) * a.scale : 0.f;
      }
    }
    store_scores(sm.ds, ty, tx, x4);
    __syncthreads();
    accumulate<D>(sm.ds, sm.kr, ty, tx, acc);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int pi = pos0 + 4 * ty + i;
    if (pi >= m.len) break;
    float y[N];
    row_of<N>(acc, i, y);
    store_grad<D>(static_cast<float*>(a.dq) + q0 + (long long)(4 * ty + i) * H * D + N * tx, y, a.rotate != 0,
                  (float)(a.t[m.tok_start + pi] - a.t[m.tok_start]), a.omega + N / 2 * tx);
  }
}

// dK, dV: block = (half of key tile g, key/value head and part of its query heads); thread (ty, tx)
// has key rows 4 ty ...  The part's query heads one after the other.
template <int D>
__global__ void __launch_bounds__(simt::kThreads) k_bwd_dkv(BwdArgs a) {
  using namespace simt;
  constexpr int N = D / 16;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  DkvSmem<D>& sm = *reinterpret_cast<DkvSmem<D>*>(smem_raw);
  const long long g = blockIdx.x / kPerTile;
  const int H = a.heads, Hk = H / a.group, reps = a.group / a.parts, hk = (int)blockIdx.y / a.parts;
  const int b = tile_request(a.meta, a.batch, g);
  const ReqMeta m = a.meta[b];
  const int kt = (int)(g - m.tile_start), pos0 = kt * kTile + (int)(blockIdx.x % kPerTile) * kB;
  if (pos0 >= m.len) return;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const long long tok0 = m.tok_start + pos0, k0 = (tok0 * Hk + hk) * D;
  load_tile<D>(static_cast<const float*>(a.k) + k0, (long long)Hk * D, m.len - pos0, 1.f, sm.k, nullptr);
  load_tile<D>(static_cast<const float*>(a.v) + k0, (long long)Hk * D, m.len - pos0, 1.f, sm.v, nullptr);
  sm.tk.load(a.t, a.ty, tok0, pos0, m.len, 0);
  f2 dk[2][N], dv[2][N];
#pragma unroll
  for (int c = 0; c < N; ++c) dk[0][c] = dk[1][c] = dv[0][c] = dv[1][c] = pair(0.f, 0.f);
  const uint8_t* col = a.cls + m.cls_start + kt;  // column kt of the request's class matrix
  // steps of 64 queries of one head; SKIP tiles and those past the request's end are left out
  const int halves = m.ntiles * kPerTile, steps = reps * halves;
  auto next = [&](int it) {
    while (it < steps) {
      const int half = it % halves;
      if (half * kB < m.len && col[(long long)(half / kPerTile) * m.ntiles] != REC_ATTN_TILE_SKIP) break;
      ++it;
    }
    return it;
  };
  Rows<D> nq, ngo;
  float nl = 0.f, nd = 0.f;  // the step's row constants: the first kB threads'
  auto fetch = [&](int it) {
    const int h = (int)blockIdx.y * reps + it / halves, query0 = it % halves * kB;
    const long long qtok = m.tok_start + query0, src = (qtok * H + h) * D;
    nq.fetch(static_cast<const float*>(a.q) + src, (long long)H * D, m.len - query0);
    ngo.fetch(static_cast<const float*>(a.dout_attn) + src, (long long)H * D, m.len - query0);
    const int c = threadIdx.x, pi = query0 + c;
    // pruned queries give no gradient, nor do queries that see no key
    const bool kept = c < kB && pi < m.len && query_kept(a.ty[qtok + c], pi, a.qkeep[b]);
    nl = kept ? a.lse[(qtok + c) * H + h] : -INFINITY;
    nd = kept ? a.delta[(qtok + c) * H + h] : 0.f;
  };
  int it = next(0);
  if (it < steps) fetch(it);
  while (it < steps) {
    const int query0 = it % halves * kB, qt = query0 / kTile;
    const bool full = col[(long long)qt * m.ntiles] == REC_ATTN_TILE_FULL;
    const int in_table = full ? -1 : a.pslot[m.cls_start + (long long)qt * m.ntiles + kt];
    const int slot = in_table < a.mcap ? in_table : -1;  // of the mask table
    __syncthreads();  // the last step's operands were read
    nq.put(a.scale, sm.q, sm.qr);
    ngo.put(1.f, sm.go, sm.gor);
    if (!full && slot < 0) sm.tq.load(a.t, a.ty, m.tok_start + query0, query0, m.len, a.mask.delay);
    if (threadIdx.x < kB) {
      sm.lse[threadIdx.x] = nl;
      sm.dlt[threadIdx.x] = nd;
    }
    __syncthreads();
    it = next(it + 1);
    if (it < steps) fetch(it);
    f2 s[2][4], dp[2][4];
#pragma unroll
    for (int c = 0; c < 4; ++c) s[0][c] = s[1][c] = dp[0][c] = dp[1][c] = pair(0.f, 0.f);
    scores<D>(sm.k, sm.q, ty, tx, s);
    scores<D>(sm.v, sm.go, ty, tx, dp);
    float p[4][4], x[4][4];
    uint32_t bits[4];  // of each query's keys
#pragma unroll
    for (int c = 0; c < 4; ++c)
      bits[c] = slot >= 0 ? table_bits(a.mtab, slot, query0 % kTile + 4 * tx + c, (pos0 % kTile >> 2) + ty) : 15u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float si[4], di[4];
      row_of<4>(s, i, si);
      row_of<4>(dp, i, di);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float lse = sm.lse[4 * tx + c];
        const bool vis = lse != -INFINITY && (bits[c] >> i & 1u) &&
                         (full || slot >= 0 || visible(a.mask, sm.tq, 4 * tx + c, sm.tk, 4 * ty + i));
        p[i][c] = vis ? __expf(si[c] - lse) : 0.f;
        x[i][c] = p[i][c] * (di[c] - sm.dlt[4 * tx + c]);  // (sm.q carries the scale)
      }
    }
    store_scores(sm.p, ty, tx, p);
    store_scores(sm.ds, ty, tx, x);
    __syncthreads();
    accumulate<D>(sm.p, sm.gor, ty, tx, dv);
    accumulate<D>(sm.ds, sm.qr, ty, tx, dk);
  }
  const long long T = a.rows / H, n_part = (long long)Hk * a.parts * T * D;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int pj = pos0 + 4 * ty + i;
    if (pj >= m.len) break;
    float yk[N], yv[N];
    row_of<N>(dk, i, yk);
    row_of<N>(dv, i, yv);
    if (a.kv_part) {  // the part's sums as they are
      float* dst = a.kv_part + ((long long)blockIdx.y * T + m.tok_start + pj) * D + N * tx;
      store_grad<D>(dst, yk, false, 0.f, a.omega);
      store_grad<D>(dst + n_part, yv, false, 0.f, a.omega);
    } else {
      const long long at = k0 + (long long)(4 * ty + i) * Hk * D + N * tx;
      store_grad<D>(static_cast<float*>(a.dk) + at, yk, a.rotate != 0,
                    (float)(a.t[m.tok_start + pj] - a.t[m.tok_start]), a.omega + N / 2 * tx);
      store_grad<D>(static_cast<float*>(a.dv) + at, yv, false, 0.f, a.omega);
    }
  }
}

// The parts' sums in order; dK is turned back.  A thread has two columns of a token and key/value head.
template <int D>
__global__ void __launch_bounds__(256) k_bwd_kv_add(BwdArgs a) {
  const int Hk = a.heads / a.group;
  const long long T = a.rows / a.heads, n_part = (long long)Hk * a.parts * T * D;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= T * Hk * (D / 2)) return;
  const int c = (int)(i % (D / 2)), hk = (int)(i / (D / 2) % Hk);
  const long long tok = i / (D / 2) / Hk;
  const float* src = a.kv_part + ((long long)hk * a.parts * T + tok) * D + 2 * c;
  float k0 = 0.f, k1 = 0.f, v0 = 0.f, v1 = 0.f;
  for (int p = 0; p < a.parts; ++p) {
    const float2 k = *reinterpret_cast<const float2*>(src + (long long)p * T * D);
    const float2 v = *reinterpret_cast<const float2*>(src + (long long)p * T * D + n_part);
    k0 += k.x; k1 += k.y;
    v0 += v.x; v1 += v.y;
  }
  if (a.rotate) {
    int lo = 0, hi = a.batch;  // the token's request
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.meta[mid].tok_start <= tok) lo = mid;
      else hi = mid;
    }
    float sn, cs;
    sincosf((float)(a.t[tok] - a.t[a.meta[lo].tok_start]) * a.omega[c], &sn, &cs);
    const float u = k0;
    k0 = u * cs + k1 * sn;
    k1 = -u * sn + k1 * cs;
  }
  const long long at = (tok * Hk + hk) * D + 2 * c;
  *reinterpret_cast<float2*>(static_cast<float*>(a.dk) + at) = make_float2(k0, k1);
  *reinterpret_cast<float2*>(static_cast<float*>(a.dv) + at) = make_float2(v0, v1);
}

template <int D>
cudaError_t launch_delta_t(const BwdArgs& a, cudaStream_t st) {
  if (a.rows <= 0) return cudaSuccess;
  k_bwd_delta<D><<<(unsigned)((a.rows * (D / 4) + 255) / 256), 256, 0, st>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_bwd_t(const BwdArgs& a, long long n_tiles, cudaStream_t st) {
  if (n_tiles <= 0) return cudaSuccess;
  static std::atomic<unsigned long long> done_q{0}, done_kv{0};
  cudaError_t e = allow_smem(done_q, (const void*)k_bwd_dq<D>, (int)sizeof(DqSmem<D>));
  if (e == cudaSuccess) e = allow_smem(done_kv, (const void*)k_bwd_dkv<D>, (int)sizeof(DkvSmem<D>));
  if (e != cudaSuccess) return e;
  const unsigned halves = (unsigned)(n_tiles * simt::kPerTile);
  k_bwd_dq<D><<<dim3(halves, (unsigned)a.heads), simt::kThreads, sizeof(DqSmem<D>), st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int Hk = a.heads / a.group;
  k_bwd_dkv<D><<<dim3(halves, (unsigned)(Hk * a.parts)), simt::kThreads, sizeof(DkvSmem<D>), st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || !a.kv_part) return e;
  const long long threads = a.rows / a.heads * Hk * (D / 2);
  k_bwd_kv_add<D><<<(unsigned)((threads + 255) / 256), 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_bwd_delta(const BwdArgs& a, int head_dim, cudaStream_t st) {
  if (head_dim == 32) return launch_delta_t<32>(a, st);
  if (head_dim == 64) return launch_delta_t<64>(a, st);
  return cudaErrorInvalidValue;
}

cudaError_t launch_attn_bwd_simt(const BwdArgs& a, int head_dim, long long n_tiles, cudaStream_t st) {
  if (head_dim == 32) return launch_bwd_t<32>(a, n_tiles, st);
  if (head_dim == 64) return launch_bwd_t<64>(a, n_tiles, st);
  return cudaErrorInvalidValue;
}

}  // namespace recattn
