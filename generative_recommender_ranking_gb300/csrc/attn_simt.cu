// attn_simt.cu -- fp32 masked softmax attention on the CUDA cores (fp32 inputs and
// outputs; tensor-core TF32 would not hold 1e-4 against the fp64 reference).
//
// Softmax(QK^T/sqrt(d) + M) V (TM20K review page, section 2.1; LazFormer review
// page, Eq. 19-21) over the plan's non-SKIP key tiles, an online softmax in fp32 with expf.
// A block takes half a query tile (64 rows) of one head and the keys 64 at a time: S as a
// product of 64 x 64 tiles in registers, P through shared memory to the product with V
// (simt_tile.cuh).  Bound by the fp32 units and the shared memory that feeds them: 16 causal
// requests of 400 to 700 tokens, 8 query and 2 key/value heads, head_dim 64, 212 us against 63 of the
// units alone (a thread per query row, reading every key element for one multiplication: 451; three
// blocks an SM with fewer registers, which spill: 232); head_dim 32: 136 us.
// PARTIAL tiles take the plan's mask table, or without a slot evaluate the mask per element; FULL
// tiles skip it.
#include "attn_common.cuh"
#include "launchers.cuh"
#include "simt_tile.cuh"

namespace recattn {

namespace {

template <int D>
struct FwdSmem {
  __align__(16) float q[D * simt::kB];  // transposed, times the scale
  __align__(16) float k[D * simt::kB];  // transposed
  __align__(16) float v[simt::kB * D];
  __align__(16) float p[simt::kB * simt::kB];
  simt::Tokens tq, tk;
};

// One block's rows; false, with nothing written, when an output is not finite and HIDE is off.  HIDE: the
// pairs that the mask hides are left out of the product with V instead of weighted with 0.
template <int D, bool HIDE>
__device__ __forceinline__ bool attend(const AttnArgs& a) {
  using namespace simt;
  constexpr int N = D / 16;
  extern __shared__ __align__(16) unsigned char smem[];
  FwdSmem<D>& sm = *reinterpret_cast<FwdSmem<D>*>(smem);
  const WorkItem it = decode_item(a, blockIdx.x / kPerTile, true);  // (the heaviest first)
  if (it.n < 0) return true;  // every query of the tile is pruned
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int pos0 = it.qt * kTile + (int)(blockIdx.x % kPerTile) * kB;
  if (pos0 >= it.m.len) return true;
  const int H = a.heads, Hk = H / a.group, hk = it.h / a.group;
  const long long tok0 = it.m.tok_start + pos0;
  load_tile<D>(static_cast<const float*>(a.q) + (tok0 * H + it.h) * D, (long long)H * D, it.m.len - pos0, a.scale, sm.q, nullptr);
  sm.tq.load(a.t, a.ty, tok0, pos0, it.m.len, a.mask.delay);
  if (a.mask.keep_user >= 0) {  // pruned queries may hold anything (some Q' is never written): zeros
    __syncthreads();
    const int r = threadIdx.x >> 2;
    if (pos0 + r < it.m.len && !query_kept(sm.tq.ty[r], pos0 + r, it.keep))
      for (int d = threadIdx.x & 3; d < D; d += 4) sm.q[at(r >> 2, d) + (r & 3)] = 0.f;
  }
  f2 o[2][N];
  float m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
  }
#pragma unroll
  for (int j = 0; j < N; ++j) o[0][j] = o[1][j] = pair(0.f, 0.f);
  // steps of 64 keys; those past the request's end are left out
  const int steps = it.n * kPerTile;
  auto key_of = [&](int j) { return (int)(it.list[j / kPerTile] & 0xffffffu) * kTile + j % kPerTile * kB; };
  auto next = [&](int j) {
    while (j < steps && key_of(j) >= it.m.len) ++j;
    return j;
  };
  Rows<D> nk, nv;
  auto fetch = [&](int j) {
    const int key0 = key_of(j);
    const long long src = ((it.m.tok_start + key0) * Hk + hk) * D;
    nk.fetch(static_cast<const float*>(a.k) + src, (long long)Hk * D, it.m.len - key0);
    nv.fetch(static_cast<const float*>(a.v) + src, (long long)Hk * D, it.m.len - key0);
  };
  int j = next(0);
  if (j < steps) fetch(j);
  while (j < steps) {
    const int key0 = key_of(j);
    const bool full = (int)(it.list[j / kPerTile] >> 24) == REC_ATTN_TILE_FULL;
    const int slot = full ? -1 : it.slots[j / kPerTile];  // of the mask table
    __syncthreads();  // the last step's operands were read
    nk.put(1.f, sm.k, nullptr);
    nv.put(1.f, nullptr, sm.v);
    if (!full && slot < 0) sm.tk.load(a.t, a.ty, it.m.tok_start + key0, key0, it.m.len, 0);
    __syncthreads();
    j = next(j + 1);
    if (j < steps) fetch(j);
    f2 s[2][4];
#pragma unroll
    for (int c = 0; c < 4; ++c) s[0][c] = s[1][c] = pair(0.f, 0.f);
    scores<D>(sm.q, sm.k, ty, tx, s);
    float x[4][4];
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const float2 v = both(s[p][c]);
        x[2 * p][c] = v.x;
        x[2 * p + 1][c] = v.y;
      }
    float corr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (slot >= 0) {
        const uint32_t bits = table_bits(a.mtab, slot, pos0 % kTile + 4 * ty + i, (key0 % kTile >> 2) + tx);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (!(bits >> c & 1u)) x[i][c] = -INFINITY;
      } else if (!full) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (!visible(a.mask, sm.tq, 4 * ty + i, sm.tk, 4 * tx + c)) x[i][c] = -INFINITY;
      }
      const float mx = row_max(fmaxf(fmaxf(x[i][0], x[i][1]), fmaxf(x[i][2], x[i][3])));
      const float m_new = fmaxf(m[i], mx), m_use = m_new == -INFINITY ? 0.f : m_new;
      corr[i] = expf(m[i] - m_use);  // 0 while nothing was visible
      m[i] = m_new;
      l[i] *= corr[i];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float p = expf(x[i][c] - m_use);
        l[i] += p;  // this thread's columns; summed over the row at the end
        x[i][c] = HIDE && x[i][c] == -INFINITY ? kHidden : p;
      }
    }
    store_scores(sm.p, ty, tx, x);
#pragma unroll
    for (int c = 0; c < N; ++c)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const float2 v = both(o[p][c]);
        o[p][c] = pair(v.x * corr[2 * p], v.y * corr[2 * p + 1]);
      }
    __syncthreads();
    if constexpr (HIDE) accumulate_seen<D>(sm.p, sm.v, ty, tx, o);
    else accumulate<D>(sm.p, sm.v, ty, tx, o);
  }
  bool finite = true;
#pragma unroll
  for (int c = 0; c < N; ++c)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const float2 v = both(o[p][c]);
      finite = finite && fabsf(v.x) < INFINITY && fabsf(v.y) < INFINITY;
    }
  // (the barrier also serves an item without a key: the query rows' types are there)
  if (__syncthreads_or(!finite) && !HIDE) return false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ty + i, pi = pos0 + r;
    const float sum = row_sum(l[i]);
    if (pi >= it.m.len || !query_kept(sm.tq.ty[r], pi, it.keep)) continue;
    const long long row = (tok0 + r) * H + it.h;
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    float* dst = static_cast<float*>(a.out) + row * D + N * tx;
    // the attention output gate, O * sigmoid(g)
    const float* g = a.out_gate ? static_cast<const float*>(a.out_gate) + row * D + N * tx : nullptr;
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const float2 v = both(o[i >> 1][c]);
      const float y = ((i & 1) ? v.y : v.x) * inv;
      dst[c] = g ? y * sigmoid_io<float>(g[c]) : y;
    }
    if (a.lse && tx == 0) a.lse[row] = sum > 0.f ? m[i] + logf(sum) : -INFINITY;
  }
  return true;
}

// Not inlined: rare, and its registers would be taken from the usual pass.
template <int D>
__device__ __noinline__ void attend_hiding(const AttnArgs& a) {
  attend<D, true>(a);
}

// A value that is not finite is to reach the rows that see its key alone, but 0 times it is NaN: a block
// whose outputs are not all finite computes them once more, which costs the others nothing.
template <int D>
__global__ void __launch_bounds__(simt::kThreads, 2) k_attn_simt(const __grid_constant__ AttnArgs a) {
  if (!attend<D, false>(a)) attend_hiding<D>(a);
}

template <int D>
cudaError_t launch(const AttnArgs& a, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  const int smem = (int)sizeof(FwdSmem<D>);
  const cudaError_t e = allow_smem(done, (const void*)k_attn_simt<D>, smem);
  if (e != cudaSuccess) return e;
  k_attn_simt<D><<<(unsigned)(a.n_items * simt::kPerTile), simt::kThreads, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_simt(const AttnArgs& a, int head_dim, cudaStream_t st) {
  if (a.n_items <= 0) return cudaSuccess;
  switch (head_dim) {
    case 32: return launch<32>(a, st);
    case 64: return launch<64>(a, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace recattn
