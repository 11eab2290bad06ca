// layernorm.cu -- layer norm of packed token rows with a gain and bias per token type
// (MTGR notes on the blog index page: a layer norm whose parameters belong to the token's
// kind, GroupLayerNorm) or one gain and bias for all rows, forward and backward.
//
// Row x of `width` values, group g (its token type, or 0):
//   m = mean(x), r = 1 / sqrt(mean((x - m)^2) + eps), n = (x - m) r, y = n w[g] + b[g]
// and for the upstream gradient dy, with u = dy w[g]:
//   dx = r (u - mean(u) - n mean(u n)),  dw[g] = sum dy n,  db[g] = sum dy  (rows of g).
//
// Both directions are bound by HBM: every row is read once and written once.  A row is held in the
// registers of `tpr` threads, two 16-byte chunks each, so the variance is the mean of squared
// differences from the mean itself and the backward recomputes both statistics from the row it
// reads anyway.  The backward takes two reductions a row: {sum x, sum u}, then {sum (x - m)^2,
// sum u (x - m)}.  320016 rows of 512 bf16 by type: forward 111 us (5.9 TB/s, 88% of a copy's rate),
// backward 177 us (5.5 TB/s; without types 161); backward of 50001 rows of 1408 fp32: 149 us (5.7 TB/s).
// Farther from HBM's rate are rows of more than 256 threads, of which a block holds one, its two
// reductions' barriers exposed (20000 x 8192 bf16: 168 and 239 us; 10000 x 16384, whose backward spills
// at the 64 registers of 1024 threads: 206 and 741 us; 98 and 147 at a copy's rate), and short rows, half
// of whose chunks are empty at 64 values (1000000 x 64 by type: 68 and 103 us; 38 and 57).
// Statistics, sums and gradients of the gains are fp32; outputs are rounded once.
#include <cuda_bf16.h>

#include <algorithm>
#include <map>
#include <mutex>
#include <tuple>

#include "launchers.cuh"

namespace recattn {

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormMaxSmem = 160 * 1024;  // 128 KB of rows or sums at the widest

// Pairs of fp32 for the packed instructions (fma.rn.f32x2 and its kin: two values an issue).
using f2 = unsigned long long;
__device__ __forceinline__ f2 pair(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 both(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ float total(f2 v) {
  const float2 r = both(v);
  return r.x + r.y;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

template <typename E>
struct Vec;  // a 16-byte chunk: kN values, as pairs
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4 v, f2* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ uint4 pack(const f2* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = both(x[i]);
      const __nv_bfloat162 p = __floats2bfloat162_rn(v.x, v.y);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const uint4 v, f2* x) {
    x[0] = pair(__uint_as_float(v.x), __uint_as_float(v.y));
    x[1] = pair(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  static __device__ __forceinline__ uint4 pack(const f2* x) {
    const float2 a = both(x[0]), b = both(x[1]);
    return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
  }
};

// The threads of one row: LANES (8 or 16) neighbouring lanes, or with LANES = 32 whole warps.
template <int LANES>
struct RowGroup {
  int tpr, lane, id, warps;  // tpr: threads per row; lane: thread within the row; id: row group within the block
  float2* red;               // [2][warps] of this group (rows of more than one warp)
  int buf;
  __device__ __forceinline__ void init(int threads_per_row, float2* s_red) {
    tpr = LANES < 32 ? LANES : threads_per_row;
    lane = threadIdx.x % tpr;
    id = threadIdx.x / tpr;
    warps = LANES < 32 ? 1 : tpr / 32;
    red = s_red + id * 2 * warps;
    buf = 0;
  }
  // Sums over the row's threads, to every thread: of a and b, or of a alone.
  __device__ __forceinline__ float2 sum2(float a, float b) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    return warps == 1 ? make_float2(a, b) : across(make_float2(a, b));
  }
  __device__ __forceinline__ float sum1(float a) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    return warps == 1 ? a : across(make_float2(a, 0.f)).x;
  }
  __device__ __forceinline__ float2 across(float2 v) {
    float2* r = red + buf * warps;
    buf ^= 1;  // the next reduction writes the other half: one barrier each suffices
    if ((lane & 31) == 0) r[lane >> 5] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(tpr) : "memory");
    float2 t = r[0];
    for (int w = 1; w < warps; ++w) {
      t.x += r[w].x;
      t.y += r[w].y;
    }
    return t;
  }
};

template <int N>
__device__ __forceinline__ void load_gain(const float* p, f2* x) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
    x[i / 2] = pair(v.x, v.y);
    x[i / 2 + 1] = pair(v.z, v.w);
  }
}

// Where a thread stands in a row: its chunks are lane, lane + tpr, ... and `act` those that the
// row has (FULL: all of them, so no test remains).
template <int NV, bool FULL>
struct Chunks {
  bool act[NV];
  __device__ __forceinline__ void init(int lane, int tpr, int chunks) {
#pragma unroll
    for (int i = 0; i < NV; ++i) act[i] = FULL || i * tpr + lane < chunks;
  }
  __device__ __forceinline__ bool has(int i) const { return FULL || act[i]; }
};

// Rows on their way: each thread copies its own chunks into its own slots of shared memory,
// NS - 1 rows ahead (cp.async), and reads them back itself, so no barrier is needed and no
// register holds them meanwhile.
__device__ __forceinline__ void copy16(void* smem, const void* global) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(global)
               : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// The types of a group's rows r0, r0 + stride, ...: the group's lanes (of each warp) hold the next
// LANES of them, loaded together, so a row's type costs a shuffle and no wait on memory.
template <int LANES>
struct RowTypes {
  const int8_t* ty;
  int held, k;
  __device__ __forceinline__ void init(const int8_t* types) {
    ty = types;
    held = 0;
    k = LANES;
  }
  // The type of row r (0 without types, -1 past `last`); r goes up by stride from call to call.
  __device__ __forceinline__ int next(int r, int stride, int last) {
    if (!ty) return 0;
    if (k == LANES) {
      const int mine = r + (int)(threadIdx.x & (LANES - 1)) * stride;
      held = mine < last ? ty[mine] : -1;
      k = 0;
    }
    return __shfl_sync(0xffffffffu, held, k++, LANES);
  }
};

// Forward.  Block k takes the contiguous rows [k R, (k + 1) R), its groups in turn, and keeps
// the gain and bias of its columns in registers while the type stays the same (a request's
// types come in a few runs; read for every row they would fill the L1 pipe).  With whole warps
// per row each group walks its own rows; groups within a warp walk together, `in` false past the
// end (their lanes take part in shuffles).  A row whose type is outside 0..3 belongs to no group:
// its output (or gradient) is zero.
template <typename E, int NV, int LANES, bool FULL, int THREADS, int NS>
__global__ void __launch_bounds__(THREADS, THREADS > 256 ? 1 : 2) k_layernorm_fwd(NormArgs a) {
  constexpr int N = Vec<E>::kN, EPT = NV * N;
  __shared__ float2 s_red[64];
  extern __shared__ uint4 s_rows[];  // [NS][NV][threads]
  RowGroup<LANES> g;
  g.init(a.tpr, s_red);
  const int groups = blockDim.x / g.tpr, chunks = a.width / N;
  Chunks<NV, FULL> ch;
  ch.init(g.lane, g.tpr, chunks);
  const float inv_w = 1.f / (float)a.width;
  const long long first = (long long)blockIdx.x * a.rows_per_block;
  const int last = (int)min(first + a.rows_per_block, a.rows);
  int left = last - (int)first;  // rows from the block's (whole warps: the group's) next on
  if (LANES == 32) left -= g.id;
  const int lead = LANES == 32 ? 0 : g.id;  // the row is in while left > lead
  const int step = groups * chunks;
  const uint4* const px = static_cast<const uint4*>(a.x);
  uint4* const py = static_cast<uint4*>(a.y);
  long long at = (first + g.id) * chunks + g.lane;
  int r = (int)first + g.id;
  int slot = 0, ahead_left = left;
  long long ahead = at;  // the next row to copy
  auto copy = [&]() {
    if (ahead_left > lead) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (ch.has(i)) copy16(s_rows + (slot * NV + i) * blockDim.x + threadIdx.x, px + ahead + i * g.tpr);
    }
    copies_end();
    slot = slot + 1 == NS ? 0 : slot + 1;
    ahead += step;
    ahead_left -= groups;
  };
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) copy();
  RowTypes<LANES> types;
  types.init(a.ty);
  f2 w[EPT / 2], b[EPT / 2];
#pragma unroll
  for (int e = 0; e < EPT / 2; ++e) w[e] = b[e] = 0ull;
  int cur = -1, here = 0;
  for (; left > 0; left -= groups, at += step, r += groups) {
    copy();
    const int ty = types.next(r, groups, last);
    const bool in = left > lead, ok = (unsigned)ty <= 3u;
    if (ok && ty != cur) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!ch.has(i)) continue;
        const long long col = (long long)ty * a.width + (i * g.tpr + g.lane) * N;
        load_gain<N>(a.w + col, w + i * (N / 2));
        if (a.b) load_gain<N>(a.b + col, b + i * (N / 2));
      }
      cur = ty;
    }
    copies_wait<NS - 1>();
    f2 x[EPT / 2];
#pragma unroll
    for (int i = 0; i < NV; ++i) Vec<E>::unpack(s_rows[(here * NV + i) * blockDim.x + threadIdx.x], x + i * (N / 2));
    here = here + 1 == NS ? 0 : here + 1;
    f2 s = 0ull;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!ch.has(i)) continue;
#pragma unroll
      for (int e = i * (N / 2); e < (i + 1) * (N / 2); ++e) s = add2(s, x[e]);
    }
    const float mean = g.sum1(total(s)) * inv_w;
    f2 q = 0ull;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!ch.has(i)) continue;
#pragma unroll
      for (int e = i * (N / 2); e < (i + 1) * (N / 2); ++e) {
        x[e] = add2(x[e], pair(-mean, -mean));
        q = fma2(x[e], x[e], q);
      }
    }
    const float rstd = rsqrtf(g.sum1(total(q)) * inv_w + a.eps);
    if (LANES < 32 && !in) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!ch.has(i)) continue;
      f2 y[N / 2];
#pragma unroll
      for (int e = 0; e < N / 2; ++e) {
        const int k = i * (N / 2) + e;
        y[e] = fma2(mul2(x[k], pair(rstd, rstd)), w[k], b[k]);
      }
      __stcs(py + at + i * g.tpr, ok ? Vec<E>::pack(y) : make_uint4(0, 0, 0, 0));
    }
  }
}

// Four sums into a thread's own slot: stored the first time, added afterwards (without waiting
// for the old value; one thread's operations on an address happen in its order).
__device__ __forceinline__ void slot_put(float* p, f2 a, f2 b, bool add) {
  const float2 x = both(a), y = both(b);
  if (add)
    asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(x.x), "f"(x.y), "f"(y.x),
                 "f"(y.y) : "memory");
  else
    *reinterpret_cast<float4*>(p) = make_float4(x.x, x.y, y.x, y.y);
}

// Backward.  Block k takes the contiguous rows [k R, (k + 1) R), its groups in turn, and
// keeps the gains and the gains' gradients of its columns in registers while the type stays the
// same (a request's types come in a few runs).  When the type changes, a group adds what it
// holds to a slot of its own in a.flush; at the end the block sums its groups, type by type,
// into its row of a.part.  k_layernorm_dw then sums the blocks.  Every sum has a fixed order, so
// the gradients do not change from call to call.
template <typename E, int NV, int LANES, bool FULL, int THREADS, int NS>
__global__ void __launch_bounds__(THREADS, THREADS > 256 ? 1 : sizeof(E) == 2 ? 2 : 3) k_layernorm_bwd(NormArgs a) {
  constexpr int N = Vec<E>::kN, EPT = NV * N;
  __shared__ float2 s_red[64];
  __shared__ int s_open[32];                  // per group: the type it still holds (-1: none)
  __shared__ unsigned s_flushed[32];          // per group: types with sums in its slot
  extern __shared__ float s_sum[];            // [groups][2][width]: open sums
  RowGroup<LANES> g;
  g.init(a.tpr, s_red);
  const int groups = blockDim.x / g.tpr, chunks = a.width / N;
  Chunks<NV, FULL> ch;
  ch.init(g.lane, g.tpr, chunks);
  const float inv_w = 1.f / (float)a.width;
  f2 w[EPT / 2], dw[EPT / 2], db[EPT / 2];
#pragma unroll
  for (int e = 0; e < EPT / 2; ++e) w[e] = dw[e] = db[e] = 0ull;
  int cur = -1;
  unsigned flushed = 0;
  // the type changes: what is held goes to the group's slot, the new type's gains come in
  auto change = [&](int ty) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!ch.has(i)) continue;
      const int col = (i * g.tpr + g.lane) * N;
      if (cur >= 0) {
        float* p = a.flush + (((long long)blockIdx.x * groups + g.id) * 4 + cur) * 2 * a.width + col;
        const bool add = (flushed >> cur) & 1u;
#pragma unroll
        for (int e = 0; e < N / 2; e += 2) {
          slot_put(p + 2 * e, dw[i * (N / 2) + e], dw[i * (N / 2) + e + 1], add);
          slot_put(p + a.width + 2 * e, db[i * (N / 2) + e], db[i * (N / 2) + e + 1], add);
        }
#pragma unroll
        for (int e = 0; e < N / 2; ++e) dw[i * (N / 2) + e] = db[i * (N / 2) + e] = 0ull;
      }
      load_gain<N>(a.w + (long long)ty * a.width + col, w + i * (N / 2));
    }
    if (cur >= 0) flushed |= 1u << cur;
    cur = ty;
  };
  const long long first = (long long)blockIdx.x * a.rows_per_block;
  const int last = (int)min(first + a.rows_per_block, a.rows);
  int left = last - (int)first;
  if (LANES == 32) left -= g.id;
  const int lead = LANES == 32 ? 0 : g.id;
  const int step = groups * chunks;
  // one running offset for x, dy and dx (their bases stay in constant memory)
  const uint4* const px = static_cast<const uint4*>(a.x);
  const uint4* const py = static_cast<const uint4*>(a.dy);
  uint4* const pd = static_cast<uint4*>(a.dx);
  long long at = (first + g.id) * chunks + g.lane;
  int r = (int)first + g.id;
  uint4* const s_rows = reinterpret_cast<uint4*>(s_sum);  // [NS][x, dy][NV][threads], before the sums
  int slot = 0, ahead_left = left;
  long long ahead = at;  // the next row to copy
  auto copy = [&]() {
    if (ahead_left > lead) {
      uint4* const s = s_rows + slot * 2 * NV * blockDim.x + threadIdx.x;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (ch.has(i)) {
          copy16(s + i * blockDim.x, px + ahead + i * g.tpr);
          copy16(s + (NV + i) * blockDim.x, py + ahead + i * g.tpr);
        }
    }
    copies_end();
    slot = slot + 1 == NS ? 0 : slot + 1;
    ahead += step;
    ahead_left -= groups;
  };
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) copy();
  int here = 0;  // the slot of this row
  RowTypes<LANES> types;
  types.init(a.ty);
  for (; left > 0; left -= groups, at += step, r += groups) {
    copy();
    const bool in = left > lead;
    const int ty = in || a.ty ? types.next(r, groups, last) : -1;
    const bool ok = (unsigned)ty <= 3u;
    copies_wait<NS - 1>();
    f2 x[EPT / 2], dy[EPT / 2];
    const uint4* const s_row = s_rows + here * 2 * NV * blockDim.x + threadIdx.x;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Vec<E>::unpack(s_row[i * blockDim.x], x + i * (N / 2));
      Vec<E>::unpack(s_row[(NV + i) * blockDim.x], dy + i * (N / 2));
    }
    here = here + 1 == NS ? 0 : here + 1;
    if (ok && ty != cur) change(ty);
    f2 s = 0ull, su = 0ull;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!ch.has(i)) continue;
#pragma unroll
      for (int e = i * (N / 2); e < (i + 1) * (N / 2); ++e) {
        s = add2(s, x[e]);
        su = fma2(dy[e], w[e], su);
      }
    }
    const float2 t1 = g.sum2(total(s), total(su));
    const float mean = t1.x * inv_w, mu = t1.y * inv_w;
    f2 q = 0ull, ux = 0ull;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!ch.has(i)) continue;
#pragma unroll
      for (int e = i * (N / 2); e < (i + 1) * (N / 2); ++e) {
        x[e] = add2(x[e], pair(-mean, -mean));
        q = fma2(x[e], x[e], q);
        ux = fma2(mul2(dy[e], w[e]), x[e], ux);
      }
    }
    const float2 t2 = g.sum2(total(q), total(ux));
    const float rstd = rsqrtf(t2.x * inv_w + a.eps);
    const float mun = t2.y * inv_w * rstd;  // mean of u n
    if (LANES < 32 && !in) continue;
    if (!ok) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (ch.has(i)) __stcs(pd + at + i * g.tpr, make_uint4(0, 0, 0, 0));
      continue;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!ch.has(i)) continue;
      f2 d[N / 2];
#pragma unroll
      for (int e = 0; e < N / 2; ++e) {
        const int k = i * (N / 2) + e;
        const f2 n = mul2(x[k], pair(rstd, rstd));
        d[e] = mul2(fma2(n, pair(-mun, -mun), fma2(dy[k], w[k], pair(-mu, -mu))), pair(rstd, rstd));
        dw[k] = fma2(dy[k], n, dw[k]);
        db[k] = add2(db[k], dy[k]);
      }
      __stcs(pd + at + i * g.tpr, Vec<E>::pack(d));
    }
  }
  copies_wait<0>();
  __syncthreads();  // the rows' slots are read: the sums take their place
  // the block's sums, type by type: each group's slot, then what it still holds
  if (g.lane == 0) {
    s_open[g.id] = cur;
    s_flushed[g.id] = flushed;
  }
  if (cur >= 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!ch.has(i)) continue;
#pragma unroll
      for (int e = 0; e < N / 2; ++e) {
        float* p = s_sum + g.id * 2 * a.width + (i * g.tpr + g.lane) * N + 2 * e;
        *reinterpret_cast<float2*>(p) = both(dw[i * (N / 2) + e]);
        *reinterpret_cast<float2*>(p + a.width) = both(db[i * (N / 2) + e]);
      }
    }
  }
  __syncthreads();  // slots (global) and open sums (shared) of every group are written
  const int n_types = a.ty ? 4 : 1;
  unsigned seen = 0;
  for (int k = 0; k < groups; ++k) seen |= s_flushed[k] | (s_open[k] >= 0 ? 1u << s_open[k] : 0u);
  if (threadIdx.x == 0) a.seen[blockIdx.x] = seen;
  // four columns of one type at a time, the slots of eight groups read together
  const int cols4 = 2 * a.width / 4;
  for (int x = threadIdx.x; x < n_types * cols4; x += blockDim.x) {
    const int t = x / cols4, c = x - t * cols4;
    if (!((seen >> t) & 1u)) continue;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < groups; k0 += 8) {
      float4 u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = k0 + i;
        u[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k < groups && ((s_flushed[k] >> t) & 1u))
          u[i] = __ldcg(reinterpret_cast<const float4*>(
                            a.flush + (((long long)blockIdx.x * groups + k) * 4 + t) * 2 * a.width) + c);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = k0 + i;
        if (k < groups && s_open[k] == t) {
          const float4 o = reinterpret_cast<const float4*>(s_sum + k * 2 * a.width)[c];
          u[i].x += o.x; u[i].y += o.y; u[i].z += o.z; u[i].w += o.w;
        }
        v.x += u[i].x; v.y += u[i].y; v.z += u[i].z; v.w += u[i].w;
      }
    }
    reinterpret_cast<float4*>(a.part + ((long long)blockIdx.x * n_types + t) * 2 * a.width)[c] = v;
  }
}

// Sums of the blocks' rows: 32 columns of one type's {dw | db} per block, 32 threads a column
// over the blocks k, k + 32, ...
__global__ void __launch_bounds__(1024) k_layernorm_dw(NormArgs a, int blocks) {
  __shared__ float s[32][33];
  const int types = a.ty ? 4 : 1, t = blockIdx.y;
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
  float v = 0.f;
  if (c < 2 * a.width)
#pragma unroll 4
    for (int k = part; k < blocks; k += 32)
      if ((a.seen[k] >> t) & 1u) v += a.part[((long long)k * types + t) * 2 * a.width + c];
  s[part][threadIdx.x & 31] = v;
  __syncthreads();
  if (part != 0 || c >= 2 * a.width) return;
#pragma unroll
  for (int p = 1; p < 32; ++p) v += s[p][threadIdx.x];
  if (c < a.width) {
    if (a.dw) a.dw[(long long)t * a.width + c] = v;
  } else if (a.db) {
    a.db[(long long)t * a.width + c - a.width] = v;
  }
}

// Two 16-byte chunks of a row per thread (four for rows of more than 32 KB), the threads
// rounded up to a power of two of at least 8 (within a warp; so a block has at most 32 rows at
// a time) or to whole warps.
struct NormShape {
  int nv, tpr, threads, groups;
  bool full;  // every thread has all its chunks
  // rows on their way per thread, this one included.  Two: with three or four the backward
  // of 320016 x 512 bf16 without types took 183 and 187 us instead of 165, the forward 112 and 120 instead of 112
  int ns;
  int rows_smem(bool bwd) const { return ns * nv * threads * 16 * (bwd ? 2 : 1); }
};
NormShape norm_shape(int width, int dtype) {
  const int chunks = width * (dtype == REC_ATTN_BF16 ? 2 : 4) / 16;
  NormShape s;
  s.nv = chunks > 2048 ? 4 : 2;
  const int n = (chunks + s.nv - 1) / s.nv;
  if (n > 32) {
    s.tpr = (n + 31) / 32 * 32;
  } else {
    s.tpr = 8;
    while (s.tpr < n) s.tpr *= 2;
  }
  s.threads = s.tpr <= kNormThreads ? kNormThreads / s.tpr * s.tpr : s.tpr;
  s.groups = s.threads / s.tpr;
  s.full = chunks == s.nv * s.tpr;
  s.ns = s.nv > 2 ? 1 : 2;
  return s;
}

using NormKernel = void (*)(NormArgs);
template <typename E, int NV, int LANES, bool FULL, int THREADS, int NS>
NormKernel norm_dir(bool bwd) {
  return bwd ? k_layernorm_bwd<E, NV, LANES, FULL, THREADS, NS> : k_layernorm_fwd<E, NV, LANES, FULL, THREADS, NS>;
}
template <typename E>
NormKernel norm_kernel(const NormShape& s, bool bwd) {
  if constexpr (sizeof(E) == 4)  // (the widest bf16 rows are 32 KB)
    if (s.nv > 2) return norm_dir<E, 4, 32, false, 1024, 1>(bwd);
  if (s.threads > 512) return norm_dir<E, 2, 32, false, 1024, 2>(bwd);
  if (s.threads > kNormThreads) return norm_dir<E, 2, 32, false, 512, 2>(bwd);
  if (s.tpr == 8) return norm_dir<E, 2, 8, false, kNormThreads, 2>(bwd);
  if (s.tpr == 16) return norm_dir<E, 2, 16, false, kNormThreads, 2>(bwd);
  return s.full ? norm_dir<E, 2, 32, true, kNormThreads, 2>(bwd) : norm_dir<E, 2, 32, false, kNormThreads, 2>(bwd);
}
NormKernel norm_kernel(const NormShape& s, int dtype, bool bwd) {
  return dtype == REC_ATTN_BF16 ? norm_kernel<__nv_bfloat16>(s, bwd) : norm_kernel<float>(s, bwd);
}

// Blocks of a kernel that an SM of the current device holds (asked once per device, kernel and
// shape; one that cannot be asked counts as 1, and its failure shows at the launch).
int blocks_per_sm(NormKernel fn, int threads, int smem) {
  static std::mutex mu;
  static std::map<std::tuple<int, NormKernel, int, int>, int> known;
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  std::lock_guard<std::mutex> lk(mu);
  const auto key = std::make_tuple(dev, fn, threads, smem);
  const auto at = known.find(key);
  if (at != known.end()) return at->second;
  const OutsideCapture now;
  // one limit for every shape of a kernel
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormMaxSmem) != cudaSuccess) return 1;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, threads, smem) != cudaSuccess || n < 1) return 1;
  try {
    known[key] = n;
  } catch (...) {  // asked again by the next call
  }
  return n;
}

}  // namespace

// Contiguous runs of rows, one per resident block, in whole turns of the block's groups.
static void split_rows(long long rows, int groups, long long places, int* blocks, long long* rows_per_block) {
  const long long turns = (rows + groups - 1) / groups, n = turns < places ? turns : places;
  *rows_per_block = (turns + n - 1) / n * groups;
  *blocks = (int)((rows + *rows_per_block - 1) / *rows_per_block);
}

cudaError_t launch_layernorm_fwd(NormArgs a, int dtype, int num_sms, cudaStream_t st) {
  if (a.rows <= 0) return cudaSuccess;
  const NormShape s = norm_shape(a.width, dtype);
  a.tpr = s.tpr;
  const NormKernel fn = norm_kernel(s, dtype, false);
  int blocks = 0;
  split_rows(a.rows, s.groups, (long long)num_sms * blocks_per_sm(fn, s.threads, s.rows_smem(false)), &blocks,
             &a.rows_per_block);
  fn<<<blocks, s.threads, s.rows_smem(false), st>>>(a);
  return cudaGetLastError();
}

NormBwdPlan layernorm_bwd_plan(long long rows, int width, int dtype, bool by_type, int num_sms) {
  NormBwdPlan p;
  const NormShape s = norm_shape(width, dtype);
  p.smem = std::max(s.groups * 2 * width * (int)sizeof(float), s.rows_smem(true));
  split_rows(rows, s.groups, (long long)num_sms * blocks_per_sm(norm_kernel(s, dtype, true), s.threads, p.smem),
             &p.blocks, &p.rows_per_block);
  const int types = by_type ? 4 : 1;
  p.off_part = ((size_t)p.blocks * sizeof(unsigned) + 255) & ~(size_t)255;
  p.off_flush = p.off_part + (size_t)p.blocks * types * 2 * width * sizeof(float);
  p.bytes = p.off_flush + (by_type ? (size_t)p.blocks * s.groups * 4 * 2 * width * sizeof(float) : 0);
  return p;
}

cudaError_t launch_layernorm_bwd(NormArgs a, const NormBwdPlan& p, void* ws, int dtype, cudaStream_t st) {
  const NormShape s = norm_shape(a.width, dtype);
  a.tpr = s.tpr;
  a.rows_per_block = p.rows_per_block;
  char* w = static_cast<char*>(ws);
  a.seen = reinterpret_cast<unsigned*>(w);
  a.part = reinterpret_cast<float*>(w + p.off_part);
  a.flush = a.ty ? reinterpret_cast<float*>(w + p.off_flush) : nullptr;
  norm_kernel(s, dtype, true)<<<p.blocks, s.threads, p.smem, st>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((2 * a.width + 31) / 32), a.ty ? 4u : 1u);
  k_layernorm_dw<<<grid, 1024, 0, st>>>(a, p.blocks);
  return cudaGetLastError();
}

}  // namespace recattn
