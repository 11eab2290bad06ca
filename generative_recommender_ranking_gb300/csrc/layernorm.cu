// layernorm.cu -- layer norm of packed token rows with a gain and bias per token type
// (MTGR notes on the blog index page: a layer norm whose parameters belong to the token's
// kind, GroupLayerNorm) or one gain and bias for all rows, forward and backward.
//
// Row x of `width` values, group g (its token type, or 0):
//   m = mean(x), r = 1 / sqrt(mean((x - m)^2) + eps), n = (x - m) r, y = n w[g] + b[g]
// and for the upstream gradient dy, with u = dy w[g]:
//   dx = r (u - mean(u) - n mean(u n)),  dw[g] = sum dy n,  db[g] = sum dy  (rows of g).
//
// Both directions are bound by HBM: every row is read once and written once.  A row is
// held in the registers of `tpr` threads, two 16-byte chunks each, so the variance is the mean of squared differences from the mean itself and
// the backward recomputes both statistics from the row it reads anyway.  The backward takes
// two reductions a row: {sum x, sum u}, then {sum (x - m)^2, sum u (x - m)}.
// Statistics, sums and gradients of the gains are fp32; outputs are rounded once.
#include <cuda_bf16.h>

#include "launchers.cuh"

namespace recattn {

namespace {

constexpr int kNormThreads = 256;

template <typename E>
struct Vec;  // a 16-byte chunk
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4 v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const uint4 v, float* x) {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};

// The threads of one row: a power of two from 8 to 32, or a multiple of 32.
struct RowGroup {
  int tpr, lane, id, warps;  // tpr: threads per row; lane: thread within the row; id: row group within the block
  float2* red;               // [2][warps] of this group (rows of more than one warp)
  int buf;
  __device__ __forceinline__ void init(int threads_per_row, float2* s_red) {
    tpr = threads_per_row;
    lane = threadIdx.x % tpr;
    id = threadIdx.x / tpr;
    warps = tpr > 32 ? tpr / 32 : 1;
    red = s_red + id * 2 * warps;
    buf = 0;
  }
  // Sums over the row's threads, to every thread: of a and b, or of a alone.
  __device__ __forceinline__ float2 sum2(float a, float b) {
    for (int o = min(tpr, 32) >> 1; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    return warps == 1 ? make_float2(a, b) : across(make_float2(a, b));
  }
  __device__ __forceinline__ float sum1(float a) {
    for (int o = min(tpr, 32) >> 1; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
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
__device__ __forceinline__ void load_gain(const float* p, float* x) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
    x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
  }
}

// A row's 16-byte chunks lane, lane + tpr, ... (zeros past the row or for no row).
template <typename E, int NV>
__device__ __forceinline__ void load_row(const void* base, long long row, bool in, int width, int chunks,
                                         const RowGroup& g, uint4 (&raw)[NV]) {
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const E*>(base) + (in ? row : 0) * width);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = i * g.tpr + g.lane;
    raw[i] = in && c < chunks ? __ldcs(src + c) : make_uint4(0, 0, 0, 0);
  }
}

// A block's groups take consecutive rows in turn; the next row's chunks are loaded before
// this row's reductions.  A row whose type is outside 0..3 belongs to no group: its output (or
// gradient) is zero.
template <typename E, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) k_layernorm_fwd(NormArgs a) {
  constexpr int N = Vec<E>::kN, EPT = NV * N;
  __shared__ float2 s_red[64];
  RowGroup g;
  g.init(a.tpr, s_red);
  const int groups = blockDim.x / a.tpr, chunks = a.width / N;
  const float inv_w = 1.f / (float)a.width;
  const long long stride = (long long)gridDim.x * groups;
  long long row = (long long)blockIdx.x * groups + g.id;
  uint4 next[NV];
  load_row<E, NV>(a.x, row, row < a.rows, a.width, chunks, g, next);
  // whole warps run every iteration (rows past the end are loaded as zeros and not stored)
  for (long long r0 = (long long)blockIdx.x * groups; r0 < a.rows; r0 += stride, row += stride) {
    const bool in = row < a.rows;
    float x[EPT];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) Vec<E>::unpack(next[i], x + i * N);
    load_row<E, NV>(a.x, row + stride, row + stride < a.rows, a.width, chunks, g, next);
    const int ty = in && a.ty ? a.ty[row] : 0;
#pragma unroll
    for (int e = 0; e < EPT; ++e) s += x[e];
    const float mean = g.sum1(s) * inv_w;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i * a.tpr + g.lane >= chunks) continue;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        x[i * N + e] -= mean;
        q = fmaf(x[i * N + e], x[i * N + e], q);
      }
    }
    const float rstd = rsqrtf(g.sum1(q) * inv_w + a.eps);
    if (!in) continue;
    const bool ok = (unsigned)ty <= 3u;
    const float* w = a.w + (long long)(ok ? ty : 0) * a.width;
    const float* b = a.b ? a.b + (long long)(ok ? ty : 0) * a.width : nullptr;
    uint4* dst = reinterpret_cast<uint4*>(static_cast<E*>(a.y) + row * a.width);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * a.tpr + g.lane;
      if (c >= chunks) continue;
      float wv[N], bv[N], y[N];
      load_gain<N>(w + c * N, wv);
      if (b) load_gain<N>(b + c * N, bv);
#pragma unroll
      for (int e = 0; e < N; ++e) y[e] = ok ? fmaf(x[i * N + e] * rstd, wv[e], b ? bv[e] : 0.f) : 0.f;
      __stcs(dst + c, Vec<E>::pack(y));
    }
  }
}

// Backward.  Block k takes the contiguous rows [k R, (k + 1) R), its groups in turn, and
// keeps the gains and the gains' gradients of its columns in registers while the type stays the
// same (a request's types come in a few runs).  When the type changes, a group adds what it
// holds to a slot of its own in a.flush; at the end the block sums its groups, type by type,
// into its row of a.part.  k_layernorm_dw then sums the blocks.  Every sum has a fixed order, so
// the gradients do not change from call to call.
template <typename E, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) k_layernorm_bwd(NormArgs a) {
  constexpr int N = Vec<E>::kN, EPT = NV * N;
  __shared__ float2 s_red[64];
  __shared__ int s_open[32];                  // per group: the type it still holds (-1: none)
  __shared__ unsigned s_flushed[32];          // per group: types with sums in its slot
  extern __shared__ float s_sum[];            // [groups][2][width]: open sums
  RowGroup g;
  g.init(a.tpr, s_red);
  const int groups = blockDim.x / a.tpr, chunks = a.width / N;
  const float inv_w = 1.f / (float)a.width;
  float w[EPT], dw[EPT], db[EPT];
#pragma unroll
  for (int e = 0; e < EPT; ++e) w[e] = dw[e] = db[e] = 0.f;
  int cur = -1;
  unsigned flushed = 0;
  float* slots = a.flush ? a.flush + ((long long)blockIdx.x * groups + g.id) * 4 * 2 * a.width : nullptr;
  // the type changes: what is held goes to the group's slot, the new type's gains come in
  auto change = [&](int ty) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * a.tpr + g.lane;
      if (c >= chunks) continue;
      if (cur >= 0) {
        float* p = slots + (long long)cur * 2 * a.width + c * N;
        const bool add = (flushed >> cur) & 1u;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          p[e] = add ? p[e] + dw[i * N + e] : dw[i * N + e];
          p[a.width + e] = add ? p[a.width + e] + db[i * N + e] : db[i * N + e];
          dw[i * N + e] = db[i * N + e] = 0.f;
        }
      }
      load_gain<N>(a.w + (long long)ty * a.width + c * N, w + i * N);
    }
    if (cur >= 0) flushed |= 1u << cur;
    cur = ty;
  };
  const long long first = (long long)blockIdx.x * a.rows_per_block;
  const long long last = min(first + a.rows_per_block, a.rows);
  long long row = first + g.id;
  uint4 nx[NV], ny[NV];
  load_row<E, NV>(a.x, row, row < last, a.width, chunks, g, nx);
  load_row<E, NV>(a.dy, row, row < last, a.width, chunks, g, ny);
  int nty = row < last ? (a.ty ? a.ty[row] : 0) : -1;
  for (long long r0 = first; r0 < last; r0 += groups, row += groups) {
    const bool in = row < last;
    float x[EPT], dy[EPT];
    const int ty = nty;
    const bool ok = (unsigned)ty <= 3u;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Vec<E>::unpack(nx[i], x + i * N);
      Vec<E>::unpack(ny[i], dy + i * N);
    }
    {
      const long long nr = row + groups;
      load_row<E, NV>(a.x, nr, nr < last, a.width, chunks, g, nx);
      load_row<E, NV>(a.dy, nr, nr < last, a.width, chunks, g, ny);
      nty = nr < last ? (a.ty ? a.ty[nr] : 0) : -1;
    }
    if (ok && ty != cur) change(ty);
    float s = 0.f, su = 0.f;
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
      s += x[e];
      su = fmaf(dy[e], w[e], su);
    }
    const float2 t1 = g.sum2(s, su);
    const float mean = t1.x * inv_w, mu = t1.y * inv_w;
    float q = 0.f, ux = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i * a.tpr + g.lane >= chunks) continue;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int k = i * N + e;
        x[k] -= mean;
        q = fmaf(x[k], x[k], q);
        ux = fmaf(dy[k] * w[k], x[k], ux);
      }
    }
    const float2 t2 = g.sum2(q, ux);
    const float rstd = rsqrtf(t2.x * inv_w + a.eps);
    const float mun = t2.y * inv_w * rstd;  // mean of u n
    if (!in) continue;
    uint4* dst = reinterpret_cast<uint4*>(static_cast<E*>(a.dx) + row * a.width);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * a.tpr + g.lane;
      if (c >= chunks) continue;
      float d[N];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int k = i * N + e;
        const float n = x[k] * rstd;
        d[e] = ok ? rstd * (fmaf(dy[k], w[k], -mu) - n * mun) : 0.f;
        if (ok) {
          dw[k] = fmaf(dy[k], n, dw[k]);
          db[k] += dy[k];
        }
      }
      __stcs(dst + c, Vec<E>::pack(d));
    }
  }
  // the block's sums, type by type: each group's slot, then what it still holds
  if (g.lane == 0) {
    s_open[g.id] = cur;
    s_flushed[g.id] = flushed;
  }
  if (cur >= 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * a.tpr + g.lane;
      if (c >= chunks) continue;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        s_sum[(g.id * 2 + 0) * a.width + c * N + e] = dw[i * N + e];
        s_sum[(g.id * 2 + 1) * a.width + c * N + e] = db[i * N + e];
      }
    }
  }
  __syncthreads();  // slots (global) and open sums (shared) of every group are written
  const int types = a.ty ? 4 : 1;
  unsigned seen = 0;
  for (int k = 0; k < groups; ++k) seen |= s_flushed[k] | (s_open[k] >= 0 ? 1u << s_open[k] : 0u);
  if (threadIdx.x == 0) a.seen[blockIdx.x] = seen;
  for (int t = 0; t < types; ++t) {
    if (!((seen >> t) & 1u)) continue;
    float* out = a.part + ((long long)blockIdx.x * types + t) * 2 * a.width;
    for (int c = threadIdx.x; c < 2 * a.width; c += blockDim.x) {
      float v = 0.f;
      for (int k = 0; k < groups; ++k) {
        if ((s_flushed[k] >> t) & 1u)
          v += a.flush[(((long long)blockIdx.x * groups + k) * 4 + t) * 2 * a.width + c];
        if (s_open[k] == t) v += s_sum[k * 2 * a.width + c];
      }
      out[c] = v;
    }
  }
}

// Sums of the blocks' rows: 32 columns of one type's {dw | db} per block, eight threads a
// column over the blocks k, k + 8, ...
__global__ void __launch_bounds__(256) k_layernorm_dw(NormArgs a, int blocks) {
  __shared__ float s[8][33];
  const int types = a.ty ? 4 : 1, t = blockIdx.y;
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
  float v = 0.f;
  if (c < 2 * a.width)
    for (int k = part; k < blocks; k += 8)
      if ((a.seen[k] >> t) & 1u) v += a.part[((long long)k * types + t) * 2 * a.width + c];
  s[part][threadIdx.x & 31] = v;
  __syncthreads();
  if (part != 0 || c >= 2 * a.width) return;
  for (int p = 1; p < 8; ++p) v += s[p][threadIdx.x];
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
  return s;
}

using NormKernel = void (*)(NormArgs);
template <typename E>
NormKernel norm_kernel(const NormShape& s, bool bwd) {
  if (s.nv > 2) return bwd ? k_layernorm_bwd<E, 4, 1024> : k_layernorm_fwd<E, 4, 1024>;
  if (s.threads > 512) return bwd ? k_layernorm_bwd<E, 2, 1024> : k_layernorm_fwd<E, 2, 1024>;
  if (s.threads > kNormThreads && s.threads <= 512) return bwd ? k_layernorm_bwd<E, 2, 512> : k_layernorm_fwd<E, 2, 512>;
  return bwd ? k_layernorm_bwd<E, 2, kNormThreads> : k_layernorm_fwd<E, 2, kNormThreads>;
}
NormKernel norm_kernel(const NormShape& s, int dtype, bool bwd) {
  return dtype == REC_ATTN_BF16 ? norm_kernel<__nv_bfloat16>(s, bwd) : norm_kernel<float>(s, bwd);
}

}  // namespace

cudaError_t launch_layernorm_fwd(NormArgs a, int dtype, int num_sms, cudaStream_t st) {
  if (a.rows <= 0) return cudaSuccess;
  const NormShape s = norm_shape(a.width, dtype);
  a.tpr = s.tpr;
  const long long need = (a.rows + s.groups - 1) / s.groups, cap = (long long)num_sms * (2048 / s.threads);
  norm_kernel(s, dtype, false)<<<(unsigned)(need < cap ? need : cap), s.threads, 0, st>>>(a);
  return cudaGetLastError();
}

NormBwdPlan layernorm_bwd_plan(long long rows, int width, int dtype, bool by_type, int num_sms) {
  NormBwdPlan p;
  const NormShape s = norm_shape(width, dtype);
  const long long need = (rows + s.groups - 1) / s.groups, cap = (long long)num_sms * (s.threads > kNormThreads ? 1 : 2);
  p.blocks = (int)(need < cap ? need : cap);
  p.rows_per_block = (rows + p.blocks - 1) / p.blocks;
  p.rows_per_block = (p.rows_per_block + s.groups - 1) / s.groups * s.groups;
  p.blocks = (int)((rows + p.rows_per_block - 1) / p.rows_per_block);
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
  const int smem = s.groups * 2 * a.width * (int)sizeof(float);
  const NormKernel fn = norm_kernel(s, dtype, true);
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  fn<<<p.blocks, s.threads, smem, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((2 * a.width + 31) / 32), a.ty ? 4u : 1u);
  k_layernorm_dw<<<grid, 256, 0, st>>>(a, p.blocks);
  return cudaGetLastError();
}

}  // namespace recattn
