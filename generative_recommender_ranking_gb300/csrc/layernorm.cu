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
// held in the registers of `tpr` threads, 16 values each (two 16-byte chunks of bf16, four
// of fp32), so the variance is the mean of squared differences from the mean itself and
// the backward recomputes both statistics from the row it reads anyway.  The backward takes
// two reductions a row: {sum x, sum u}, then {sum (x - m)^2, sum u (x - m)}.
// Statistics, sums and gradients of the gains are fp32; outputs are rounded once.
#include <cuda_bf16.h>

#include "launchers.cuh"

namespace recattn {

namespace {

constexpr int kEpt = 16;       // values of a row per thread
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
  // Sums of a and b over the row's threads, to every thread.
  __device__ __forceinline__ float2 sum2(float a, float b) {
    for (int o = min(tpr, 32) >> 1; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (warps == 1) return make_float2(a, b);
    float2* r = red + buf * warps;
    buf ^= 1;  // the next reduction writes the other half: one barrier each suffices
    if ((lane & 31) == 0) r[lane >> 5] = make_float2(a, b);
    asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(tpr) : "memory");
    float2 t = r[0];
    for (int w = 1; w < warps; ++w) {
      t.x += r[w].x;
      t.y += r[w].y;
    }
    return t;
  }
};

__device__ __forceinline__ void load_gain(const float* p, float* x, int n) {
  for (int i = 0; i < n; i += 4) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
    x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
  }
}

// Rows of a block: groups of tpr threads take consecutive rows in turn, so at any time a
// block reads neighbouring rows.  A row whose type is outside 0..3 belongs to no group:
// its output (or gradient) is zero.
template <typename E>
__global__ void __launch_bounds__(1024) k_layernorm_fwd(NormArgs a) {
  constexpr int N = Vec<E>::kN, NV = kEpt / N;
  __shared__ float2 s_red[64];
  RowGroup g;
  g.init(a.tpr, s_red);
  const int groups = blockDim.x / a.tpr, chunks = a.width / N;
  const float inv_w = 1.f / (float)a.width;
  // whole warps run every iteration (rows past the end are loaded as zeros and not stored)
  const long long stride = (long long)gridDim.x * groups;
  for (long long r0 = (long long)blockIdx.x * groups; r0 < a.rows; r0 += stride) {
    const long long row = r0 + g.id;
    const bool in = row < a.rows;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const E*>(a.x) + (in ? row : 0) * a.width);
    float x[kEpt];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * a.tpr + g.lane;
      Vec<E>::unpack(in && c < chunks ? src[c] : make_uint4(0, 0, 0, 0), x + i * N);
    }
    const int ty = in && a.ty ? a.ty[row] : 0;
#pragma unroll
    for (int e = 0; e < kEpt; ++e) s += x[e];
    const float mean = g.sum2(s, 0.f).x * inv_w;
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
    const float rstd = rsqrtf(g.sum2(q, 0.f).x * inv_w + a.eps);
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
      load_gain(w + c * N, wv, N);
      if (b) load_gain(b + c * N, bv, N);
#pragma unroll
      for (int e = 0; e < N; ++e) y[e] = ok ? fmaf(x[i * N + e] * rstd, wv[e], b ? bv[e] : 0.f) : 0.f;
      dst[c] = Vec<E>::pack(y);
    }
  }
}

// Backward.  Block k takes the contiguous rows [k R, (k + 1) R), its groups in turn, and
// keeps the gains' gradients of its columns in registers while the type stays the same (a
// request's types come in a few runs).  When the type changes, a group adds what it holds
// to a slot of its own in a.flush; at the end the block sums its groups, type by type, into
// its row of a.part.  k_layernorm_dw then sums the blocks.  Every sum has a fixed order, so
// the gradients do not change from call to call.
template <typename E>
__global__ void __launch_bounds__(1024) k_layernorm_bwd(NormArgs a) {
  constexpr int N = Vec<E>::kN, NV = kEpt / N;
  __shared__ float2 s_red[64];
  __shared__ int s_open[32];                  // per group: the type it still holds (-1: none)
  __shared__ unsigned s_flushed[32];          // per group: types with sums in its slot
  extern __shared__ float s_sum[];            // [groups][2][width padded to 4]: open sums
  RowGroup g;
  g.init(a.tpr, s_red);
  const int groups = blockDim.x / a.tpr, chunks = a.width / N;
  const float inv_w = 1.f / (float)a.width;
  float dw[kEpt], db[kEpt];
#pragma unroll
  for (int e = 0; e < kEpt; ++e) dw[e] = db[e] = 0.f;
  int cur = -1;
  unsigned flushed = 0;
  float* slots = a.flush ? a.flush + ((long long)blockIdx.x * groups + g.id) * 4 * 2 * a.width : nullptr;
  auto flush = [&]() {
    float* p = slots + (long long)cur * 2 * a.width;
    const bool add = (flushed >> cur) & 1u;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * a.tpr + g.lane;
      if (c >= chunks) continue;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        float* pw = p + c * N + e;
        float* pb = pw + a.width;
        *pw = add ? *pw + dw[i * N + e] : dw[i * N + e];
        *pb = add ? *pb + db[i * N + e] : db[i * N + e];
      }
    }
    flushed |= 1u << cur;
#pragma unroll
    for (int e = 0; e < kEpt; ++e) dw[e] = db[e] = 0.f;
  };
  const long long first = (long long)blockIdx.x * a.rows_per_block;
  const long long last = min(first + a.rows_per_block, a.rows);
  for (long long r0 = first; r0 < last; r0 += groups) {
    const long long row = r0 + g.id;
    const bool in = row < last;
    const uint4* sx = reinterpret_cast<const uint4*>(static_cast<const E*>(a.x) + (in ? row : 0) * a.width);
    const uint4* sy = reinterpret_cast<const uint4*>(static_cast<const E*>(a.dy) + (in ? row : 0) * a.width);
    float x[kEpt], u[kEpt], dy[kEpt];
    const int ty = in ? (a.ty ? a.ty[row] : 0) : -1;
    const bool ok = (unsigned)ty <= 3u;
    const float* w = a.w + (long long)(ok ? ty : 0) * a.width;
    float s = 0.f, su = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * a.tpr + g.lane;
      const bool act = in && c < chunks;
      Vec<E>::unpack(act ? sx[c] : make_uint4(0, 0, 0, 0), x + i * N);
      Vec<E>::unpack(act ? sy[c] : make_uint4(0, 0, 0, 0), dy + i * N);
      float wv[N];
#pragma unroll
      for (int e = 0; e < N; ++e) wv[e] = 0.f;
      if (act) load_gain(w + c * N, wv, N);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        u[i * N + e] = dy[i * N + e] * wv[e];
        s += x[i * N + e];
        su += u[i * N + e];
      }
    }
    const float2 t1 = g.sum2(s, su);
    const float mean = t1.x * inv_w, mu = t1.y * inv_w;
    float q = 0.f, ux = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i * a.tpr + g.lane >= chunks) continue;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        x[i * N + e] -= mean;
        q = fmaf(x[i * N + e], x[i * N + e], q);
        ux = fmaf(u[i * N + e], x[i * N + e], ux);
      }
    }
    const float2 t2 = g.sum2(q, ux);
    const float rstd = rsqrtf(t2.x * inv_w + a.eps);
    const float mun = t2.y * inv_w * rstd;  // mean of u n
    if (!in) continue;
    if (ok && ty != cur) {
      if (cur >= 0) flush();
      cur = ty;
    }
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
        d[e] = ok ? rstd * (u[k] - mu - n * mun) : 0.f;
        if (ok) {
          dw[k] = fmaf(dy[k], n, dw[k]);
          db[k] += dy[k];
        }
      }
      dst[c] = Vec<E>::pack(d);
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

// Threads per row: 16 values each, rounded up to a power of two of at least 8 (within a
// warp; so a block has at most 32 rows at a time) or to whole warps.
int threads_per_row(int width) {
  const int n = (width + kEpt - 1) / kEpt;
  if (n > 32) return (n + 31) / 32 * 32;
  int t = 8;
  while (t < n) t *= 2;
  return t;
}

int block_threads(int tpr) { return tpr <= kNormThreads ? kNormThreads / tpr * tpr : tpr; }

}  // namespace

cudaError_t launch_layernorm_fwd(NormArgs a, int dtype, int num_sms, cudaStream_t st) {
  if (a.rows <= 0) return cudaSuccess;
  a.tpr = threads_per_row(a.width);
  const int threads = block_threads(a.tpr), groups = threads / a.tpr;
  const long long need = (a.rows + groups - 1) / groups, cap = (long long)num_sms * (2048 / threads);
  const unsigned grid = (unsigned)(need < cap ? need : cap);
  if (dtype == REC_ATTN_BF16) k_layernorm_fwd<__nv_bfloat16><<<grid, threads, 0, st>>>(a);
  else k_layernorm_fwd<float><<<grid, threads, 0, st>>>(a);
  return cudaGetLastError();
}

NormBwdPlan layernorm_bwd_plan(long long rows, int width, bool by_type, int num_sms) {
  NormBwdPlan p;
  const int tpr = threads_per_row(width), threads = block_threads(tpr), groups = threads / tpr;
  const long long need = (rows + groups - 1) / groups, cap = 2LL * num_sms;
  p.blocks = (int)(need < cap ? need : cap);
  p.rows_per_block = (rows + p.blocks - 1) / p.blocks;
  p.rows_per_block = (p.rows_per_block + groups - 1) / groups * groups;
  p.blocks = (int)((rows + p.rows_per_block - 1) / p.rows_per_block);
  const int types = by_type ? 4 : 1;
  p.off_part = ((size_t)p.blocks * sizeof(unsigned) + 255) & ~(size_t)255;
  p.off_flush = p.off_part + (size_t)p.blocks * types * 2 * width * sizeof(float);
  p.bytes = p.off_flush + (by_type ? (size_t)p.blocks * groups * 4 * 2 * width * sizeof(float) : 0);
  return p;
}

cudaError_t launch_layernorm_bwd(NormArgs a, const NormBwdPlan& p, void* ws, int dtype, cudaStream_t st) {
  a.tpr = threads_per_row(a.width);
  const int threads = block_threads(a.tpr), groups = threads / a.tpr;
  a.rows_per_block = p.rows_per_block;
  char* w = static_cast<char*>(ws);
  a.seen = reinterpret_cast<unsigned*>(w);
  a.part = reinterpret_cast<float*>(w + p.off_part);
  a.flush = a.ty ? reinterpret_cast<float*>(w + p.off_flush) : nullptr;
  const int smem = groups * 2 * a.width * (int)sizeof(float);
  const void* fn = dtype == REC_ATTN_BF16 ? (const void*)k_layernorm_bwd<__nv_bfloat16> : (const void*)k_layernorm_bwd<float>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  if (dtype == REC_ATTN_BF16) k_layernorm_bwd<__nv_bfloat16><<<p.blocks, threads, smem, st>>>(a);
  else k_layernorm_bwd<float><<<p.blocks, threads, smem, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)((2 * a.width + 31) / 32), a.ty ? 4u : 1u);
  k_layernorm_dw<<<grid, 256, 0, st>>>(a, p.blocks);
  return cudaGetLastError();
}

}  // namespace recattn
