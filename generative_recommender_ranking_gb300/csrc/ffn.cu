// ffn.cu -- host side of the feed-forward entry points: argument checks (before any CUDA call),
// workspaces in stream order from the library's pool, tensor maps and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "dense.cuh"
#include "few.cuh"
#include "launchers.cuh"
#include "rec_attn.h"
#include "scaled.cuh"
#include "workspace.cuh"

#define REC_ATTN_API extern "C" __attribute__((visibility("default")))

using namespace recattn;

namespace {

constexpr long long kMaxRows = (1LL << 31) - 65536;  // tiles past the last row are still 32-bit coordinates
constexpr long long kMaxWidth = 65536;

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool wide_rows(const void* p, long long cols) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0 && cols % 16 == 0; }

struct Range {
  const void* p;
  size_t bytes;
};
// Whether one of the first `outs` ranges overlaps another range (NULL ranges apart).
bool clash(const Range* r, int outs, int n) {
  for (int i = 0; i < outs; ++i)
    for (int j = i + 1; j < n; ++j)
      if (r[i].p && r[j].p && overlaps(r[i].p, r[i].bytes, r[j].p, r[j].bytes)) return true;
  return false;
}

// The checks that both directions share.
rec_attn_status check_ffn(int32_t dtype, int32_t act, int64_t rows, int64_t width, int64_t hidden) {
  if (dtype != REC_ATTN_BF16 && dtype != REC_ATTN_FP32) return REC_ATTN_ERR_INVALID_ARG;
  if (act != REC_ATTN_SILU && act != REC_ATTN_GELU) return REC_ATTN_ERR_INVALID_ARG;
  const int unit = dtype == REC_ATTN_BF16 ? 8 : 4;  // 16 bytes
  if (rows < 0 || width < 1 || hidden < 1 || width % unit || hidden % unit) return REC_ATTN_ERR_INVALID_ARG;
  if (rows > kMaxRows || width > kMaxWidth || hidden > kMaxWidth) return REC_ATTN_ERR_UNSUPPORTED;
  // a launch's tiles are counted in 32 bits
  if (((rows + kTile - 1) / kTile) * ((2 * std::max(hidden, width) + kTile - 1) / kTile) > INT32_MAX / 2)
    return REC_ATTN_ERR_UNSUPPORTED;
  return REC_ATTN_OK;
}

// Columns behind a row of h, and a half of p, in a workspace: rows of whole 32-byte sectors.  (bf16, 5003 rows of 1408
// with hidden 4104, backward 355 -> 320 us, of which 13 by whole sectors in other rows; 40000 of 512 with 1000 328 -> 251.)
long long row_pad(long long hidden) { return (16 - hidden % 16) % 16; }

int blocks64(int64_t n) { return (int)((n + 63) / 64); }
int blocks_of_p(int64_t hidden) { return row_pad(hidden) ? 2 * blocks64(hidden) : blocks64(2 * hidden); }

// A workspace of the library's pool, given back in stream order.
struct Workspace {
  void* p = nullptr;
  cudaStream_t st;
  explicit Workspace(cudaStream_t s) : st(s) {}
  cudaError_t take(int dev, size_t bytes) {
    cudaMemPool_t pool;
    cudaError_t e = pool_for(dev, &pool);
    if (e == cudaSuccess) e = cudaMallocFromPoolAsync(&p, bytes, pool, st);
    return e;
  }
  cudaError_t give_back() { return p ? cudaFreeAsync(p, st) : cudaSuccess; }
};

cudaError_t dense(DenseOp op, const DenseArgs& a, int sms, cudaStream_t st, bool encoded, const CUtensorMap (&m)[4]) {
  return encoded ? launch_dense(op, m, a, sms, st) : cudaErrorInvalidValue;
}

// A product whose summed axis may be in parts.
cudaError_t summed(DenseOp op, const DenseArgs& a, int sms, cudaStream_t st, bool encoded, const CUtensorMap (&m)[4]) {
  const cudaError_t e = dense(op, a, sms, st, encoded, m);
  return e == cudaSuccess && a.splits > 1
             ? launch_dense_sum(a.part, a.out, (long long)a.M * a.N, a.splits, REC_ATTN_BF16, st) : e;
}

// fp32 matrices as bf16 planes, laid out one after the other in a workspace.
struct PlaneLayout {
  size_t bytes = 0;
  Planes add(long long rows, long long cols) {  // p: the offset, until the workspace is there
    Planes a{reinterpret_cast<void*>(bytes), rows, cols, (cols + 15) / 16 * 16};  // rows of whole 32-byte sectors
    bytes += ws_up(3 * a.plane());
    return a;
  }
};
Planes placed(const Planes& a, const Workspace& ws) {
  Planes b = a;
  b.p = static_cast<char*>(ws.p) + reinterpret_cast<size_t>(a.p);
  return b;
}

// out = a b' over `depth`, the sums of parts of it (s > 1) in part.  cut: the columns of a half of a, and rows of
// a half of b, where a's halves do not adjoin.
cudaError_t plain32(DenseOp op, const Planes& a, const Planes& b, long long M, long long N, long long depth, int s,
                    float* part, void* out, int sms, cudaStream_t st, long long cut = 0) {
  CUtensorMap m[4];
  Dense32Args d{};
  d.d.cut = (int)cut;
  d.d.pad = cut ? (int)row_pad(cut) : 0;
  if (op == DenseOp::kDx && d.d.pad) {
    Planes ha = a, hb = b;
    ha.cols = cut;
    bool ok = encode_planes(&m[0], ha, 128) && encode_planes(&m[1], hb, 64, cut);
    ha.p = static_cast<char*>(a.p) + (cut + d.d.pad) * 2;
    hb.p = static_cast<char*>(b.p) + cut * b.ld * 2;
    ok = ok && encode_planes(&m[2], ha, 128) && encode_planes(&m[3], hb, 64, cut);
    if (!ok) return cudaErrorInvalidValue;
  } else if (!encode_planes(&m[0], a, op == DenseOp::kDw ? 64 : 128) || !encode_planes(&m[1], b, 64)) {
    return cudaErrorInvalidValue;
  }
  d.d.M = (int)M;
  d.d.N = (int)N;
  d.d.kblocks = op == DenseOp::kDx ? blocks_of_p(cut) : blocks64(depth);
  d.d.splits = s;
  d.d.part = part;
  d.d.out = out;
  d.d.status = dense_status();
  const cudaError_t e = launch_dense32(op, m, d, sms, st);
  return e == cudaSuccess && s > 1 ? launch_dense_sum(part, out, M * N, s, REC_ATTN_FP32, st) : e;
}

// The forward for few rows: two kernels, h [rows][hidden] between them.
cudaError_t ffn_few(bool bf16, int act, long long R, long long W, long long H, const void* x, const void* w_in,
                    const void* w_out, void* y, int dev, int sms, cudaStream_t st) {
  Workspace ws(st);
  cudaError_t e = ws.take(dev, R * H * (bf16 ? 2 : 4));
  if (e != cudaSuccess) return e;
  FewArgs a{};
  a.rows = (int)R;
  a.N = (int)H;
  a.K = (int)W;
  a.x = x;
  a.w = w_in;
  a.act = act;
  a.out = ws.p;
  a.status = dense_status();
  e = bf16 ? launch_few(false, true, a, sms, st) : launch_few32(true, a, st);
  a.N = (int)W;
  a.K = (int)H;
  a.x = ws.p;
  a.w = w_out;
  a.out = y;
  a.follows = 1;
  if (e == cudaSuccess) e = bf16 ? launch_few(false, false, a, sms, st) : launch_few32(false, a, st);
  const cudaError_t ef = ws.give_back();
  return e != cudaSuccess ? e : ef;
}

cudaError_t ffn32_fwd(int act, long long R, long long W, long long H, const void* x, const void* w_in, const void* w_out,
                      void* y, int dev, int sms, cudaStream_t st) {
  PlaneLayout l;
  Planes px = l.add(R, W), pi = l.add(2 * H, W), po = l.add(W, H), ph = l.add(R, H);
  const int s = dense32_splits((int)R, (int)W, blocks64(H), sms);
  const size_t off_part = l.bytes;
  Workspace ws(st);
  cudaError_t e = ws.take(dev, off_part + (s > 1 ? (size_t)s * R * W * 4 : 0));
  if (e != cudaSuccess) return e;
  px = placed(px, ws), pi = placed(pi, ws), po = placed(po, ws), ph = placed(ph, ws);
  e = launch_split({3, {x, w_in, w_out}, {px, pi, po}}, st);
  CUtensorMap m[4];
  if (e == cudaSuccess && !(encode_planes(&m[0], px, 128) && encode_planes(&m[1], pi, 64))) e = cudaErrorInvalidValue;
  Dense32Args d{};
  d.d.M = (int)R;
  d.d.N = (int)H;
  d.d.kblocks = blocks64(W);
  d.d.splits = 1;
  d.d.act = act;
  d.d.status = dense_status();
  d.h = ph;
  if (e == cudaSuccess) e = launch_dense32(DenseOp::kGlu, m, d, sms, st);
  if (e == cudaSuccess)
    e = plain32(DenseOp::kOut, ph, po, R, W, H, s, reinterpret_cast<float*>(static_cast<char*>(ws.p) + off_part), y, sms, st);
  const cudaError_t ef = ws.give_back();
  return e != cudaSuccess ? e : ef;
}

cudaError_t ffn32_bwd(int act, long long R, long long W, long long H, const void* x, const void* w_in, const void* w_out,
                      const void* dy, void* dx, void* dw_in, void* dw_out, int dev, int sms, cudaStream_t st) {
  PlaneLayout l;
  Planes px = l.add(R, W), pdy = l.add(R, W), pi = l.add(2 * H, W), po = l.add(W, H), ph = l.add(R, H);
  Planes pp = l.add(R, 2 * (H + row_pad(H)));
  const int sx = dense32_splits((int)R, (int)W, blocks_of_p(H), sms);
  const int si = dense32_splits((int)(2 * H), (int)W, blocks64(R), sms), so = dense32_splits((int)W, (int)H, blocks64(R), sms);
  size_t n_part = 0;
  if (dx && sx > 1) n_part = (size_t)sx * R * W;
  if (dw_in && si > 1) n_part = std::max(n_part, (size_t)(si * 2 * H * W));
  if (dw_out && so > 1) n_part = std::max(n_part, (size_t)(so * H * W));
  const size_t off_part = l.bytes;
  Workspace ws(st);
  cudaError_t e = ws.take(dev, off_part + 4 * n_part);
  if (e != cudaSuccess) return e;
  px = placed(px, ws), pdy = placed(pdy, ws), pi = placed(pi, ws), po = placed(po, ws), ph = placed(ph, ws), pp = placed(pp, ws);
  float* const part = reinterpret_cast<float*>(static_cast<char*>(ws.p) + off_part);
  e = launch_split({4, {x, w_in, w_out, dy}, {px, pi, po, pdy}}, st);
  CUtensorMap m[4];
  if (e == cudaSuccess &&
      !(encode_planes(&m[0], px, 128) && encode_planes(&m[1], pi, 64) && encode_planes(&m[2], pdy, 128) &&
        encode_planes(&m[3], po, 64)))
    e = cudaErrorInvalidValue;
  Dense32Args d{};
  d.d.M = (int)R;
  d.d.N = (int)H;
  d.d.kblocks = blocks64(W);
  d.d.splits = 1;
  d.d.act = act;
  d.d.status = dense_status();
  d.d.pad = (int)row_pad(H);
  d.h = ph;
  d.p = pp;
  if (e == cudaSuccess) e = launch_dense32(DenseOp::kDglu, m, d, sms, st);
  if (e == cudaSuccess && dx) e = plain32(DenseOp::kDx, pp, pi, R, W, 2 * H, sx, part, dx, sms, st, H);
  if (e == cudaSuccess && dw_in) e = plain32(DenseOp::kDw, pp, px, 2 * H, W, R, si, part, dw_in, sms, st, H);
  if (e == cudaSuccess && dw_out) e = plain32(DenseOp::kDw, pdy, ph, W, H, R, so, part, dw_out, sms, st);
  const cudaError_t ef = ws.give_back();
  return e != cudaSuccess ? e : ef;
}

}  // namespace

REC_ATTN_API rec_attn_status rec_attn_ffn_fwd(int32_t dtype, int32_t activation, int64_t rows, int64_t width,
                                              int64_t hidden, const void* x, const void* w_in, const void* w_out,
                                              void* y, void* stream) {
  const rec_attn_status s = check_ffn(dtype, activation, rows, width, hidden);
  if (s != REC_ATTN_OK) return s;
  if (rows == 0) return REC_ATTN_OK;
  if (!x || !w_in || !w_out || !y || misaligned(x) || misaligned(w_in) || misaligned(w_out) || misaligned(y))
    return REC_ATTN_ERR_INVALID_ARG;
  const size_t es = dtype == REC_ATTN_BF16 ? 2 : 4;
  const Range all[4] = {{y, rows * width * es}, {x, rows * width * es}, {w_in, 2 * hidden * width * es},
                        {w_out, hidden * width * es}};
  if (clash(all, 1, 4)) return REC_ATTN_ERR_INVALID_ARG;
  int dev = -1, sms = 0;
  cudaError_t e = device_and_sms(&dev, &sms);
  if (e != cudaSuccess) return from_cuda(e);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool bf16 = dtype == REC_ATTN_BF16;
  if (rows <= (bf16 ? kFewRows : kFewRows32))
    return from_cuda(ffn_few(bf16, activation, rows, width, hidden, x, w_in, w_out, y, dev, sms, st));
  if (!bf16) return from_cuda(ffn32_fwd(activation, rows, width, hidden, x, w_in, w_out, y, dev, sms, st));
  const int s_out = dense_splits((int)rows, (int)width, blocks64(hidden), kBlockUs, sms);
  const long long pad = row_pad(hidden), ld = hidden + pad;
  const size_t off_part = ws_up(rows * ld * es);
  Workspace ws(st);
  e = ws.take(dev, off_part + (s_out > 1 ? 4 * (size_t)s_out * rows * width : 0));
  if (e != cudaSuccess) return from_cuda(e);
  CUtensorMap m[4];
  DenseArgs a{};
  a.act = activation;
  a.splits = 1;
  a.status = dense_status();
  a.M = (int)rows;
  a.N = (int)hidden;
  a.kblocks = blocks64(width);
  a.out = ws.p;
  a.pad = (int)pad;
  a.wide = 1;
  e = dense(DenseOp::kGlu, a, sms, st,
            encode_dense(&m[0], x, rows, width, false) && encode_dense(&m[1], w_in, 2 * hidden, width, false), m);
  a.N = (int)width;
  a.kblocks = blocks64(hidden);
  a.splits = s_out;
  a.part = reinterpret_cast<float*>(static_cast<char*>(ws.p) + off_part);
  a.out = y;
  a.wide = wide_rows(y, width);
  a.follows = 1;
  if (e == cudaSuccess)
    e = summed(DenseOp::kOut, a, sms, st,
               encode_dense(&m[0], ws.p, rows, hidden, false, ld) && encode_dense(&m[1], w_out, width, hidden, false), m);
  const cudaError_t ef = ws.give_back();
  return from_cuda(e != cudaSuccess ? e : ef);
}

REC_ATTN_API rec_attn_status rec_attn_ffn_bwd(int32_t dtype, int32_t activation, int64_t rows, int64_t width,
                                              int64_t hidden, const void* x, const void* w_in, const void* w_out,
                                              const void* dy, void* dx, void* dw_in, void* dw_out, void* stream) {
  const rec_attn_status s = check_ffn(dtype, activation, rows, width, hidden);
  if (s != REC_ATTN_OK) return s;
  const size_t es = dtype == REC_ATTN_BF16 ? 2 : 4;
  const size_t nx = rows * width * es, ni = 2 * hidden * width * es, no = hidden * width * es;
  if (misaligned(dw_in) || misaligned(dw_out)) return REC_ATTN_ERR_INVALID_ARG;
  if (rows > 0 && (!x || !w_in || !w_out || !dy || misaligned(x) || misaligned(w_in) || misaligned(w_out) ||
                   misaligned(dy) || misaligned(dx)))
    return REC_ATTN_ERR_INVALID_ARG;
  const Range all[7] = {{rows > 0 ? dx : nullptr, nx}, {dw_in, ni}, {dw_out, no}, {rows > 0 ? x : nullptr, nx},
                        {w_in, ni}, {w_out, no}, {rows > 0 ? dy : nullptr, nx}};
  if (clash(all, 3, 7)) return REC_ATTN_ERR_INVALID_ARG;
  if (!(rows > 0 && dx) && !dw_in && !dw_out) return REC_ATTN_OK;  // nothing wanted
  int dev = -1, sms = 0;
  cudaError_t e = device_and_sms(&dev, &sms);
  if (e != cudaSuccess) return from_cuda(e);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0) {  // no row: the weights' gradients are zero
    if (dw_in) e = cudaMemsetAsync(dw_in, 0, ni, st);
    if (e == cudaSuccess && dw_out) e = cudaMemsetAsync(dw_out, 0, no, st);
    return from_cuda(e);
  }
  if (dtype == REC_ATTN_FP32)
    return from_cuda(ffn32_bwd(activation, rows, width, hidden, x, w_in, w_out, dy, dx, dw_in, dw_out, dev, sms, st));
  const int kr = blocks64(rows), W = (int)width, H = (int)hidden;
  const long long pad = row_pad(hidden), ld = hidden + pad;
  const int kp = blocks_of_p(hidden);
  const int sx = dx ? dense_splits((int)rows, W, kp, kBlockUs, sms) : 1;
  const int si = dw_in ? dense_splits(2 * H, W, kr, kBlockUs, sms) : 1, so = dw_out ? dense_splits(W, H, kr, kBlockUs, sms) : 1;
  const size_t n_part = std::max({sx > 1 ? (size_t)sx * rows * W : 0, si > 1 ? (size_t)si * 2 * H * W : 0,
                                  so > 1 ? (size_t)so * H * W : 0});
  const size_t off_h = ws_up(rows * 2 * ld * es), off_part = off_h + ws_up(rows * ld * es);
  Workspace ws(st);
  e = ws.take(dev, off_part + 4 * n_part);
  if (e != cudaSuccess) return from_cuda(e);
  char* const p = static_cast<char*>(ws.p);
  char* const h = p + off_h;
  CUtensorMap m[4];
  DenseArgs a{};
  a.act = activation;
  a.splits = 1;
  a.status = dense_status();
  a.part = reinterpret_cast<float*>(p + off_part);
  a.M = (int)rows;
  a.N = H;
  a.kblocks = blocks64(width);
  a.out = p;
  a.out2 = h;
  a.pad = (int)pad;
  a.cut = H;
  a.wide = 1;
  e = dense(DenseOp::kDglu, a, sms, st,
            encode_dense(&m[0], x, rows, width, false) && encode_dense(&m[1], w_in, 2 * hidden, width, false) &&
                encode_dense(&m[2], dy, rows, width, false) && encode_dense(&m[3], w_out, width, hidden, true),
            m);
  a.follows = 1;
  if (e == cudaSuccess && dx) {
    a.N = W;
    a.kblocks = kp;
    a.out = dx;
    a.wide = wide_rows(dx, width);
    a.splits = sx;
    e = summed(DenseOp::kDx, a, sms, st,
               pad ? encode_dense(&m[0], p, rows, hidden, false, 2 * ld) && encode_dense(&m[1], w_in, hidden, width, true) &&
                         encode_dense(&m[2], p + ld * es, rows, hidden, false, 2 * ld) &&
                         encode_dense(&m[3], static_cast<const char*>(w_in) + hidden * width * es, hidden, width, true)
                   : encode_dense(&m[0], p, rows, 2 * hidden, false) && encode_dense(&m[1], w_in, 2 * hidden, width, true),
               m);
  }
  a.kblocks = kr;
  for (int i = 0; i < 2; ++i) {
    void* const dw = i ? dw_out : dw_in;
    if (e != cudaSuccess || !dw) continue;
    a.M = i ? W : 2 * H;
    if (i) a.pad = 0;
    a.N = i ? H : W;
    a.splits = i ? so : si;
    a.out = dw;
    a.wide = wide_rows(dw, a.N);
    e = summed(DenseOp::kDw, a, sms, st,
               (i ? encode_dense(&m[0], dy, rows, width, true) && encode_dense(&m[1], h, rows, hidden, true, ld)
                  : encode_dense(&m[0], p, rows, ld + hidden, true, 2 * ld) && encode_dense(&m[1], x, rows, width, true)),
               m);
  }
  const cudaError_t ef = ws.give_back();
  return from_cuda(e != cudaSuccess ? e : ef);
}

namespace {

long long blocks128(long long n) { return (n + kScaleBlock - 1) / kScaleBlock; }

bool scaled_tiles_ok(long long rows, long long cols) {  // a launch's tiles are counted in 32 bits
  return blocks128(rows) * blocks128(cols) <= INT32_MAX / 2;
}

// The product of one scaled layer.
cudaError_t scaled(bool gated, const void* a, const float* a_scale, long long rows, const void* b, const float* b_scale,
                   long long cols, long long depth, int act, void* out, float* out_scale, bool follows, int splits,
                   float* part, int sms, cudaStream_t st) {
  CUtensorMap ma, mb;
  if (!encode_scaled(&ma, a, rows, depth) || !encode_scaled(&mb, b, gated ? 2 * cols : cols, depth))
    return cudaErrorInvalidValue;
  ScaledArgs s{};
  s.M = (int)rows;
  s.N = (int)cols;
  s.kblocks = (int)blocks128(depth);
  s.a_scale = a_scale;
  s.b_scale = b_scale;
  s.act = act;
  s.wide = wide_rows(out, cols);
  s.out = out;
  s.out_scale = out_scale;
  s.follows = follows;
  s.splits = splits;
  s.part = part;
  s.status = dense_status();
  const cudaError_t e = launch_scaled(gated, ma, mb, s, sms, st);
  return e == cudaSuccess && splits > 1 ? launch_dense_sum(part, out, rows * cols, splits, REC_ATTN_BF16, st) : e;
}

}  // namespace

REC_ATTN_API rec_attn_status rec_attn_scaled_quantize(int32_t dtype, int32_t block_rows, int64_t rows, int64_t width,
                                                      const void* x, void* q, float* scale, void* stream) {
  if (dtype != REC_ATTN_BF16 && dtype != REC_ATTN_FP32) return REC_ATTN_ERR_INVALID_ARG;
  if ((block_rows != 1 && block_rows != kScaleBlock) || rows < 0 || width < 1 || width % 16) return REC_ATTN_ERR_INVALID_ARG;
  if (rows > kMaxRows || width > 2 * kMaxWidth || !scaled_tiles_ok(rows, width)) return REC_ATTN_ERR_UNSUPPORTED;
  if (rows == 0) return REC_ATTN_OK;
  if (!x || !q || !scale || misaligned(x) || misaligned(q) || misaligned(scale)) return REC_ATTN_ERR_INVALID_ARG;
  const size_t n_scale = 4 * (size_t)((rows + block_rows - 1) / block_rows * blocks128(width));
  const Range all[3] = {{q, (size_t)(rows * width)}, {scale, n_scale},
                        {x, (size_t)(rows * width) * (dtype == REC_ATTN_BF16 ? 2 : 4)}};
  if (clash(all, 2, 3)) return REC_ATTN_ERR_INVALID_ARG;
  int dev = -1, sms = 0;
  const cudaError_t e = device_and_sms(&dev, &sms);
  if (e != cudaSuccess) return from_cuda(e);
  const QuantArgs a{x, static_cast<uint8_t*>(q), scale, rows, (int)width, (int)blocks128(width)};
  return from_cuda(launch_quantize(a, dtype, block_rows, sms, static_cast<cudaStream_t>(stream)));
}

REC_ATTN_API rec_attn_status rec_attn_scaled_matmul(int64_t rows, int64_t cols, int64_t depth, const void* a,
                                                    const float* a_scale, const void* b, const float* b_scale, void* y,
                                                    void* stream) {
  if (rows < 0 || cols < 1 || depth < 1 || cols % 8 || depth % 16) return REC_ATTN_ERR_INVALID_ARG;
  if (rows > kMaxRows || cols > 2 * kMaxWidth || depth > 2 * kMaxWidth || !scaled_tiles_ok(rows, cols))
    return REC_ATTN_ERR_UNSUPPORTED;
  if (rows == 0) return REC_ATTN_OK;
  if (!a || !a_scale || !b || !b_scale || !y || misaligned(a) || misaligned(a_scale) || misaligned(b) ||
      misaligned(b_scale) || misaligned(y))
    return REC_ATTN_ERR_INVALID_ARG;
  const size_t kb = blocks128(depth);
  const Range all[5] = {{y, (size_t)(2 * rows * cols)}, {a, (size_t)(rows * depth)}, {a_scale, 4 * rows * kb},
                        {b, (size_t)(cols * depth)}, {b_scale, 4 * blocks128(cols) * kb}};
  if (clash(all, 1, 5)) return REC_ATTN_ERR_INVALID_ARG;
  int dev = -1, sms = 0;
  const cudaError_t e = device_and_sms(&dev, &sms);
  if (e != cudaSuccess) return from_cuda(e);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows <= kFewRows)
    return from_cuda(launch_few(true, false, {(int)rows, (int)cols, (int)depth, a, a_scale, b, b_scale, 0, y, nullptr, 0,
                                              dense_status()}, sms, st));
  const int s = dense_splits((int)rows, (int)cols, (int)kb, kScaledBlockUs, sms);
  Workspace ws(st);
  cudaError_t ew = s > 1 ? ws.take(dev, 4 * (size_t)s * rows * cols) : cudaSuccess;
  if (ew == cudaSuccess)
    ew = scaled(false, a, a_scale, rows, b, b_scale, cols, depth, 0, y, nullptr, false, s, static_cast<float*>(ws.p), sms, st);
  const cudaError_t ef = ws.give_back();
  return from_cuda(ew != cudaSuccess ? ew : ef);
}

REC_ATTN_API rec_attn_status rec_attn_ffn_scaled_fwd(int32_t activation, int64_t rows, int64_t width, int64_t hidden,
                                                     const void* x, const void* w_in, const float* w_in_scale,
                                                     const void* w_out, const float* w_out_scale, void* y,
                                                     void* stream) {
  if (activation != REC_ATTN_SILU && activation != REC_ATTN_GELU) return REC_ATTN_ERR_INVALID_ARG;
  if (rows < 0 || width < 1 || hidden < 1 || width % 16 || hidden % kScaleBlock) return REC_ATTN_ERR_INVALID_ARG;
  if (rows > kMaxRows || width > kMaxWidth || hidden > kMaxWidth || !scaled_tiles_ok(rows, std::max(2 * hidden, width)))
    return REC_ATTN_ERR_UNSUPPORTED;
  if (rows == 0) return REC_ATTN_OK;
  if (!x || !w_in || !w_in_scale || !w_out || !w_out_scale || !y || misaligned(x) || misaligned(w_in) ||
      misaligned(w_in_scale) || misaligned(w_out) || misaligned(w_out_scale) || misaligned(y))
    return REC_ATTN_ERR_INVALID_ARG;
  const size_t kw = blocks128(width), kh = blocks128(hidden), n = rows * width;
  const Range all[6] = {{y, 2 * n}, {x, 2 * n}, {w_in, (size_t)(2 * hidden * width)}, {w_in_scale, 8 * kh * kw},
                        {w_out, (size_t)(hidden * width)}, {w_out_scale, 4 * kh * kw}};
  if (clash(all, 1, 6)) return REC_ATTN_ERR_INVALID_ARG;
  int dev = -1, sms = 0;
  cudaError_t e = device_and_sms(&dev, &sms);
  if (e != cudaSuccess) return from_cuda(e);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool few = rows <= kFewRows;
  const size_t off_xs = ws_up(n), off_h = off_xs + ws_up(4 * rows * kw), off_hs = off_h + ws_up(rows * hidden);
  const int s = few ? 1 : dense_splits((int)rows, (int)width, (int)kh, kScaledBlockUs, sms);
  const size_t off_part = off_hs + ws_up(4 * rows * kh);
  Workspace ws(st);
  e = ws.take(dev, off_part + (s > 1 ? 4 * (size_t)s * n : 0));
  if (e != cudaSuccess) return from_cuda(e);
  uint8_t* const xq = static_cast<uint8_t*>(ws.p);
  float* const xs = reinterpret_cast<float*>(xq + off_xs);
  uint8_t* const hq = xq + off_h;
  float* const hs = reinterpret_cast<float*>(xq + off_hs);
  e = launch_quantize({x, xq, xs, rows, (int)width, (int)kw}, REC_ATTN_BF16, 1, sms, st);
  if (few) {
    const int R = (int)rows, W = (int)width, H = (int)hidden;
    int* const word = dense_status();
    if (e == cudaSuccess)
      e = launch_few(true, true, {R, H, W, xq, xs, w_in, w_in_scale, activation, hq, hs, 1, word}, sms, st);
    if (e == cudaSuccess)
      e = launch_few(true, false, {R, W, H, hq, hs, w_out, w_out_scale, 0, y, nullptr, 1, word}, sms, st);
  } else {
    if (e == cudaSuccess)
      e = scaled(true, xq, xs, rows, w_in, w_in_scale, hidden, width, activation, hq, hs, true, 1, nullptr, sms, st);
    if (e == cudaSuccess)
      e = scaled(false, hq, hs, rows, w_out, w_out_scale, width, hidden, 0, y, nullptr, true, s,
                 reinterpret_cast<float*>(xq + off_part), sms, st);
  }
  const cudaError_t ef = ws.give_back();
  return from_cuda(e != cudaSuccess ? e : ef);
}

REC_ATTN_API rec_attn_status rec_attn_dense_device_status(int32_t* status_out, void* stream) {
  if (!status_out) return REC_ATTN_ERR_INVALID_ARG;
  int* const word = dense_status();
  if (!word) return REC_ATTN_ERR_CUDA;
  int s = 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemcpyAsync(&s, word, sizeof s, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && s != REC_ATTN_OK) {  // reported: later calls start anew (while it was set, no other error was kept)
    e = cudaMemsetAsync(word, 0, sizeof s, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  }
  if (e == cudaSuccess) *status_out = s;
  return from_cuda(e);
}

REC_ATTN_API rec_attn_status rec_attn_check_dense_wait_timeout(uint32_t limit_ms, void* stream) {
  if (limit_ms < 1 || limit_ms > 10000) return REC_ATTN_ERR_INVALID_ARG;
  int* const word = dense_status();
  if (!word) return REC_ATTN_ERR_CUDA;
  return from_cuda(launch_wait_timeout(word, limit_ms * 1000000ull, static_cast<cudaStream_t>(stream)));
}
