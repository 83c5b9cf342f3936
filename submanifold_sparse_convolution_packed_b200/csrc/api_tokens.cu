// C ABI of the token-wise layers (include/smc.h): layer norm, rotary
// positions, attention.  Arguments are checked before anything is launched;
// scratch comes from the library's stream-ordered pool, so calls on several
// streams, or captured into several graphs, never share it.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <numeric>

#include "smc.h"
#include "common.cuh"
#include "kernels.h"

namespace {

// First and last byte of [rows, heads, dim] elements at strides (row, head).
struct Bytes {
  uintptr_t lo, hi;
};

Bytes bytes_of(const void* p, int64_t rows, int64_t heads, int64_t dim, const int64_t* stride, size_t esz) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  if (!p || rows < 1 || heads < 1) return {lo, lo};
  return {lo, lo + static_cast<uintptr_t>((rows - 1) * stride[0] + (heads - 1) * stride[1] + dim) * esz};
}

bool overlap(Bytes a, Bytes b) { return a.lo < b.hi && b.lo < a.hi && a.lo < a.hi && b.lo < b.hi; }

// Strides as the kernels take them: those of axes with one entry do not
// matter and become the dense ones.
bool take_stride(const int64_t in[2], int64_t rows, int64_t heads, int64_t dim, int64_t out[2]) {
  out[1] = in && heads > 1 ? in[1] : dim;
  out[0] = in && rows > 1 ? in[0] : heads * dim;
  constexpr int64_t kMost = int64_t{1} << 58;  // no extent overflows
  return out[0] >= 0 && out[1] >= 0 && out[0] <= kMost / (rows > 1 ? rows : 1) && out[1] <= kMost / heads;
}

// Whether no two elements of an output share a place.
bool distinct(const int64_t st[2], int64_t rows, int64_t heads, int64_t dim) {
  return (st[1] >= dim && st[0] >= (heads - 1) * st[1] + dim) ||
         (st[0] >= dim && st[1] >= (rows - 1) * st[0] + dim);
}

// A strided output as its buffer sees it: [rows, heads, dim] at `p`.
struct View {
  const void* p;
  int64_t rows, heads, dim;
  const int64_t* st;
};

// Whether two outputs can be told apart: their bytes as a whole, or their places
// modulo a distance that both repeat at, be it of rows (heads of packed rows), of
// heads (rows of packed heads) or of both (interleaved heads).  Modulo m, each lies
// in one interval that starts at its address; intervals apart on the circle of m
// never meet.  An axis with one entry repeats at any distance.
bool apart(const View& a, const View& b, size_t esz) {
  if (a.rows < 1 || b.rows < 1) return true;
  if (!overlap(bytes_of(a.p, a.rows, a.heads, a.dim, a.st, esz), bytes_of(b.p, b.rows, b.heads, b.dim, b.st, esz)))
    return true;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  const bool b_first = pb < pa;
  const uintptr_t bytes = b_first ? pa - pb : pb - pa;
  if (bytes % esz) return false;
  const View &lo = b_first ? b : a, &hi = b_first ? a : b;
  const int64_t gap = static_cast<int64_t>(bytes / esz);
  auto row = [](const View& v) { return v.rows > 1 ? v.st[0] : 0; };
  auto head = [](const View& v) { return v.heads > 1 ? v.st[1] : 0; };
  auto separate = [&](int64_t m, int64_t lo_size, int64_t hi_size) {
    const int64_t at = m ? gap % m : 0;  // of hi's interval, lo's starts at 0
    return m && at >= lo_size && at + hi_size <= m;
  };
  const int64_t rows = std::gcd(row(lo), row(hi)), heads = std::gcd(head(lo), head(hi));
  return separate(rows, (lo.heads - 1) * head(lo) + lo.dim, (hi.heads - 1) * head(hi) + hi.dim) ||
         separate(heads, (lo.rows - 1) * row(lo) + lo.dim, (hi.rows - 1) * row(hi) + hi.dim) ||
         separate(std::gcd(rows, heads), lo.dim, hi.dim);
}

// Rows, and blocks along a grid's x, with room for the blocks of splits.
constexpr int64_t kRows = (int64_t{1} << 31) - (1 << 20);

bool known_dtype(int32_t d) { return d == SMC_F32 || d == SMC_BF16 || d == SMC_F16; }

size_t size_of(int32_t d) { return d == SMC_F32 ? 4 : 2; }

bool misaligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

int outcome(cudaError_t e) {
  if (e == cudaSuccess) return SMC_OK;
  cudaGetLastError();
  return e == cudaErrorMemoryAllocation ? SMC_E_OOM : SMC_E_CUDA;
}

struct Device {
  int id = 0, sms = 0;
  bool ok() {
    return cudaGetDevice(&id) == cudaSuccess &&
           cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, id) == cudaSuccess;
  }
};

int attention_args(smc::AttnArgs& a, const void* q, const int64_t* qs, const void* k, const int64_t* ks, const void* v,
                   const int64_t* vs, const int32_t* q_off, const int32_t* k_off, int32_t items, int64_t n, int64_t m,
                   int32_t heads, int32_t kv_heads, int32_t dim, float scale, int32_t causal, int32_t dtype) {
  if (items < 0 || n < 0 || m < 0 || heads < 1 || kv_heads < 1 || dim < 1) return SMC_E_ARG;
  if (!(scale > 0.f) || std::isinf(scale) || (causal != 0 && causal != 1)) return SMC_E_ARG;
  if (!known_dtype(dtype)) return SMC_E_DTYPE;
  if (heads % kv_heads != 0 || heads / kv_heads > 64 || dim > 128 || kv_heads > 65535) return SMC_E_SHAPE;
  if (n * (heads / kv_heads) >= kRows || n >= kRows || m >= kRows || n + m + items >= kRows) return SMC_E_SHAPE;
  if (items > 0 && (!q_off || !k_off || (n > 0 && !q) || (m > 0 && (!k || !v)))) return SMC_E_ARG;
  if (misaligned(q_off, 4) || misaligned(k_off, 4)) return SMC_E_ALIGN;
  const size_t esz = size_of(dtype);
  if (misaligned(q, esz) || misaligned(k, esz) || misaligned(v, esz)) return SMC_E_ALIGN;
  if (!take_stride(qs, n, heads, dim, a.q_stride) || !take_stride(ks, m, kv_heads, dim, a.k_stride) ||
      !take_stride(vs, m, kv_heads, dim, a.v_stride))
    return SMC_E_ARG;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_off = q_off;
  a.k_off = k_off;
  a.n = n;
  a.m = m;
  a.items = items;
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.dim = dim;
  a.dtype = dtype;
  a.scale = scale;
  a.causal = causal != 0;
  return SMC_OK;
}

}  // namespace

extern "C" {

int smc_layer_norm(const void* x, int64_t n, int64_t c, const void* gamma, const void* beta, float eps, int32_t act,
                   void* out, float* stats, int32_t dtype, void* stream) {
  if (n < 0 || c < 1 || !(eps >= 0.f) || std::isinf(eps)) return SMC_E_ARG;
  if (act != SMC_ACT_NONE && act != SMC_ACT_RELU && act != SMC_ACT_SILU) return SMC_E_ARG;
  if (!known_dtype(dtype)) return SMC_E_DTYPE;
  if (c > (1 << 24) || n > (int64_t{1} << 56) / c) return SMC_E_SHAPE;
  if (n == 0) return SMC_OK;
  if (!x || !out) return SMC_E_ARG;
  const size_t esz = size_of(dtype);
  if (misaligned(x, esz) || misaligned(out, esz) || misaligned(gamma, esz) || misaligned(beta, esz) ||
      misaligned(stats, 8))
    return SMC_E_ALIGN;
  const int64_t row[2] = {c, c}, one[2] = {2, 2};
  const Bytes bo = bytes_of(out, n, 1, c, row, esz), bs = bytes_of(stats, n, 1, 2, one, 4);
  const Bytes bg = bytes_of(gamma, 1, 1, c, row, esz), bb = bytes_of(beta, 1, 1, c, row, esz);
  const Bytes bx = bytes_of(x, n, 1, c, row, esz);
  if ((out != x && overlap(bo, bx)) || overlap(bo, bg) || overlap(bo, bb) || overlap(bs, bo) || overlap(bs, bx) ||
      overlap(bs, bg) || overlap(bs, bb))
    return SMC_E_ALIAS;
  if (smc::pending_error() != SMC_OK) return SMC_E_CUDA;
  Device dev;
  if (!dev.ok()) return outcome(cudaErrorUnknown);
  smc::LayerNormArgs a = {};
  a.x = x;
  a.gamma = gamma;
  a.beta = beta;
  a.stats = stats;
  a.out = out;
  a.n = n;
  a.c = static_cast<int>(c);
  a.act = act;
  a.dtype = dtype;
  a.eps = eps;
  return outcome(smc::launch_layer_norm(a, dev.sms, static_cast<cudaStream_t>(stream)));
}

int smc_layer_norm_backward(const void* dy, const void* x, int64_t n, int64_t c, const float* stats, const void* gamma,
                            const void* beta, int32_t act, void* dx, void* dgamma, void* dbeta, int32_t dtype,
                            void* stream) {
  if (n < 0 || c < 1) return SMC_E_ARG;
  if (act != SMC_ACT_NONE && act != SMC_ACT_RELU && act != SMC_ACT_SILU) return SMC_E_ARG;
  if (!known_dtype(dtype)) return SMC_E_DTYPE;
  if (c > (1 << 24) || n > (int64_t{1} << 56) / c) return SMC_E_SHAPE;
  if (n == 0 && !dgamma && !dbeta) return SMC_OK;
  if (n > 0 && (!dy || !x || !stats || !dx)) return SMC_E_ARG;
  const size_t esz = size_of(dtype);
  if (misaligned(dy, esz) || misaligned(x, esz) || misaligned(dx, esz) || misaligned(gamma, esz) ||
      misaligned(beta, esz) || misaligned(dgamma, esz) || misaligned(dbeta, esz) || misaligned(stats, 8))
    return SMC_E_ALIGN;
  const int64_t row[2] = {c, c}, one[2] = {2, 2};
  const Bytes outs[3] = {bytes_of(dx, n, 1, c, row, esz), bytes_of(dgamma, 1, 1, c, row, esz),
                         bytes_of(dbeta, 1, 1, c, row, esz)};
  const Bytes ins[5] = {bytes_of(x, n, 1, c, row, esz), bytes_of(dy, n, 1, c, row, esz),
                        bytes_of(gamma, 1, 1, c, row, esz), bytes_of(beta, 1, 1, c, row, esz),
                        bytes_of(stats, n, 1, 2, one, 4)};
  for (int o = 0; o < 3; ++o) {
    for (int i = 0; i < 5; ++i)  // dx may be dy or x itself
      if (overlap(outs[o], ins[i]) && !(o == 0 && ((i == 0 && dx == x) || (i == 1 && dx == dy)))) return SMC_E_ALIAS;
    for (int i = 0; i < o; ++i)
      if (overlap(outs[o], outs[i])) return SMC_E_ALIAS;
  }
  if (smc::pending_error() != SMC_OK) return SMC_E_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (n == 0) {  // sums over no rows
    cudaError_t e = cudaSuccess;
    if (dgamma) e = cudaMemsetAsync(dgamma, 0, static_cast<size_t>(c) * esz, s);
    if (dbeta && e == cudaSuccess) e = cudaMemsetAsync(dbeta, 0, static_cast<size_t>(c) * esz, s);
    return outcome(e);
  }
  Device dev;
  if (!dev.ok()) return outcome(cudaErrorUnknown);
  smc::LayerNormArgs a = {};
  a.x = x;
  a.dy = dy;
  a.gamma = gamma;
  a.beta = beta;
  a.stats = const_cast<float*>(stats);
  a.out = dx;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.n = n;
  a.c = static_cast<int>(c);
  a.act = act;
  a.dtype = dtype;
  void* part = nullptr;
  if (dgamma || dbeta) {
    const size_t bytes = static_cast<size_t>(smc::layer_norm_parts(a, dev.sms)) * 2 * c * sizeof(float);
    if (smc::scratch_alloc(&part, bytes, dev.id, s) != cudaSuccess) {
      cudaGetLastError();
      return SMC_E_OOM;
    }
    a.part = static_cast<float*>(part);
  }
  const cudaError_t e = smc::launch_layer_norm(a, dev.sms, s);
  if (part) cudaFreeAsync(part, s);
  return outcome(e);
}

int smc_rotary(const void* x, const int64_t x_stride[2], int64_t n, int32_t heads, int32_t dim,
               const int32_t* positions, const int64_t pos_stride[2], const double* freqs, int32_t axes,
               int32_t nfreq, int32_t layout, float scale, int32_t inverse, void* out, const int64_t out_stride[2],
               int32_t dtype, void* stream) {
  if (n < 0 || heads < 1 || dim < 1 || axes < 1 || nfreq < 1 || std::isnan(scale) || std::isinf(scale))
    return SMC_E_ARG;
  if ((layout != SMC_ROTARY_INTERLEAVED && layout != SMC_ROTARY_HALF) || (inverse != 0 && inverse != 1))
    return SMC_E_ARG;
  if (!known_dtype(dtype)) return SMC_E_DTYPE;
  if (2ll * axes * nfreq > dim || dim > (1 << 20) || n >= (int64_t{1} << 40) / dim / heads) return SMC_E_SHAPE;
  if (n == 0) return SMC_OK;
  if (!x || !out || !positions || !freqs) return SMC_E_ARG;
  const size_t esz = size_of(dtype);
  if (misaligned(x, esz) || misaligned(out, esz) || misaligned(positions, 4) || misaligned(freqs, 8))
    return SMC_E_ALIGN;
  smc::RotaryArgs a = {};
  if (!take_stride(x_stride, n, heads, dim, a.x_stride) || !take_stride(out_stride, n, heads, dim, a.out_stride) ||
      !take_stride(pos_stride, n, axes, 1, a.pos_stride) || !distinct(a.out_stride, n, heads, dim))
    return SMC_E_ARG;
  const bool same = x == out && a.x_stride[0] == a.out_stride[0] && a.x_stride[1] == a.out_stride[1];
  const Bytes bo = bytes_of(out, n, heads, dim, a.out_stride, esz);
  const int64_t fs[2] = {nfreq, nfreq};
  if ((!same && overlap(bo, bytes_of(x, n, heads, dim, a.x_stride, esz))) ||
      overlap(bo, bytes_of(positions, n, axes, 1, a.pos_stride, 4)) ||
      overlap(bo, bytes_of(freqs, axes, 1, nfreq, fs, 8)))
    return SMC_E_ALIAS;
  if (smc::pending_error() != SMC_OK) return SMC_E_CUDA;
  Device dev;
  if (!dev.ok()) return outcome(cudaErrorUnknown);
  a.x = x;
  a.out = out;
  a.positions = positions;
  a.freqs = freqs;
  a.n = n;
  a.heads = heads;
  a.dim = dim;
  a.axes = axes;
  a.nfreq = nfreq;
  a.dtype = dtype;
  a.scale = scale;
  a.half = layout == SMC_ROTARY_HALF;
  a.inverse = inverse != 0;
  return outcome(smc::launch_rotary(a, dev.sms, static_cast<cudaStream_t>(stream)));
}

int smc_attention(const void* q, const int64_t q_stride[2], const void* k, const int64_t k_stride[2], const void* v,
                  const int64_t v_stride[2], const int32_t* q_offsets, const int32_t* k_offsets, int32_t items,
                  int64_t n, int64_t m, int32_t heads, int32_t kv_heads, int32_t dim, float scale, int32_t causal,
                  void* out, float* lse, int32_t dtype, void* stream) {
  smc::AttnArgs a = {};
  const int rc = attention_args(a, q, q_stride, k, k_stride, v, v_stride, q_offsets, k_offsets, items, n, m, heads,
                                kv_heads, dim, scale, causal, dtype);
  if (rc != SMC_OK) return rc;
  if (items == 0 || n == 0) return SMC_OK;
  if (!out) return SMC_E_ARG;
  const size_t esz = size_of(dtype);
  if (misaligned(out, esz) || misaligned(lse, 4)) return SMC_E_ALIGN;
  const int64_t dense[2] = {static_cast<int64_t>(heads) * dim, dim}, one[2] = {heads, 1}, off[2] = {1, 1};
  const Bytes outs[2] = {bytes_of(out, n, heads, dim, dense, esz), bytes_of(lse, n, heads, 1, one, 4)};
  const Bytes ins[5] = {bytes_of(q, n, heads, dim, a.q_stride, esz), bytes_of(k, m, kv_heads, dim, a.k_stride, esz),
                        bytes_of(v, m, kv_heads, dim, a.v_stride, esz), bytes_of(q_offsets, items + 1ll, 1, 1, off, 4),
                        bytes_of(k_offsets, items + 1ll, 1, 1, off, 4)};
  for (const Bytes& o : outs)
    for (const Bytes& i : ins)
      if (overlap(o, i)) return SMC_E_ALIAS;
  if (overlap(outs[0], outs[1])) return SMC_E_ALIAS;
  if (smc::pending_error() != SMC_OK) return SMC_E_CUDA;
  Device dev;
  if (!dev.ok()) return outcome(cudaErrorUnknown);
  a.err = smc::status_word(dev.id);
  if (!a.err) return SMC_E_OOM;
  a.out_w = out;
  a.lse_w = lse;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool tc = smc::attn_tc_supported(a);
  void* scratch = nullptr;
  const int64_t bytes = tc ? smc::attn_tc_scratch(a, dev.sms) : smc::attn_simt_scratch(a, dev.sms);
  if (bytes > 0 && smc::scratch_alloc(&scratch, static_cast<size_t>(bytes), dev.id, s) != cudaSuccess) {
    cudaGetLastError();
    return SMC_E_OOM;
  }
  const cudaError_t e =
      tc ? smc::launch_attn_tc(a, scratch, dev.sms, s) : smc::launch_attn_simt(a, false, scratch, dev.sms, s);
  if (scratch) cudaFreeAsync(scratch, s);
  return outcome(e);
}

int smc_attention_backward(const void* dout, const int64_t dout_stride[2], const void* q, const int64_t q_stride[2],
                           const void* k, const int64_t k_stride[2], const void* v, const int64_t v_stride[2],
                           const void* out, const float* lse, const int32_t* q_offsets, const int32_t* k_offsets,
                           int32_t items, int64_t n, int64_t m, int32_t heads, int32_t kv_heads, int32_t dim,
                           float scale, int32_t causal, void* dq, const int64_t dq_stride[2], void* dk,
                           const int64_t dk_stride[2], void* dv, const int64_t dv_stride[2], int32_t dtype,
                           void* stream) {
  smc::AttnArgs a = {};
  const int rc = attention_args(a, q, q_stride, k, k_stride, v, v_stride, q_offsets, k_offsets, items, n, m, heads,
                                kv_heads, dim, scale, causal, dtype);
  if (rc != SMC_OK) return rc;
  if (n + m + 2ll * items >= kRows) return SMC_E_SHAPE;  // both sides' blocks are one grid
  if (items == 0 || (n == 0 && m == 0)) return SMC_OK;
  if (n > 0 && (!dout || !out || !lse || !dq)) return SMC_E_ARG;
  if (m > 0 && (!dk || !dv)) return SMC_E_ARG;
  const size_t esz = size_of(dtype);
  if (misaligned(dout, esz) || misaligned(out, esz) || misaligned(lse, 4) || misaligned(dq, esz) ||
      misaligned(dk, esz) || misaligned(dv, esz))
    return SMC_E_ALIGN;
  if (!take_stride(dout_stride, n, heads, dim, a.dout_stride) || !take_stride(dq_stride, n, heads, dim, a.dq_stride) ||
      !take_stride(dk_stride, m, kv_heads, dim, a.dk_stride) || !take_stride(dv_stride, m, kv_heads, dim, a.dv_stride))
    return SMC_E_ARG;
  if (!distinct(a.dq_stride, n, heads, dim) || !distinct(a.dk_stride, m, kv_heads, dim) ||
      !distinct(a.dv_stride, m, kv_heads, dim))
    return SMC_E_ARG;
  const int64_t dense[2] = {static_cast<int64_t>(heads) * dim, dim}, one[2] = {heads, 1}, off[2] = {1, 1};
  const Bytes outs[3] = {bytes_of(dq, n, heads, dim, a.dq_stride, esz), bytes_of(dk, m, kv_heads, dim, a.dk_stride, esz),
                         bytes_of(dv, m, kv_heads, dim, a.dv_stride, esz)};
  const Bytes ins[8] = {bytes_of(q, n, heads, dim, a.q_stride, esz), bytes_of(k, m, kv_heads, dim, a.k_stride, esz),
                        bytes_of(v, m, kv_heads, dim, a.v_stride, esz), bytes_of(out, n, heads, dim, dense, esz),
                        bytes_of(dout, n, heads, dim, a.dout_stride, esz), bytes_of(lse, n, heads, 1, one, 4),
                        bytes_of(q_offsets, items + 1ll, 1, 1, off, 4), bytes_of(k_offsets, items + 1ll, 1, 1, off, 4)};
  for (const Bytes& o : outs)
    for (const Bytes& i : ins)
      if (overlap(o, i)) return SMC_E_ALIAS;
  // the three gradients may interleave (views of one packed buffer), but share no place
  const View grads[3] = {{dq, n, heads, dim, a.dq_stride}, {dk, m, kv_heads, dim, a.dk_stride},
                         {dv, m, kv_heads, dim, a.dv_stride}};
  for (int i = 0; i < 3; ++i)
    for (int j = 0; j < i; ++j)
      if (!apart(grads[i], grads[j], esz)) return SMC_E_ALIAS;
  if (smc::pending_error() != SMC_OK) return SMC_E_CUDA;
  Device dev;
  if (!dev.ok()) return outcome(cudaErrorUnknown);
  a.err = smc::status_word(dev.id);
  if (!a.err) return SMC_E_OOM;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  a.out = out;
  a.dout = dout;
  a.lse = lse;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  // scratch: delta and the scaled lse, [n, heads] each, the bounds of fp16, partial sums
  const bool tc = smc::attn_bwd_tc_supported(a), bounds = tc && dtype == SMC_F16;
  const int64_t count = n * heads, part = (2 * count + (bounds ? 2 * count + m * kv_heads : 0) + 63) / 64 * 64;
  const int64_t floats = part + (tc ? smc::attn_bwd_tc_scratch(a, dev.sms) : smc::attn_simt_bwd_scratch(a, dev.sms));
  void* scratch = nullptr;
  if (n > 0 && smc::scratch_alloc(&scratch, static_cast<size_t>(floats) * sizeof(float), dev.id, s) != cudaSuccess) {
    cudaGetLastError();
    return SMC_E_OOM;
  }
  a.delta = static_cast<float*>(scratch);
  const smc::BwdScratch x = {a.delta + count, bounds ? reinterpret_cast<float2*>(a.delta + 2 * count) : nullptr,
                             bounds ? a.delta + 4 * count : nullptr, a.delta + part};
  const cudaError_t e = tc ? smc::launch_attn_bwd_tc(a, x, dev.sms, s) : smc::launch_attn_simt(a, true, x.part, dev.sms, s);
  if (scratch) cudaFreeAsync(scratch, s);
  return outcome(e);
}

}  // extern "C"
