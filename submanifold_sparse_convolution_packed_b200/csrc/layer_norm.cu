// Layer norm over the channels of each row, with an activation behind it, and
// its gradients (the sparse ResBlocks' norm and SiLU before each conv, the
// transformer blocks' norms with and without affine parameters: shared
// sparse-core commit log, "affine asymmetry").
//
//   z = gamma * (x - mean) * rstd + beta,  y = act(z)
//   dz = dy * act'(z),  g = dz * gamma,  xh = (x - mean) * rstd
//   dx = rstd * (g - mean_c(g) - xh * mean_c(g * xh))
//   dgamma = sum_rows dz * xh,  dbeta = sum_rows dz
//
// Both are bound by HBM: each row is read once into registers (two passes over
// the registers for mean and variance, fp32) and written once.  A group of
// TPR lanes holds a row as 16-byte chunks; blocks are persistent, and the forward
// pass fetches the next row before it works on the current one and keeps gamma and
// beta in registers.
// Measured: 1,300,007 x 64 fp16 with SiLU 77 us (4.5 TB/s; HBM at 46% and the
// special-function unit at 41% of their peaks, an exponential and half a reciprocal
// a value: what is left is the latency of a row, its load, two sums over its lanes and
// its exponentials, with one row ahead), 410 x 16 fp32 1.7 us;
// gradients of 133,450 x 128 bf16 with SiLU 33 us (3.1 TB/s: the sums over the rows
// take the registers that more loads in flight would need), of 20,011 x 512 fp32
// 23 us (5.3 TB/s).  The backward pass keeps the channel sums of its rows in
// registers (fp32, at most kSumRows rows each), adds them up per block in a fixed
// order and leaves one partial row per block, which k_ln_fold adds in fp64:
// no atomics, so the same call gives the same bits.
#include <type_traits>

#include "epilogue.cuh"
#include "kernels.h"
#include "tokens.cuh"

namespace smc {

namespace {

constexpr int kThreads = 256;

// 1 / (1 + exp(-z)).  fp32 rows take the accurate exponential and a division;
// the others the fast exponential (an error of a few fp32 ulp, far below the
// rounding of the result).
template <typename T> __device__ __forceinline__ float sigmoid(float z) {
  return std::is_same<T, float>::value ? 1.f / (1.f + expf(-z)) : __fdividef(1.f, 1.f + exp2_fast(z * -kLog2e));
}

// Two of them with one reciprocal: 1/a = b * 1/(ab), three special operations for two
// values instead of four.  The exponent is cut at 62 (z = -43), so that ab stays
// in range, and so is the z that the sigmoid is multiplied by (silu_arg): what is
// behind the cut is below 1e-17 either way.  A NaN leaves its neighbour alone
// and comes back with its own z.
template <typename T> __device__ __forceinline__ void sigmoid2(float z0, float z1, float* s0, float* s1) {
  if (std::is_same<T, float>::value) {
    *s0 = sigmoid<T>(z0);
    *s1 = sigmoid<T>(z1);
    return;
  }
  const float2 t = mul2(make_float2(z0, z1), make_float2(-kLog2e, -kLog2e));
  const float a = 1.f + exp2_fast(fminf(t.x, 62.f)), b = 1.f + exp2_fast(fminf(t.y, 62.f));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a * b));
  *s0 = r * b;
  *s1 = r * a;
}

__device__ __forceinline__ float2 silu_arg(float z0, float z1) {
  return make_float2(z0 < -43.f ? -43.f : z0, z1 < -43.f ? -43.f : z1);
}

template <typename T> __device__ __forceinline__ float act_value(float z, int act) {
  if (act == kActRelu) return z < 0.f ? 0.f : z;  // a NaN stays
  if (act == kActSilu) return z * sigmoid<T>(z);
  return z;
}

template <typename T> __device__ __forceinline__ float act_slope(float z, int act) {
  if (act == kActRelu) return z > 0.f ? 1.f : 0.f;
  if (act == kActSilu) {
    const float s = sigmoid<T>(z);
    return s * (1.f + z * (1.f - s));
  }
  return 1.f;
}

// act over a lane's values, and its slopes there.
template <typename T, int N> __device__ __forceinline__ void act_values(float (&z)[N], int act) {
  if (act == kActNone) return;
  if (act == kActSilu && N % 2 == 0) {
#pragma unroll
    for (int i = 0; i + 1 < N; i += 2) {
      float2 s;
      sigmoid2<T>(z[i], z[i + 1], &s.x, &s.y);
      s = mul2(silu_arg(z[i], z[i + 1]), s);
      z[i] = s.x;
      z[i + 1] = s.y;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) z[i] = act_value<T>(z[i], act);
}

template <typename T, int N> __device__ __forceinline__ void act_slopes(float (&z)[N], int act) {
  if (act == kActSilu && N % 2 == 0) {
#pragma unroll
    for (int i = 0; i + 1 < N; i += 2) {
      float2 s;
      sigmoid2<T>(z[i], z[i + 1], &s.x, &s.y);
      const float2 zz = silu_arg(z[i], z[i + 1]), one = make_float2(1.f, 1.f);
      // s (1 + z (1 - s))
      const float2 t = mul2(s, fma2(zz, add2(one, make_float2(-s.x, -s.y)), one));
      z[i] = t.x;
      z[i + 1] = t.y;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) z[i] = act_slope<T>(z[i], act);
}

// Blocks that an SM should hold, by the elements a lane holds: more rows in
// flight for short rows, registers for long ones.  (Forward, 8 elements: 3, 4,
// 5, 6 blocks took 86, 75, 82, 90 us on 1.3M x 64 fp16; backward: 2, 3, 4 took
// 37, 33, 34 us on 133450 x 128 bf16, where fetching the next row ahead, as the
// forward pass does, cost 3 us in registers.)
constexpr int fwd_blocks(int elems) { return elems <= 8 ? 4 : elems <= 16 ? 2 : 1; }
constexpr int bwd_blocks(int elems) { return elems <= 8 ? 3 : elems <= 16 ? 2 : 1; }

// Rows in one running fp32 sum of the backward pass, at most: its roundings are
// then below 2^-16 of it, whatever the values (4000 and 6250 rows of a constant were
// off by 6e-5 and 8e-5).
constexpr int kSumRows = 512;

template <typename T>
struct NormArgs {
  const T *x, *dy, *gamma, *beta;
  const float* stats_in;
  T *out, *dgamma, *dbeta;
  float *stats, *part;
  int64_t n;
  int c, act;
  float eps;
};

// Elementwise steps over a lane's values, two to an instruction.
template <int N> __device__ __forceinline__ float sum_of(const float (&x)[N]) {
  if constexpr (N % 2 == 0) {
    float2 s = make_float2(x[0], x[1]);
#pragma unroll
    for (int i = 2; i < N; i += 2) s = add2(s, make_float2(x[i], x[i + 1]));
    return s.x + s.y;
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) s += x[i];
  return s;
}

template <int N> __device__ __forceinline__ float dot_of(const float (&x)[N], const float (&y)[N]) {
  if constexpr (N % 2 == 0) {
    float2 s = mul2(make_float2(x[0], x[1]), make_float2(y[0], y[1]));
#pragma unroll
    for (int i = 2; i < N; i += 2) s = fma2(make_float2(x[i], x[i + 1]), make_float2(y[i], y[i + 1]), s);
    return s.x + s.y;
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) s += x[i] * y[i];
  return s;
}

// z = x * y + w, elementwise (z may be any of them).
template <int N>
__device__ __forceinline__ void fma_all(const float (&x)[N], const float (&y)[N], const float (&w)[N], float (&z)[N]) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 t = fma2(make_float2(x[i], x[i + 1]), make_float2(y[i], y[i + 1]), make_float2(w[i], w[i + 1]));
      z[i] = t.x;
      z[i + 1] = t.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = fmaf(x[i], y[i], w[i]);
  }
}

template <int N> __device__ __forceinline__ void mul_all(float (&z)[N], const float (&x)[N]) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 t = mul2(make_float2(z[i], z[i + 1]), make_float2(x[i], x[i + 1]));
      z[i] = t.x;
      z[i + 1] = t.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] *= x[i];
  }
}

// z = (z + a) * m
template <int N> __device__ __forceinline__ void shift_scale(float (&z)[N], float a, float m) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 t = mul2(add2(make_float2(z[i], z[i + 1]), make_float2(a, a)), make_float2(m, m));
      z[i] = t.x;
      z[i + 1] = t.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = (z[i] + a) * m;
  }
}

// A lane's chunks of a row: chunk k * TPR + l of each of its NCH (kWhole: the
// row has all of them).
template <typename T, int EPC, int NCH, int TPR, bool kWhole>
struct Row {
  using C = Chunk<T, EPC>;
  C c[NCH];
  __device__ __forceinline__ void load(const C* p, int l, int chunks, bool there) {
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int j = k * TPR + l;
      if (there && (kWhole || j < chunks)) {
        c[k] = p[j];
      } else {
        float f[EPC];
#pragma unroll
        for (int i = 0; i < EPC; ++i) f[i] = 0.f;
        c[k] = pack<T, EPC>(f);
      }
    }
  }
  __device__ __forceinline__ void values(float (&f)[NCH * EPC]) const {
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      float t[EPC];
      unpack(c[k], t);
#pragma unroll
      for (int i = 0; i < EPC; ++i) f[k * EPC + i] = t[i];
    }
  }
  static __device__ __forceinline__ void store(C* p, const float (&f)[NCH * EPC], int l, int chunks) {
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int j = k * TPR + l;
      float t[EPC];
#pragma unroll
      for (int i = 0; i < EPC; ++i) t[i] = f[k * EPC + i];
      if (kWhole || j < chunks) p[j] = pack<T, EPC>(t);
    }
  }
};

// gamma (or 1) and beta (or 0) of a lane's channels.
template <typename T, int EPC, int NCH, int TPR, bool kWhole>
__device__ __forceinline__ void parameter(const T* p, float otherwise, int l, int chunks, float (&f)[NCH * EPC]) {
  if (p) {
    Row<T, EPC, NCH, TPR, kWhole> r;
    r.load(reinterpret_cast<const Chunk<T, EPC>*>(p), l, chunks, true);
    r.values(f);
  } else {
#pragma unroll
    for (int i = 0; i < NCH * EPC; ++i) f[i] = otherwise;
  }
}

template <typename T, int EPC, int NCH, int TPR, bool kWhole>
__global__ void __launch_bounds__(kThreads, fwd_blocks(EPC* NCH)) k_layer_norm(const NormArgs<T> a) {
  using C = Chunk<T, EPC>;
  constexpr int kRows = kThreads / TPR, N = NCH * EPC;
  const int l = threadIdx.x % TPR, chunks = a.c / EPC;
  const C* x = reinterpret_cast<const C*>(a.x);
  C* y = reinterpret_cast<C*>(a.out);
  float gam[N], bet[N], f[N];
  parameter<T, EPC, NCH, TPR, kWhole>(a.gamma, 1.f, l, chunks, gam);
  parameter<T, EPC, NCH, TPR, kWhole>(a.beta, 0.f, l, chunks, bet);
  const float inv = 1.f / static_cast<float>(a.c);
  // channels a lane holds beyond the row's, as zeros
  bool pad = false;
#pragma unroll
  for (int k = 0; k < NCH; ++k) pad = pad || (!kWhole && k * TPR + l >= chunks);
  Row<T, EPC, NCH, TPR, kWhole> cur;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  int64_t base = static_cast<int64_t>(blockIdx.x) * kRows, row = base + threadIdx.x / TPR;
  const int64_t jump = step * chunks;
  x += row * chunks;
  y += row * chunks;
  cur.load(x, l, chunks, row < a.n);
  for (; base < a.n; base += step, row += step, y += jump) {
    cur.values(f);
    x += jump;
    cur.load(x, l, chunks, row + step < a.n);  // the next row
    const float mean = group_sum<TPR>(sum_of(f)) * inv;
    shift_scale(f, -mean, 1.f);
    float s = dot_of(f, f);
    if (pad) {  // a padded channel's 0 - mean does not count
#pragma unroll
      for (int k = 0; k < NCH; ++k)
        if (k * TPR + l >= chunks) {
#pragma unroll
          for (int i = 0; i < EPC; ++i) f[k * EPC + i] = 0.f;
        }
      s = dot_of(f, f);
    }
    const float rstd = rsqrtf(group_sum<TPR>(s) * inv + a.eps);
    shift_scale(f, 0.f, rstd);
    fma_all(f, gam, bet, f);
    act_values<T, N>(f, a.act);
    if (row < a.n) {
      Row<T, EPC, NCH, TPR, kWhole>::store(y, f, l, chunks);
      if (a.stats && l == 0) reinterpret_cast<float2*>(a.stats)[row] = make_float2(mean, rstd);
    }
  }
}

template <typename T, int EPC, int NCH, int TPR, bool kWhole>
__global__ void __launch_bounds__(kThreads, bwd_blocks(EPC* NCH)) k_layer_norm_bwd(const NormArgs<T> a) {
  using C = Chunk<T, EPC>;
  constexpr int kRows = kThreads / TPR, N = NCH * EPC;
  extern __shared__ float s_sum[];  // [warps, c]
  const int l = threadIdx.x % TPR, chunks = a.c / EPC;
  const C* x = reinterpret_cast<const C*>(a.x);
  const C* dy = reinterpret_cast<const C*>(a.dy);
  C* dx = reinterpret_cast<C*>(a.out);
  const float2* st = reinterpret_cast<const float2*>(a.stats_in);
  float dg[N], db[N], xh[N], g[N];
#pragma unroll
  for (int i = 0; i < N; ++i) dg[i] = db[i] = 0.f;
  const float inv = 1.f / static_cast<float>(a.c);
  Row<T, EPC, NCH, TPR, kWhole> cx, cd;
  float2 cs;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  int64_t base = static_cast<int64_t>(blockIdx.x) * kRows, row = base + threadIdx.x / TPR;
  const int64_t jump = step * chunks;
  int64_t at = row * chunks;  // of the row to fetch
  auto fetch = [&](int64_t r) {
    cx.load(x + at, l, chunks, r < a.n);
    cd.load(dy + at, l, chunks, r < a.n);
    cs = r < a.n ? st[r] : make_float2(0.f, 0.f);
    at += jump;
  };
  dx += row * chunks;
  for (; base < a.n; base += step, row += step, dx += jump) {
    fetch(row);
    cx.values(xh);
    cd.values(g);
    const float mean = cs.x, rstd = cs.y;
    shift_scale(xh, -mean, rstd);
    float gam[N];  // gamma and beta come from the cache each time: registers are scarcer
    parameter<T, EPC, NCH, TPR, kWhole>(a.gamma, 1.f, l, chunks, gam);
    // rows and chunks that are not there have dy = 0, so they add nothing
    if (a.act != kActNone) {
      float z[N];
      parameter<T, EPC, NCH, TPR, kWhole>(a.beta, 0.f, l, chunks, z);
      fma_all(xh, gam, z, z);
      act_slopes<T, N>(z, a.act);
      mul_all(g, z);
    }
    fma_all(g, xh, dg, dg);
#pragma unroll
    for (int i = 0; i < N; i += (N % 2 ? 1 : 2)) {
      if constexpr (N % 2 == 0) {
        const float2 t = add2(make_float2(db[i], db[i + 1]), make_float2(g[i], g[i + 1]));
        db[i] = t.x;
        db[i + 1] = t.y;
      } else {
        db[i] += g[i];
      }
    }
    mul_all(g, gam);
    const float s1 = group_sum<TPR>(sum_of(g)) * inv;
    const float s2 = group_sum<TPR>(dot_of(g, xh)) * -inv;
    if (row < a.n) {
      // (g - s1 - xh * mean(g xh)) * rstd
#pragma unroll
      for (int i = 0; i < N; i += (N % 2 ? 1 : 2)) {
        if constexpr (N % 2 == 0) {
          const float2 t = fma2(make_float2(xh[i], xh[i + 1]), make_float2(s2, s2), make_float2(g[i], g[i + 1]));
          g[i] = t.x;
          g[i + 1] = t.y;
        } else {
          g[i] = fmaf(xh[i], s2, g[i]);
        }
      }
      shift_scale(g, -s1, rstd);
      Row<T, EPC, NCH, TPR, kWhole>::store(dx, g, l, chunks);
    }
  }
  if (!a.part) return;
  // the block's channel sums: across the row groups of each warp, then over the
  // warps in order
#pragma unroll
  for (int e = 0; e < N; ++e) {
#pragma unroll
    for (int o = TPR; o < 32; o <<= 1) {
      dg[e] += __shfl_xor_sync(0xffffffffu, dg[e], o);
      db[e] += __shfl_xor_sync(0xffffffffu, db[e], o);
    }
  }
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.c;
  const int warp = threadIdx.x >> 5;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (which) __syncthreads();
    if ((threadIdx.x & 31) < TPR) {
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        const int j = k * TPR + l;
        if (j >= chunks) continue;
#pragma unroll
        for (int i = 0; i < EPC; ++i) s_sum[warp * a.c + j * EPC + i] = which ? db[k * EPC + i] : dg[k * EPC + i];
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.c; i += kThreads) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) t += s_sum[w * a.c + i];
      part[which * a.c + i] = t;
    }
  }
}

// Rows too long for registers: one block per row, which reads it again for
// each pass (from L2), an element at a time: 20,011 x 1536 bf16 take 84 us forward and
// 236 us backward, x 1024 take 14 us forward (the same buffers each time, in L2).
__device__ __forceinline__ float block_sum(float x) {
  __shared__ float s_w[kThreads / 32];
  x = group_sum<32>(x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_w[threadIdx.x >> 5] = x;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) t += s_w[w];
  return t;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_layer_norm_long(const NormArgs<T> a) {
  const float width = static_cast<float>(a.c);
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    const T* x = a.x + row * a.c;
    T* y = a.out + row * a.c;
    float s = 0.f;
    for (int j = threadIdx.x; j < a.c; j += kThreads) s += to_f(x[j]);
    const float mean = block_sum(s) / width;
    s = 0.f;
    for (int j = threadIdx.x; j < a.c; j += kThreads) s += (to_f(x[j]) - mean) * (to_f(x[j]) - mean);
    const float rstd = 1.f / sqrtf(block_sum(s) / width + a.eps);
    // y may be x: every element is read and written by one thread
    for (int j = threadIdx.x; j < a.c; j += kThreads)
      y[j] = from_f<T>(act_value<T>((to_f(x[j]) - mean) * rstd * (a.gamma ? to_f(a.gamma[j]) : 1.f) +
                                        (a.beta ? to_f(a.beta[j]) : 0.f), a.act));
    if (a.stats && threadIdx.x == 0) {
      a.stats[2 * row] = mean;
      a.stats[2 * row + 1] = rstd;
    }
  }
}

template <typename T>
__device__ __forceinline__ float dz_of(const NormArgs<T>& a, int64_t row, int j, float mean, float rstd, float* xh) {
  *xh = (to_f(a.x[row * a.c + j]) - mean) * rstd;
  const float z = *xh * (a.gamma ? to_f(a.gamma[j]) : 1.f) + (a.beta ? to_f(a.beta[j]) : 0.f);
  return to_f(a.dy[row * a.c + j]) * act_slope<T>(z, a.act);
}

// The channel sums of a slice of rows (blockIdx.y) for 256 channels.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_layer_norm_long_sums(const NormArgs<T> a) {
  const int j = blockIdx.x * kThreads + threadIdx.x;
  if (j >= a.c) return;
  float dg = 0.f, db = 0.f, xh;
  for (int64_t row = blockIdx.y; row < a.n; row += gridDim.y) {
    const float dz = dz_of(a, row, j, a.stats_in[2 * row], a.stats_in[2 * row + 1], &xh);
    dg += dz * xh;
    db += dz;
  }
  float* part = a.part + static_cast<int64_t>(blockIdx.y) * 2 * a.c;
  part[j] = dg;
  part[a.c + j] = db;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_layer_norm_long_bwd(const NormArgs<T> a) {
  const float width = static_cast<float>(a.c);
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    const float mean = a.stats_in[2 * row], rstd = a.stats_in[2 * row + 1];
    float s1 = 0.f, s2 = 0.f, xh;
    for (int j = threadIdx.x; j < a.c; j += kThreads) {
      const float g = dz_of(a, row, j, mean, rstd, &xh) * (a.gamma ? to_f(a.gamma[j]) : 1.f);
      s1 += g;
      s2 += g * xh;
    }
    s1 = block_sum(s1) / width;
    s2 = block_sum(s2) / width;
    // dx may be dy: every element is read and written by one thread
    for (int j = threadIdx.x; j < a.c; j += kThreads) {
      const float g = dz_of(a, row, j, mean, rstd, &xh) * (a.gamma ? to_f(a.gamma[j]) : 1.f);
      a.out[row * a.c + j] = from_f<T>((g - s1 - xh * s2) * rstd);
    }
  }
}

// dgamma[j], dbeta[j] = the partial rows added up in fp64, in a fixed order:
// 32 channels x 32 runs of partials per block, so that the few hundred
// dependent loads of a channel are spread over 32 warps.
template <typename T>
__global__ void __launch_bounds__(1024) k_ln_fold(const float* part, int parts, int c, T* dgamma, T* dbeta) {
  __shared__ double s_run[32][33];
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5, j = blockIdx.x * 32 + lane;
  double s = 0.0;
  grid_wait();
  if (j < 2 * c)
#pragma unroll 8
    for (int p = run; p < parts; p += 32) s += part[static_cast<int64_t>(p) * 2 * c + j];
  s_run[run][lane] = s;
  __syncthreads();
  // warp `run` adds up channel `run` of the 32
  s = s_run[lane][run];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int jj = blockIdx.x * 32 + run;
  if (lane == 0 && jj < 2 * c) {
    T* to = jj < c ? dgamma : dbeta;
    if (to) to[jj < c ? jj : jj - c] = from_f<T>(static_cast<float>(s));
  }
}

constexpr int kMaxElems = 32;  // elements of a row that one lane holds

template <typename T, int EPC, int NCH, int TPR>
void launch_one(const NormArgs<T>& a, bool backward, int blocks, cudaStream_t s) {
  const size_t sums = a.part ? kThreads / 32 * a.c * sizeof(float) : 0;
  // the common widths (every lane's chunks full) without the checks of the others
  if (EPC > 1 && a.c == EPC * NCH * TPR) {
    if (backward) k_layer_norm_bwd<T, EPC, NCH, TPR, (EPC > 1)><<<blocks, kThreads, sums, s>>>(a);
    else k_layer_norm<T, EPC, NCH, TPR, (EPC > 1)><<<blocks, kThreads, 0, s>>>(a);
    return;
  }
  if (backward) k_layer_norm_bwd<T, EPC, NCH, TPR, false><<<blocks, kThreads, sums, s>>>(a);
  else k_layer_norm<T, EPC, NCH, TPR, false><<<blocks, kThreads, 0, s>>>(a);
}

// Lanes per row: as many as it has chunks, up to a warp, then more chunks per
// lane.
template <typename T, int EPC>
void launch_width(const NormArgs<T>& a, bool backward, int blocks, int tpr, cudaStream_t s) {
  const int nch = (a.c / EPC + tpr - 1) / tpr;
  if (tpr == 1) launch_one<T, EPC, 1, 1>(a, backward, blocks, s);
  else if (tpr == 2) launch_one<T, EPC, 1, 2>(a, backward, blocks, s);
  else if (tpr == 4) launch_one<T, EPC, 1, 4>(a, backward, blocks, s);
  else if (tpr == 8) launch_one<T, EPC, 1, 8>(a, backward, blocks, s);
  else if (tpr == 16) launch_one<T, EPC, 1, 16>(a, backward, blocks, s);
  else if (nch == 1) launch_one<T, EPC, 1, 32>(a, backward, blocks, s);
  else if (nch == 2) launch_one<T, EPC, 2, 32>(a, backward, blocks, s);
  else if (nch <= 4) launch_one<T, EPC, 4, 32>(a, backward, blocks, s);
  else if (EPC <= 4 && nch <= 8) launch_one<T, EPC, EPC <= 4 ? 8 : 1, 32>(a, backward, blocks, s);
  else if (EPC == 1 && nch <= 16) launch_one<T, EPC, EPC == 1 ? 16 : 1, 32>(a, backward, blocks, s);
  else if (EPC == 1) launch_one<T, EPC, EPC == 1 ? 32 : 1, 32>(a, backward, blocks, s);
}

struct NormPlan {
  int epc, tpr, blocks;  // epc 0: the long-row kernels
};

// Row slices of the long rows' channel sums.
int64_t long_slices(int64_t n) {
  constexpr int64_t kFew = 64, kMost = 65535;  // to fill the machine; a grid's y (33 million rows)
  const int64_t few = n < kFew ? n : kFew, s = (n + kSumRows - 1) / kSumRows;
  return s < few ? few : (s < kMost ? s : kMost);
}

NormPlan plan(int64_t n, int c, size_t esz, bool aligned, bool backward, int sms) {
  NormPlan p;
  const int wide = static_cast<int>(16 / esz);
  p.epc = aligned && c % wide == 0 ? wide : 1;
  if (c > 32 * kMaxElems) {
    p.epc = 0;
    p.tpr = kThreads;
    p.blocks = static_cast<int>(n < 8ll * sms ? n : 8ll * sms);
    return p;
  }
  p.tpr = 1;
  while (p.tpr < 32 && p.tpr * p.epc < c) p.tpr *= 2;
  const int64_t need = (n + kThreads / p.tpr - 1) / (kThreads / p.tpr);
  const int elems = (c + p.tpr - 1) / p.tpr;
  const int64_t most = static_cast<int64_t>(backward ? bwd_blocks(elems) : fwd_blocks(elems)) * sms;
  p.blocks = static_cast<int>(need < most ? need : most);
  if (backward && need > most * kSumRows) {  // whole waves
    const int64_t sums = most * kSumRows;
    p.blocks = static_cast<int>((need + sums - 1) / sums * most);
  }
  return p;
}

bool aligned_to_chunks(const LayerNormArgs& a) {
  const uintptr_t bits = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.dy) |
                         reinterpret_cast<uintptr_t>(a.gamma) | reinterpret_cast<uintptr_t>(a.beta) |
                         reinterpret_cast<uintptr_t>(a.out);
  return (bits & 15u) == 0;
}

template <typename T>
cudaError_t launch_typed(const LayerNormArgs& b, int sms, cudaStream_t s) {
  NormArgs<T> a;
  a.x = static_cast<const T*>(b.x);
  a.dy = static_cast<const T*>(b.dy);
  a.gamma = static_cast<const T*>(b.gamma);
  a.beta = static_cast<const T*>(b.beta);
  a.stats_in = b.stats;
  a.out = static_cast<T*>(b.out);
  a.dgamma = static_cast<T*>(b.dgamma);
  a.dbeta = static_cast<T*>(b.dbeta);
  a.stats = b.stats;
  a.part = b.part;
  a.n = b.n;
  a.c = b.c;
  a.act = b.act;
  a.eps = b.eps;
  const bool backward = b.dy != nullptr;
  const NormPlan p = plan(b.n, b.c, sizeof(T), aligned_to_chunks(b), backward, sms);
  int parts = p.blocks, launches = 1;
  if (p.epc == 0) {
    if (!backward) {
      k_layer_norm_long<T><<<p.blocks, kThreads, 0, s>>>(a);
    } else {
      if (a.part) {  // before dx, which may overwrite dy
        parts = static_cast<int>(long_slices(b.n));
        k_layer_norm_long_sums<T><<<dim3((b.c + kThreads - 1) / kThreads, parts), kThreads, 0, s>>>(a);
        ++launches;
      }
      k_layer_norm_long_bwd<T><<<p.blocks, kThreads, 0, s>>>(a);
    }
  } else if (p.epc == 1) {
    launch_width<T, 1>(a, backward, p.blocks, p.tpr, s);
  } else {
    launch_width<T, 16 / sizeof(T)>(a, backward, p.blocks, p.tpr, s);
  }
  if (backward && a.part) {
    const cudaError_t e = launch_after(k_ln_fold<T>, dim3((2 * b.c + 31) / 32), 1024, 0, s, a.part, parts, b.c,
                                       a.dgamma, a.dbeta);
    if (e != cudaSuccess) return e;
    ++launches;
  }
  count_launches(launches);
  return cudaGetLastError();
}

}  // namespace

int64_t layer_norm_parts(const LayerNormArgs& a, int sms) {
  const NormPlan p = plan(a.n, a.c, a.dtype == kF32 ? 4 : 2, aligned_to_chunks(a), a.dy != nullptr, sms);
  return p.epc == 0 ? long_slices(a.n) : p.blocks;
}

cudaError_t launch_layer_norm(const LayerNormArgs& a, int sms, cudaStream_t s) {
  if (a.dtype == kF32) return launch_typed<float>(a, sms, s);
  if (a.dtype == kBF16) return launch_typed<__nv_bfloat16>(a, sms, s);
  return launch_typed<__half>(a, sms, s);
}

}  // namespace smc
