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
// TPR lanes holds a row as 16-byte chunks; blocks are persistent and fetch the
// next row before they work on the current one, and gamma and beta stay in
// registers.  The backward pass keeps the channel sums of its rows in
// registers (fp32, a few hundred rows each), adds them up per block in a fixed
// order and leaves one partial row per block, which k_ln_fold adds in fp64:
// no atomics, so the same call gives the same bits.
#include <type_traits>

#include "epilogue.cuh"
#include "kernels.h"
#include "tokens.cuh"

namespace smc {

namespace {

constexpr int kThreads = 256;

// The exponential is the accurate one for fp32 rows and the fast one (an
// error of a few fp32 ulp, far below the rounding of the result) otherwise.
template <typename T> __device__ __forceinline__ float exp_for(float x) {
  return std::is_same<T, float>::value ? expf(x) : __expf(x);
}

template <typename T> __device__ __forceinline__ float act_value(float z, int act) {
  if (act == kActRelu) return z > 0.f ? z : (z != z ? z : 0.f);
  if (act == kActSilu) return z / (1.f + exp_for<T>(-z));
  return z;
}

template <typename T> __device__ __forceinline__ float act_slope(float z, int act) {
  if (act == kActRelu) return z > 0.f ? 1.f : 0.f;
  if (act == kActSilu) {
    const float s = 1.f / (1.f + exp_for<T>(-z));
    return s * (1.f + z * (1.f - s));
  }
  return 1.f;
}

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

template <typename T, int EPC, int NCH, int TPR>
__global__ void __launch_bounds__(kThreads) k_layer_norm(const NormArgs<T> a) {
  using C = Chunk<T, EPC>;
  constexpr int kRows = kThreads / TPR;
  const int l = threadIdx.x % TPR, chunks = a.c / EPC;
  const C* x = reinterpret_cast<const C*>(a.x);
  C* y = reinterpret_cast<C*>(a.out);
  C gam[NCH], bet[NCH], cur[NCH], nxt[NCH];
  float f[EPC];
#pragma unroll
  for (int i = 0; i < EPC; ++i) f[i] = 1.f;
  const C one = pack<T, EPC>(f);
#pragma unroll
  for (int i = 0; i < EPC; ++i) f[i] = 0.f;
  const C zero = pack<T, EPC>(f);
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
    const int j = k * TPR + l;
    gam[k] = a.gamma && j < chunks ? reinterpret_cast<const C*>(a.gamma)[j] : one;
    bet[k] = a.beta && j < chunks ? reinterpret_cast<const C*>(a.beta)[j] : zero;
  }
  const float inv = static_cast<float>(a.c);
  auto fetch = [&](int64_t row, C(&to)[NCH]) {
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int j = k * TPR + l;
      to[k] = row < a.n && j < chunks ? x[row * chunks + j] : zero;
    }
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  int64_t base = static_cast<int64_t>(blockIdx.x) * kRows;
  fetch(base + threadIdx.x / TPR, cur);
  for (; base < a.n; base += step) {
    const int64_t row = base + threadIdx.x / TPR;
    fetch(row + step, nxt);
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      unpack(cur[k], f);
#pragma unroll
      for (int i = 0; i < EPC; ++i) s += f[i];
    }
    const float mean = group_sum<TPR>(s) / inv;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      unpack(cur[k], f);
      const bool there = k * TPR + l < chunks;
#pragma unroll
      for (int i = 0; i < EPC; ++i) s += there ? (f[i] - mean) * (f[i] - mean) : 0.f;
    }
    const float rstd = 1.f / sqrtf(group_sum<TPR>(s) / inv + a.eps);
    if (row < a.n) {
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        const int j = k * TPR + l;
        float g[EPC], b[EPC];
        unpack(cur[k], f);
        unpack(gam[k], g);
        unpack(bet[k], b);
#pragma unroll
        for (int i = 0; i < EPC; ++i) f[i] = act_value<T>((f[i] - mean) * rstd * g[i] + b[i], a.act);
        if (j < chunks) y[row * chunks + j] = pack<T, EPC>(f);
      }
      if (a.stats && l == 0) {
        a.stats[2 * row] = mean;
        a.stats[2 * row + 1] = rstd;
      }
    }
#pragma unroll
    for (int k = 0; k < NCH; ++k) cur[k] = nxt[k];
  }
}

template <typename T, int EPC, int NCH, int TPR>
__global__ void __launch_bounds__(kThreads) k_layer_norm_bwd(const NormArgs<T> a) {
  using C = Chunk<T, EPC>;
  constexpr int kRows = kThreads / TPR;
  extern __shared__ float s_sum[];  // [2, c]
  const int l = threadIdx.x % TPR, chunks = a.c / EPC;
  const C* x = reinterpret_cast<const C*>(a.x);
  const C* dy = reinterpret_cast<const C*>(a.dy);
  C* dx = reinterpret_cast<C*>(a.out);
  const float2* st = reinterpret_cast<const float2*>(a.stats_in);
  C gam[NCH], bet[NCH], cx[NCH], cd[NCH], nx[NCH], nd[NCH];
  float f[EPC];
#pragma unroll
  for (int i = 0; i < EPC; ++i) f[i] = 1.f;
  const C one = pack<T, EPC>(f);
#pragma unroll
  for (int i = 0; i < EPC; ++i) f[i] = 0.f;
  const C zero = pack<T, EPC>(f);
  float dg[NCH * EPC], db[NCH * EPC];
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
    const int j = k * TPR + l;
    gam[k] = a.gamma && j < chunks ? reinterpret_cast<const C*>(a.gamma)[j] : one;
    bet[k] = a.beta && j < chunks ? reinterpret_cast<const C*>(a.beta)[j] : zero;
#pragma unroll
    for (int i = 0; i < EPC; ++i) dg[k * EPC + i] = db[k * EPC + i] = 0.f;
  }
  const float width = static_cast<float>(a.c);
  float2 cs, ns;
  auto fetch = [&](int64_t row, C(&tx)[NCH], C(&td)[NCH], float2& ts) {
    const bool in = row < a.n;
    ts = in ? st[row] : make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int j = k * TPR + l;
      tx[k] = in && j < chunks ? x[row * chunks + j] : zero;
      td[k] = in && j < chunks ? dy[row * chunks + j] : zero;
    }
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  int64_t base = static_cast<int64_t>(blockIdx.x) * kRows;
  fetch(base + threadIdx.x / TPR, cx, cd, cs);
  for (; base < a.n; base += step) {
    const int64_t row = base + threadIdx.x / TPR;
    fetch(row + step, nx, nd, ns);
    // rows and chunks that are not there have dy = 0, so they add nothing
    float s1 = 0.f, s2 = 0.f;
    float g[NCH * EPC], xh[NCH * EPC];
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      float fx[EPC], fd[EPC], fg[EPC], fb[EPC];
      unpack(cx[k], fx);
      unpack(cd[k], fd);
      unpack(gam[k], fg);
      unpack(bet[k], fb);
#pragma unroll
      for (int i = 0; i < EPC; ++i) {
        const int e = k * EPC + i;
        xh[e] = (fx[i] - cs.x) * cs.y;
        const float dz = a.act == kActNone ? fd[i] : fd[i] * act_slope<T>(xh[e] * fg[i] + fb[i], a.act);
        dg[e] += dz * xh[e];
        db[e] += dz;
        g[e] = dz * fg[i];
        s1 += g[e];
        s2 += g[e] * xh[e];
      }
    }
    s1 = group_sum<TPR>(s1) / width;
    s2 = group_sum<TPR>(s2) / width;
    if (row < a.n) {
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        const int j = k * TPR + l;
#pragma unroll
        for (int i = 0; i < EPC; ++i) f[i] = (g[k * EPC + i] - s1 - xh[k * EPC + i] * s2) * cs.y;
        if (j < chunks) dx[row * chunks + j] = pack<T, EPC>(f);
      }
    }
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      cx[k] = nx[k];
      cd[k] = nd[k];
    }
    cs = ns;
  }
  if (!a.part) return;
  // the block's channel sums: across the row groups of each warp, then warp
  // after warp
#pragma unroll
  for (int e = 0; e < NCH * EPC; ++e) {
#pragma unroll
    for (int o = TPR; o < 32; o <<= 1) {
      dg[e] += __shfl_xor_sync(0xffffffffu, dg[e], o);
      db[e] += __shfl_xor_sync(0xffffffffu, db[e], o);
    }
  }
  for (int w = 0; w < kThreads / 32; ++w) {
    if (static_cast<int>(threadIdx.x >> 5) == w && (threadIdx.x & 31) < TPR) {
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        const int j = k * TPR + l;
        if (j >= chunks) continue;
#pragma unroll
        for (int i = 0; i < EPC; ++i) {
          float* at = s_sum + j * EPC + i;
          at[0] = (w ? at[0] : 0.f) + dg[k * EPC + i];
          at[a.c] = (w ? at[a.c] : 0.f) + db[k * EPC + i];
        }
      }
    }
    __syncthreads();
  }
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.c;
  for (int i = threadIdx.x; i < 2 * a.c; i += kThreads) part[i] = s_sum[i];
}

// Rows too long for registers: one block per row, which reads it again for
// each pass (from L2).
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
// 32 channels x 8 runs of partials per block.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_ln_fold(const float* part, int parts, int c, T* dgamma, T* dbeta) {
  __shared__ double s_run[8][33];
  const int j = blockIdx.x * 32 + (threadIdx.x & 31), run = threadIdx.x >> 5;
  double s = 0.0;
  if (j < 2 * c)
#pragma unroll 8
    for (int p = run; p < parts; p += 8) s += part[static_cast<int64_t>(p) * 2 * c + j];
  s_run[run][threadIdx.x & 31] = s;
  __syncthreads();
  if (run == 0 && j < 2 * c) {
#pragma unroll
    for (int r = 1; r < 8; ++r) s += s_run[r][threadIdx.x & 31];
    T* to = j < c ? dgamma : dbeta;
    if (to) to[j < c ? j : j - c] = from_f<T>(static_cast<float>(s));
  }
}

constexpr int kBlocksPerSm = 4;
constexpr int kMaxElems = 32;  // elements of a row that one lane holds

template <typename T, int EPC, int NCH, int TPR>
void launch_one(const NormArgs<T>& a, bool backward, int blocks, cudaStream_t s) {
  if (backward)
    k_layer_norm_bwd<T, EPC, NCH, TPR><<<blocks, kThreads, a.part ? 2 * a.c * sizeof(float) : 0, s>>>(a);
  else
    k_layer_norm<T, EPC, NCH, TPR><<<blocks, kThreads, 0, s>>>(a);
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

NormPlan plan(int64_t n, int c, size_t esz, bool aligned, int sms) {
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
  p.blocks = static_cast<int>(need < static_cast<int64_t>(kBlocksPerSm) * sms ? need : kBlocksPerSm * sms);
  return p;
}

bool aligned_to_chunks(const LayerNormArgs& a) {
  const uintptr_t bits = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.dy) |
                         reinterpret_cast<uintptr_t>(a.gamma) | reinterpret_cast<uintptr_t>(a.beta) |
                         reinterpret_cast<uintptr_t>(a.out);
  return (bits & 15u) == 0;
}

constexpr int kLongSlices = 64;  // row slices of the long rows' channel sums

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
  const NormPlan p = plan(b.n, b.c, sizeof(T), aligned_to_chunks(b), sms);
  int parts = p.blocks, launches = 1;
  if (p.epc == 0) {
    if (!backward) {
      k_layer_norm_long<T><<<p.blocks, kThreads, 0, s>>>(a);
    } else {
      if (a.part) {  // before dx, which may overwrite dy
        parts = static_cast<int>(b.n < kLongSlices ? b.n : kLongSlices);
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
    k_ln_fold<T><<<(2 * b.c + 31) / 32, kThreads, 0, s>>>(a.part, parts, b.c, a.dgamma, a.dbeta);
    ++launches;
  }
  count_launches(launches);
  return cudaGetLastError();
}

}  // namespace

int64_t layer_norm_parts(const LayerNormArgs& a, int sms) {
  const NormPlan p = plan(a.n, a.c, a.dtype == kF32 ? 4 : 2, aligned_to_chunks(a), sms);
  return p.epc == 0 ? (a.n < kLongSlices ? a.n : kLongSlices) : p.blocks;
}

cudaError_t launch_layer_norm(const LayerNormArgs& a, int sms, cudaStream_t s) {
  if (a.dtype == kF32) return launch_typed<float>(a, sms, s);
  if (a.dtype == kBF16) return launch_typed<__nv_bfloat16>(a, sms, s);
  return launch_typed<__half>(a, sms, s);
}

}  // namespace smc
