// Attention within each item and its gradients, in fp32 FMA: every type, every
// head width up to 128, every stride (the transformer blocks' attention of the
// pages, Pixal3D MLX README "Status" and working notes, over the voxels of one
// item).  The tensor-core kernels take the bf16 / fp16 shapes they can.
//
//   S = scale Q K^T,  P = softmax(S),  O = P V,  lse = log sum exp S
//   dP = dO V^T,  delta = rowsum(dO * O),  dS = P * (dP - delta)
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO,  P = exp(S - lse)
//
// The heads that share a key/value head are packed into the rows of one tile
// (row = query * G + head of the group), so a tile's keys and values are
// loaded once for all of them, and the gradients of shared heads add up in one
// accumulator.  One pass over the keys with a running maximum and sum; the
// backward pass recomputes P from the saved lse twice, one tile of queries
// (dQ) or of keys (dK, dV) per block, so nothing is added with atomics
// and a call gives the same bits every time.
//
// 64 x 64 tiles, 256 threads, each with 4 x 4 scores and 4 rows of the
// accumulator; operands are fp32 in shared memory, rows padded by 16 bytes so
// that the float4 reads along a row meet no bank twice.  Bound by the FMA pipe in
// principle (75 TFLOP/s), in fact by what stands between the products: the
// exponentials, the passes of P through shared memory, and its reads (12
// clocks of a warp's 64 in a product, four warps at once).  Where tiles leave the
// machine idle, what passes is split between blocks.  A warp whose rows are not there
// only loads: one query over 300 keys takes 25 us, 33 us with all warps at work.
// fp32, items of 3000 and 1200 rows, 8 heads over 4, 32 / 64 / 128 channels:
// forward 23 / 30 / 31 TFLOP/s, backward 21 / 25 / 25.  The backward kernel's two blocks
// to an SM leave 128 registers to a thread, which spills there at up to 64 channels
// (at 64: fp32 140 bytes, 16-bit types 180).
#include "attn_join.cuh"
#include "kernels.h"
#include "tokens.cuh"

namespace smc {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;

__device__ __forceinline__ void cp_async16(float* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// kTile rows of one operand into shared memory as fp32, zero behind `rows` and
// behind `dim`.  Row r is packed row first + r: source row (first + r) / group
// of the item, head `head` + (first + r) % group.  fp32 rows of whole 16-byte
// pieces (vec) arrive asynchronously, in the caller's group.
template <typename T, int DP>
__device__ __forceinline__ void load_tile(float* dst, const T* src, int64_t row_stride, int64_t head_stride, int head,
                                          int group, int32_t first, int rows, int dim, bool vec) {
  if (sizeof(T) == 4 && vec) {
    for (int i = threadIdx.x; i < kTile * (DP / 4); i += kThreads) {
      const int r = i / (DP / 4), c = i % (DP / 4) * 4;
      const bool there = r < rows && c < dim;
      const int pr = first + r, row = group == 1 ? pr : pr / group;
      const T* at = there ? src + static_cast<int64_t>(row) * row_stride + (head + pr - row * group) * head_stride + c : src;
      cp_async16(dst + r * (DP + 4) + c, at, there);
    }
    return;
  }
  for (int i = threadIdx.x; i < kTile * DP; i += kThreads) {
    const int r = i / DP, c = i % DP;
    float v = 0.f;
    if (r < rows && c < dim) {
      const int pr = first + r, row = group == 1 ? pr : pr / group;
      v = to_f(src[static_cast<int64_t>(row) * row_stride + (head + pr - row * group) * head_stride + c]);
    }
    dst[r * (DP + 4) + c] = v;
  }
}

// acc[i][j] = A[4 ty + i] . B[tx + 16 j], as pairs of channels (fma2: half of the
// instructions for the same rate of the FMA pipe, which leaves room for the loads).
template <int DP>
__device__ __forceinline__ void mm_nt(const float* A, const float* B, int ty, int tx, float (&acc)[4][4]) {
  float2 t[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) t[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
  for (int d = 0; d < DP; d += 4) {
    float4 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(A + (4 * ty + i) * (DP + 4) + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * (DP + 4) + d);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) t[i][j] = fma2(make_float2(a[i].x, a[i].y), make_float2(b[j].x, b[j].y), t[i][j]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) t[i][j] = fma2(make_float2(a[i].z, a[i].w), make_float2(b[j].z, b[j].w), t[i][j]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = t[i][j].x + t[i][j].y;
}

// Column of the accumulator's element j of thread tx: runs of 2 or 4.
constexpr int run_of(int dp) { return dp / 16 % 4 == 0 ? 4 : 2; }

template <int DP>
__device__ __forceinline__ int col_of(int tx, int j) {
  constexpr int kRun = run_of(DP);
  return j / kRun * 16 * kRun + tx * kRun + j % kRun;
}

// acc[i][j] += sum_k P[4 ty + i][k] * B[k][col_of(tx, j)].  The tile's sum is formed
// by itself: a long item's sum is then two sums of about its root, where one
// running sum was off by twice the plain products' error at 10,000 rows.
template <int DP>
__device__ __forceinline__ void mm_nn(const float* P, const float* B, int ty, int tx, float (&acc)[4][DP / 16]) {
  constexpr int W = DP / 16, kRun = run_of(DP);
  float2 t[4][W / 2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < W / 2; ++j) t[i][j] = make_float2(0.f, 0.f);
#pragma unroll 2
  for (int k = 0; k < kTile; k += 4) {
    float4 p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(P + (4 * ty + i) * (kTile + 4) + k);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      float b[W];
#pragma unroll
      for (int j = 0; j < W; j += kRun) {
        const float* at = B + (k + kk) * (DP + 4) + col_of<DP>(tx, j);
        if constexpr (kRun == 4) {
          const float4 x = *reinterpret_cast<const float4*>(at);
          b[j] = x.x, b[j + 1] = x.y, b[j + 2] = x.z, b[j + 3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(at);
          b[j] = x.x, b[j + 1] = x.y;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float s = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
#pragma unroll
        for (int j = 0; j < W; j += 2) t[i][j / 2] = fma2(make_float2(s, s), make_float2(b[j], b[j + 1]), t[i][j / 2]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < W; j += 2) {
      acc[i][j] += t[i][j / 2].x;
      acc[i][j + 1] += t[i][j / 2].y;
    }
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) k_attn(const AttnArgs a, const Cut cut, bool vec, float* part_o,
                                                   float* part_ml) {
  extern __shared__ float sm[];
  __shared__ Unit unit;
  constexpr int LD = DP + 4, W = DP / 16;
  float *sq = sm, *sk = sq + kTile * LD, *sv = sk + kTile * LD, *sp = sv + kTile * LD;
  const int group = a.heads / a.kv_heads, per_tile = kTile / group;
  find_unit<kThreads>(cut, blockIdx.x, &unit, a.err);
  if (unit.item < 0) return;
  const Unit u = unit;
  const int hk = blockIdx.y, ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int32_t q0 = u.tile * per_tile, queries = u.q.count - q0 < per_tile ? u.q.count - q0 : per_tile;
  const int rows = queries * group;
  const T* q = static_cast<const T*>(a.q) + u.q.begin * a.q_stride[0];
  const T* k = static_cast<const T*>(a.k) + u.k.begin * a.k_stride[0] + hk * a.k_stride[1];
  const T* v = static_cast<const T*>(a.v) + u.k.begin * a.v_stride[0] + hk * a.v_stride[1];
  load_tile<T, DP>(sq, q, a.q_stride[0], a.q_stride[1], hk * group, group, q0 * group, rows, a.dim, vec);
  const float c = a.scale * kLog2e;
  const bool live = (ty & ~1) * 4 < rows;  // a warp without rows only loads (single tokens)
  int32_t seen[4];
  float top[4], sum[4], o[4][W];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ty + i;
    seen[i] = r < rows ? keys_seen(u, q0 + r / group, a.causal) : 0;
    top[i] = -INFINITY;
    sum[i] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) o[i][j] = 0.f;
  }
  // the keys of this block: of its split, up to the last that a query sees
  const int32_t k_lo = u.split * cut.chunk;
  int32_t last = keys_seen(u, q0 + queries - 1, a.causal);
  if (u.splits > 1 && last - k_lo > cut.chunk) last = k_lo + cut.chunk;
  auto load_k = [&](int32_t k0) {
    if (k0 < last)
      load_tile<T, DP>(sk, k, a.k_stride[0], 0, 0, 1, k0, u.k.count - k0 < kTile ? u.k.count - k0 : kTile, a.dim, vec);
    cp_commit();
  };
  auto load_v = [&](int32_t k0) {
    if (k0 < last)
      load_tile<T, DP>(sv, v, a.v_stride[0], 0, 0, 1, k0, u.k.count - k0 < kTile ? u.k.count - k0 : kTile, a.dim, vec);
    cp_commit();
  };
  // V of a step arrives during its scores, K of the next during its product.
  load_k(k_lo);
  load_v(k_lo);
#pragma unroll
  for (int i = 0; i < 4; ++i) seen[i] = seen[i] < last ? seen[i] : last;
  for (int32_t k0 = k_lo; k0 < last; k0 += kTile) {
    cp_wait<1>();
    __syncthreads();
    float s[4][4];
    if (live) mm_nt<DP>(sq, sk, ty, tx, s);
    __syncthreads();
    load_k(k0 + kTile);
    if (live) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (k0 + tx + 16 * j >= seen[i]) s[i][j] = -INFINITY;
          m = fmaxf(m, s[i][j]);
        }
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        // top is the rounded product with c, so that an unchanged maximum keeps
        // the sums by exactly 1 (a fused difference would be off by an ulp of
        // the product, tile after tile)
        m = fmaxf(__fmul_rn(m, c), top[i]);
        const float base = m == -INFINITY ? 0.f : m;  // nothing seen yet: every term is exp2(-inf) = 0
        const float keep = exp2f(top[i] - base);
        float t = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = exp2f(fmaf(s[i][j], c, -base));
          t += s[i][j];
        }
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) t += __shfl_xor_sync(0xffffffffu, t, x);
        sum[i] = sum[i] * keep + t;
        top[i] = m;
#pragma unroll
        for (int j = 0; j < W; ++j) o[i][j] *= keep;
#pragma unroll
        for (int j = 0; j < 4; ++j) sp[(4 * ty + i) * (kTile + 4) + tx + 16 * j] = s[i][j];
      }
    }
    cp_wait<1>();
    __syncthreads();
    if (live) mm_nn<DP>(sp, sv, ty, tx, o);
    __syncthreads();
    load_v(k0 + kTile);
  }
  T* out = static_cast<T*>(a.out_w);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ty + i;
    if (r >= rows) continue;
    const int64_t at = static_cast<int64_t>(u.q.begin + q0 + r / group) * a.heads + hk * group + r % group;
    const float inv = sum[i] == 0.f ? 0.f : 1.f / sum[i];
    if (u.splits > 1) {  // a split: unnormalised
      const int64_t slot = static_cast<int64_t>(u.split) * a.n * a.heads + at;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        const int cc = col_of<DP>(tx, j);
        if (cc < a.dim) part_o[slot * a.dim + cc] = o[i][j];
      }
      if (tx == 0) *reinterpret_cast<float2*>(part_ml + 2 * slot) = make_float2(top[i], sum[i]);
      continue;
    }
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const int cc = col_of<DP>(tx, j);
      if (cc < a.dim) out[at * a.dim + cc] = from_f<T>(o[i][j] * inv);
    }
    if (a.lse_w && tx == 0) a.lse_w[at] = sum[i] == 0.f ? -INFINITY : (top[i] + log2f(sum[i])) * kLn2;
  }
}

// kDQ: a tile of packed queries against all its keys -> dQ.  Otherwise a tile
// of keys against all its packed queries -> dK, dV.  A1, A2 stay; B1, B2 pass.
template <typename T, int DP, bool kDQ>
__device__ __forceinline__ void gradients(const AttnArgs& a, const Cut& cut, bool vec, float* part, int64_t ux) {
  extern __shared__ float sm[];
  __shared__ Unit unit;
  __shared__ float s_lse[kTile], s_delta[kTile];
  constexpr int LD = DP + 4, W = DP / 16;
  float *a1 = sm, *a2 = a1 + kTile * LD, *b1 = a2 + kTile * LD, *b2 = b1 + kTile * LD, *sp = b2 + kTile * LD;
  const int group = a.heads / a.kv_heads, per_tile = kTile / group;
  find_unit<kThreads>(cut, ux, &unit, a.err);
  grid_wait();  // for delta
  if (unit.item < 0) return;
  const Unit u = unit;
  const int hk = blockIdx.y, ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const T* q = static_cast<const T*>(a.q) + u.q.begin * a.q_stride[0];
  const T* dout = static_cast<const T*>(a.dout) + u.q.begin * a.dout_stride[0];
  const T* k = static_cast<const T*>(a.k) + u.k.begin * a.k_stride[0] + hk * a.k_stride[1];
  const T* v = static_cast<const T*>(a.v) + u.k.begin * a.v_stride[0] + hk * a.v_stride[1];
  const float c = a.scale * kLog2e;
  auto load_q = [&](float* d1, float* d2, int32_t first, int rows) {
    load_tile<T, DP>(d1, q, a.q_stride[0], a.q_stride[1], hk * group, group, first, rows, a.dim, vec);
    load_tile<T, DP>(d2, dout, a.dout_stride[0], a.dout_stride[1], hk * group, group, first, rows, a.dim, vec);
    if (threadIdx.x < kTile) {
      const int r = threadIdx.x;
      float l = INFINITY, e = 0.f;  // exp2(s - inf) = 0: rows that are not there, or saw no key
      if (r < rows) {
        const int64_t at = static_cast<int64_t>(u.q.begin + (first + r) / group) * a.heads + hk * group + (first + r) % group;
        l = a.lse[at] == -INFINITY ? INFINITY : a.lse[at] * kLog2e;
        e = a.delta[at];
      }
      s_lse[r] = l;
      s_delta[r] = e;
    }
  };
  auto load_k = [&](float* d1, float* d2, int32_t first) {
    const int rows = u.k.count - first < kTile ? u.k.count - first : kTile;
    load_tile<T, DP>(d1, k, a.k_stride[0], 0, 0, 1, first, rows, a.dim, vec);
    load_tile<T, DP>(d2, v, a.v_stride[0], 0, 0, 1, first, rows, a.dim, vec);
  };
  float acc1[4][W], acc2[4][W];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < W; ++j) acc1[i][j] = acc2[i][j] = 0.f;
  const int32_t all = u.q.count * group;  // packed rows of the item
  int32_t t0, t1, first;                  // the tile's first row, and the range of what passes
  int rows;
  if constexpr (kDQ) {
    t0 = u.tile * per_tile * group;
    rows = all - t0 < per_tile * group ? all - t0 : per_tile * group;
    load_q(a1, a2, t0, rows);
    first = u.split * cut.chunk;
    t1 = keys_seen(u, (t0 + rows - 1) / group, a.causal);
    if (u.splits > 1 && t1 - first > cut.chunk) t1 = first + cut.chunk;
  } else {
    t0 = u.tile * kTile;
    rows = u.k.count - t0 < kTile ? u.k.count - t0 : kTile;
    load_k(a1, a2, t0);
    // the first query that sees key t0
    const int64_t f = a.causal ? static_cast<int64_t>(t0) + u.q.count - u.k.count : 0;
    const int32_t q_lo = u.split * cut.chunk;
    first = (f < q_lo ? q_lo : static_cast<int32_t>(f)) * group;
    t1 = u.splits > 1 && u.q.count - q_lo > cut.chunk ? (q_lo + cut.chunk) * group : all;
  }
  for (int32_t b0 = first; b0 < t1; b0 += kTile) {
    __syncthreads();
    if constexpr (kDQ) load_k(b1, b2, b0);
    else load_q(b1, b2, b0, t1 - b0 < kTile ? t1 - b0 : kTile);
    cp_commit();
    cp_wait<0>();
    __syncthreads();
    if ((ty & ~1) * 4 >= rows) continue;  // a warp without rows only loads
    float s[4][4], dp[4][4];
    mm_nt<DP>(a1, b1, ty, tx, s);
    mm_nt<DP>(a2, b2, ty, tx, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 4 * ty + i, x = tx + 16 * j;
        const int lr = kDQ ? r : x;  // the query's place in the tile
        const int32_t pq = (kDQ ? t0 + r : b0 + x), key = kDQ ? b0 + x : t0 + r;
        const bool see = pq < (kDQ ? all : t1) && key < keys_seen(u, pq / group, a.causal);
        const float p = see ? exp2f(s[i][j] * c - s_lse[lr]) : 0.f;
        s[i][j] = p;
        dp[i][j] = see ? p * (dp[i][j] - s_delta[lr]) : 0.f;
      }
    }
    if constexpr (!kDQ) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sp[(4 * ty + i) * (kTile + 4) + tx + 16 * j] = s[i][j];
      __syncwarp();
      mm_nn<DP>(sp, b2, ty, tx, acc2);
      __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sp[(4 * ty + i) * (kTile + 4) + tx + 16 * j] = dp[i][j];
    __syncwarp();
    mm_nn<DP>(sp, b1, ty, tx, acc1);
    __syncwarp();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ty + i;
    if (r >= rows) continue;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const int cc = col_of<DP>(tx, j);
      if (cc >= a.dim) continue;
      if (u.splits > 1) {  // k_attn_bwd_sum adds the splits up
        if constexpr (kDQ) {
          const int64_t at = static_cast<int64_t>(u.q.begin + (t0 + r) / group) * a.heads + hk * group + (t0 + r) % group;
          part[(u.split * a.n * a.heads + at) * a.dim + cc] = acc1[i][j] * a.scale;
        } else {
          const int64_t at = (u.split * a.m + u.k.begin + t0 + r) * a.kv_heads + hk;
          part[2 * at * a.dim + cc] = acc1[i][j] * a.scale;
          part[(2 * at + 1) * a.dim + cc] = acc2[i][j];
        }
      } else if constexpr (kDQ) {
        const int pr = t0 + r;
        static_cast<T*>(a.dq)[static_cast<int64_t>(u.q.begin + pr / group) * a.dq_stride[0] +
                              (hk * group + pr % group) * a.dq_stride[1] + cc] = from_f<T>(acc1[i][j] * a.scale);
      } else {
        const int64_t row = static_cast<int64_t>(u.k.begin) + t0 + r;
        static_cast<T*>(a.dk)[row * a.dk_stride[0] + hk * a.dk_stride[1] + cc] = from_f<T>(acc1[i][j] * a.scale);
        static_cast<T*>(a.dv)[row * a.dv_stride[0] + hk * a.dv_stride[1] + cc] = from_f<T>(acc2[i][j]);
      }
    }
  }
}

// One of the backward pass's two halves: how its rows are cut into blocks, and
// where the sums of its splits go.
struct Half {
  Cut cut;
  float* part;
};

// The dK / dV blocks, then those of dQ, in one grid: neither waits for the other's last.
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, DP <= 64 ? 2 : 1)
    k_attn_bwd(const __grid_constant__ AttnArgs a, const Half hk, const Half hq, uint32_t kunits, bool vec) {
  if (blockIdx.x < kunits) gradients<T, DP, false>(a, hk.cut, vec, hk.part, blockIdx.x);
  else gradients<T, DP, true>(a, hq.cut, vec, hq.part, blockIdx.x - kunits);
}

// Adds up the splits of a tile's gradients, in order.
template <typename T, bool kDQ>
__device__ __forceinline__ void add_splits(const AttnArgs& a, Cut tiles, const float* part, int64_t ux) {
  __shared__ Unit unit;
  const int chunk = tiles.chunk;
  tiles.chunk = 0;
  find_unit<kThreads>(tiles, ux, &unit, a.err);
  const Unit u = unit;
  grid_wait();
  if (u.item < 0) return;
  const int hk = blockIdx.y, group = kDQ ? a.heads / a.kv_heads : 1, per = static_cast<int>(tiles.per_tile.d);
  const Span own = kDQ ? u.q : u.k;
  const int32_t other = kDQ ? u.k.count : u.q.count, t0 = u.tile * per;
  if (other <= chunk) return;  // one split, written as it is
  const int splits = (other - 1) / chunk + 1;
  const int rows = (own.count - t0 < per ? own.count - t0 : per) * group, width = (kDQ ? 1 : 2) * a.dim;
  const int64_t step = (kDQ ? a.n * a.heads : a.m * a.kv_heads) * width;
  for (int i = blockIdx.z * kThreads + threadIdx.x; i < rows * width; i += gridDim.z * kThreads) {
    const int r = i / width, c = i - r * width;
    const int64_t row = static_cast<int64_t>(own.begin) + t0 + r / group;
    const int head = hk * group + r % group;
    const float* from = part + (row * (kDQ ? a.heads : a.kv_heads) + head) * width + c;
    float t = 0.f;
#pragma unroll 4
    for (int s = 0; s < splits; ++s) t += from[s * step];
    if (kDQ) static_cast<T*>(a.dq)[row * a.dq_stride[0] + head * a.dq_stride[1] + c] = from_f<T>(t);
    else if (c < a.dim) static_cast<T*>(a.dk)[row * a.dk_stride[0] + head * a.dk_stride[1] + c] = from_f<T>(t);
    else static_cast<T*>(a.dv)[row * a.dv_stride[0] + head * a.dv_stride[1] + c - a.dim] = from_f<T>(t);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_attn_bwd_sum(const AttnArgs a, const Half hk, const Half hq, uint32_t ktiles) {
  if (blockIdx.x < ktiles) add_splits<T, false>(a, hk.cut, hk.part, blockIdx.x);
  else add_splits<T, true>(a, hq.cut, hq.part, blockIdx.x - ktiles);
}

// delta[row, head] = sum of dO * O over the head, one warp each.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_attn_delta(const AttnArgs a) {
  allow_next();
  const int64_t total = a.n * a.heads;
  const int lane = threadIdx.x & 31;
  for (int64_t w = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5; w < total;
       w += static_cast<int64_t>(gridDim.x) * (kThreads / 32)) {
    const int64_t row = w / a.heads;
    const T* o = static_cast<const T*>(a.out) + w * a.dim;
    const T* d = static_cast<const T*>(a.dout) + row * a.dout_stride[0] + (w - row * a.heads) * a.dout_stride[1];
    float s = 0.f;
    for (int j = lane; j < a.dim; j += 32) s += to_f(o[j]) * to_f(d[j]);
    s = group_sum<32>(s);
    if (lane == 0) a.delta[w] = s;
  }
}

template <typename K>
cudaError_t allow_smem(K kern, size_t bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
}

// fp32 operands whose rows are whole 16-byte pieces at 16-byte places.
bool whole_pieces(const AttnArgs& a, bool backward) {
  auto ok = [&](const void* p, const int64_t st[2]) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && st[0] % 4 == 0 && st[1] % 4 == 0;
  };
  return a.dtype == kF32 && a.dim % 4 == 0 && ok(a.q, a.q_stride) && ok(a.k, a.k_stride) && ok(a.v, a.v_stride) &&
         (!backward || ok(a.dout, a.dout_stride));
}

// Runs of keys (attn_join.cuh), for three blocks and more to each of an SM's two
// places (1500 and 903 rows over 1374 and 700 keys, 4 heads of 64: 121 us, three at
// most: 140 us; 64 queries, 8 heads of 64 over 2: 39 us split, 35 and 59 us whole over
// 300 and 600 keys); the join moves four channels at a time.
int split_of(const AttnArgs& a, int sms) {
  const bool fits = a.dim % 4 == 0 && (reinterpret_cast<uintptr_t>(a.out_w) & 15u) == 0;
  return fits ? attn::split_keys(a, kTile / (a.heads / a.kv_heads), 6ll * sms, 384, false) : 0;
}

// Backward: rows of a split of what passes (keys for dQ, queries for dK and dV),
// or 0: where there are fewer than one and a half blocks to each of the machine's
// places, for about two and a half, whole tiles of packed rows, at least two.  (One,
// one and a half, two and a half, four blocks: 2500 causal rows, 8 heads of 128 over 2,
// took 3188, 3188, 2503, 2480 us, 3000 rows, 4 heads of 64, 975, 914, 930, 937 us.)
int bwd_split(const AttnArgs& a, int sms, bool dq) {
  const int group = a.heads / a.kv_heads, per = dq ? kTile / group : kTile;
  const int64_t places = static_cast<int64_t>(sms) * (a.dim <= 64 ? 2 : 1);
  const int64_t blocks = ((dq ? a.n : a.m) / per + a.items) * a.kv_heads, other = dq ? a.m : a.n;
  if (2 * blocks > 3 * places || a.items == 0) return 0;
  const int64_t runs = (5 * places / 2 + blocks - 1) / blocks, whole = dq ? kTile : kTile / group;
  int64_t chunk = (other / runs + whole - 1) / whole * whole;
  if (chunk < 2 * whole) chunk = 2 * whole;
  return other <= chunk ? 0 : static_cast<int>(chunk);
}

// fp32 words of the splits' sums.
int64_t bwd_words(const AttnArgs& a, int sms, bool dq) {
  const int chunk = bwd_split(a, sms, dq);
  if (!chunk) return 0;
  return dq ? ((a.m - 1) / chunk + 1) * a.n * a.heads * a.dim : ((a.n - 1) / chunk + 1) * a.m * a.kv_heads * 2 * a.dim;
}

template <typename T, int DP>
cudaError_t launch_bwd(const AttnArgs& a, float* scratch, int sms, cudaStream_t s) {
  const size_t bytes = (4 * kTile * (DP + 4) + kTile * (kTile + 4)) * sizeof(float);
  cudaError_t e = allow_smem(k_attn_bwd<T, DP>, bytes);
  if (e != cudaSuccess) return e;
  int64_t tiles[2], units[2];  // of dK and dV, of dQ
  Half half[2];
  for (int x = 0; x < 2; ++x) {
    const bool dq = x == 1;
    const int per = dq ? kTile / (a.heads / a.kv_heads) : kTile, chunk = bwd_split(a, sms, dq);
    const int64_t rows = dq ? a.n : a.m, other = dq ? a.m : a.n;
    tiles[x] = rows > 0 ? rows / per + a.items : 0;
    units[x] = chunk ? tiles[x] + (rows / per + 1) * (other / chunk) : tiles[x];
    half[x].cut = {a.q_off, a.k_off, static_cast<int32_t>(a.n), static_cast<int32_t>(a.m), a.items, chunk, divisor(per), !dq};
    half[x].part = dq ? scratch + bwd_words(a, sms, false) : scratch;
  }
  const dim3 grid(static_cast<unsigned>(units[0] + units[1]), a.kv_heads);
  const uint32_t kunits = static_cast<uint32_t>(units[0]);
  const bool vec = whole_pieces(a, true);
  if (a.n > 0) {  // behind k_attn_delta
    e = launch_after(k_attn_bwd<T, DP>, grid, kThreads, bytes, s, a, half[0], half[1], kunits, vec);
    if (e != cudaSuccess) return e;
  } else {
    k_attn_bwd<T, DP><<<grid, kThreads, bytes, s>>>(a, half[0], half[1], kunits, vec);
  }
  count_launches(1);
  for (int x = 0; x < 2; ++x)
    if (!half[x].cut.chunk) tiles[x] = 0;  // nothing to add up
  if (tiles[0] + tiles[1] > 0) {
    e = launch_after(k_attn_bwd_sum<T>, dim3(static_cast<unsigned>(tiles[0] + tiles[1]), a.kv_heads, 8), kThreads, 0, s,
                     a, half[0], half[1], static_cast<uint32_t>(tiles[0]));
    if (e != cudaSuccess) return e;
    count_launches(1);
  }
  return cudaGetLastError();
}

template <typename T, int DP>
cudaError_t launch_dim(const AttnArgs& a, bool backward, float* scratch, int chunk, int sms, cudaStream_t s) {
  const int per_tile = kTile / (a.heads / a.kv_heads);
  int64_t units = a.n / per_tile + a.items;
  if (chunk) units += (a.n / per_tile + 1) * (a.m / chunk);
  const dim3 qgrid(static_cast<unsigned>(units), a.kv_heads);
  Cut cut = {a.q_off, a.k_off, static_cast<int32_t>(a.n), static_cast<int32_t>(a.m), a.items, chunk, divisor(per_tile), false};
  if (!backward) {
    const size_t bytes = (3 * kTile * (DP + 4) + kTile * (kTile + 4)) * sizeof(float);
    const cudaError_t e = allow_smem(k_attn<T, DP>, bytes);
    if (e != cudaSuccess) return e;
    float* part_ml = chunk ? scratch + ((a.m - 1) / chunk + 1) * a.n * a.heads * a.dim : nullptr;
    k_attn<T, DP><<<qgrid, kThreads, bytes, s>>>(a, cut, whole_pieces(a, false), chunk ? scratch : nullptr, part_ml);
    count_launches(chunk ? 2 : 1);
    const cudaError_t launched = cudaGetLastError();
    return chunk && launched == cudaSuccess ? attn::launch_join<T>(a, cut, scratch, part_ml, s) : launched;
  }
  const int64_t want = (a.n * a.heads + 7) / 8;
  if (a.n > 0) {
    k_attn_delta<T><<<static_cast<unsigned>(want < 4096 ? want : 4096), kThreads, 0, s>>>(a);
    count_launches(1);
  }
  return launch_bwd<T, DP>(a, scratch, sms, s);
}

template <typename T>
cudaError_t launch_typed(const AttnArgs& a, bool backward, float* scratch, int chunk, int sms, cudaStream_t s) {
  if (a.dim <= 32) return launch_dim<T, 32>(a, backward, scratch, chunk, sms, s);
  if (a.dim <= 64) return launch_dim<T, 64>(a, backward, scratch, chunk, sms, s);
  if (a.dim <= 96) return launch_dim<T, 96>(a, backward, scratch, chunk, sms, s);
  return launch_dim<T, 128>(a, backward, scratch, chunk, sms, s);
}

}  // namespace

int64_t attn_simt_bwd_scratch(const AttnArgs& a, int sms) {
  return bwd_words(a, sms, true) + bwd_words(a, sms, false);
}

int64_t attn_simt_scratch(const AttnArgs& a, int sms) {
  return attn::split_words(a, split_of(a, sms)) * static_cast<int64_t>(sizeof(float));
}

cudaError_t launch_attn_simt(const AttnArgs& a, bool backward, void* scratch, int sms, cudaStream_t s) {
  const int chunk = backward ? 0 : split_of(a, sms);
  float* x = static_cast<float*>(scratch);
  if (a.dtype == kF32) return launch_typed<float>(a, backward, x, chunk, sms, s);
  if (a.dtype == kBF16) return launch_typed<__nv_bfloat16>(a, backward, x, chunk, sms, s);
  return launch_typed<__half>(a, backward, x, chunk, sms, s);
}

}  // namespace smc
