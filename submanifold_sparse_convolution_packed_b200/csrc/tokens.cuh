// Device helpers of the token-wise layers (layer norm, rotary positions,
// attention): element conversion, 16-byte chunks of a row, and the search for
// a block's share of the items' rows.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace smc {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
// One rounding to nearest even, of the finished fp32 value.
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }

// EPC consecutive elements moved as one access: 16 bytes, or one element.
template <typename T, int EPC> struct alignas(sizeof(T) * EPC) Chunk { T v[EPC]; };

__device__ __forceinline__ float2 to_f2(__nv_bfloat16 a, __nv_bfloat16 b) {
  return __bfloat1622float2(__halves2bfloat162(a, b));
}
__device__ __forceinline__ float2 to_f2(__half a, __half b) { return __half22float2(__halves2half2(a, b)); }

template <typename T, int EPC>
__device__ __forceinline__ void unpack(const Chunk<T, EPC>& c, float (&f)[EPC]) {
  if constexpr (sizeof(T) == 2 && EPC % 2 == 0) {
#pragma unroll
    for (int i = 0; i < EPC; i += 2) {
      const float2 t = to_f2(c.v[i], c.v[i + 1]);
      f[i] = t.x;
      f[i + 1] = t.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPC; ++i) f[i] = to_f(c.v[i]);
  }
}

__device__ __forceinline__ void from_f2(float a, float b, __nv_bfloat16* x) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  x[0] = h.x;
  x[1] = h.y;
}
__device__ __forceinline__ void from_f2(float a, float b, __half* x) {
  const __half2 h = __floats2half2_rn(a, b);
  x[0] = h.x;
  x[1] = h.y;
}

template <typename T, int EPC>
__device__ __forceinline__ Chunk<T, EPC> pack(const float (&f)[EPC]) {
  Chunk<T, EPC> c;
  if constexpr (sizeof(T) == 2 && EPC % 2 == 0) {
#pragma unroll
    for (int i = 0; i < EPC; i += 2) from_f2(f[i], f[i + 1], &c.v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < EPC; ++i) c.v[i] = from_f<T>(f[i]);
  }
  return c;
}

// 2^x, within 2 ulp; results below the normal range are zero.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Sum over groups of W neighbouring lanes (W a power of two, at most 32).
template <int W>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A kernel launched with launch_after may start while the one before it on the
// stream ends: what does not depend on that one (its share, its barriers) stands
// before grid_wait, which returns once that one is complete and its writes are
// seen.  allow_next lets the next one start once all blocks have started; without
// it, once they have exited.  (Gradients of 300 rows, 4 heads of 64 over 2, bf16: 16
// to 12 us.)  Every thread of such a kernel comes by grid_wait, so that the kernel is
// complete only behind the one before it.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_after(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kern, P(args)...);
}

// Rows [begin, begin + count) of one item, cut to [0, n): whatever the offsets
// hold, no row outside the buffers is touched.
struct Span {
  int32_t begin, count;
};

__device__ __forceinline__ Span span_of(int32_t a, int32_t b, int32_t n, bool* bad) {
  const int32_t lo = min(max(a, 0), n), hi = min(max(b, lo), n);
  *bad = *bad || a != lo || b != hi;
  return {lo, hi - lo};
}

// Division of a count below 2^31 by d, prepared on the host: x / d =
// x * ceil(2^(31 + s) / d) >> (31 + s) with 2^s >= d.
struct Divisor {
  uint32_t d, mul, shift;
};

inline Divisor divisor(uint32_t d) {
  uint32_t s = 0;
  while ((1ull << s) < d) ++s;
  return {d, static_cast<uint32_t>(((1ull << (31 + s)) + d - 1) / d), 31 + s};
}

__device__ __forceinline__ uint32_t over(uint32_t x, Divisor d) {
  return d.d == 1 ? x : static_cast<uint32_t>((static_cast<uint64_t>(x) * d.mul) >> d.shift);
}

// A block's share: tile `tile` of item `item`'s rows, over the other side's rows
// of its split (split 0 of 1: all of them).  item < 0: nothing to do.
struct Unit {
  int32_t item, tile, split, splits;
  Span q, k;
};

// Keys that query `qi` of an item sees: the first ones, this many.
__device__ __forceinline__ int32_t keys_seen(const Unit& u, int64_t qi, bool causal) {
  if (!causal) return u.k.count;
  const int64_t s = qi + u.k.count - u.q.count + 1;
  return s < 0 ? 0 : (s > u.k.count ? u.k.count : static_cast<int32_t>(s));
}

// How the items' rows are cut into units: tiles of per_tile.d rows (queries, or
// keys with by_keys) x splits of `chunk` rows of the other side (0: one split).
struct Cut {
  const int32_t *q_off, *k_off;
  int32_t n, m;
  int items, chunk;
  Divisor per_tile;
  bool by_keys;
};

__device__ __forceinline__ int32_t units_of(const Cut& c, Span q, Span k, int32_t* splits) {
  const uint32_t rows = static_cast<uint32_t>(c.by_keys ? k.count : q.count);
  const int32_t other = c.by_keys ? q.count : k.count;
  int32_t sp = 1;
  if (c.chunk > 0 && other > c.chunk) sp = (other - 1) / c.chunk + 1;
  *splits = sp;
  return static_cast<int32_t>(over(rows + c.per_tile.d - 1, c.per_tile)) * sp;
}

// Finds unit `u` (every thread of the block calls this; the answer is in
// shared memory, after a barrier).  Each thread adds up the units of a run of
// up to kRun items, whose offsets it loads together; a block scan numbers the
// runs, and the thread whose run holds u names it: one latency for up to
// kRun * kThreads items (more take further rounds), so the host needs no
// lengths and no table is built.  It stands at the start of every block, so
// its instructions count where items are short.
template <int kThreads>
__device__ __forceinline__ void find_unit(const Cut& c, int64_t u, Unit* out, uint32_t* err) {
  static_assert(kThreads % 32 == 0, "whole warps");
  constexpr int kRun = 4, kWarps = kThreads / 32;
  __shared__ int64_t s_warp[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) out->item = -1;
  int64_t done = 0;  // units of the rounds before this one
  for (int first = 0; first < c.items; first += kRun * kThreads) {
    const int left = c.items - first;
    const int run = left >= kRun * kThreads ? kRun : (left + kThreads - 1) / kThreads;
    const int i0 = first + tid * run;
    int32_t q[kRun + 1], k[kRun + 1], cnt[kRun];
    int64_t mine = 0;
    bool bad = false;
#pragma unroll
    for (int x = 0; x <= kRun; ++x)
      if (x <= run && i0 + x <= c.items) {
        q[x] = __ldg(c.q_off + i0 + x);
        k[x] = c.q_off == c.k_off ? q[x] : __ldg(c.k_off + i0 + x);
      }
#pragma unroll
    for (int x = 0; x < kRun; ++x) {
      cnt[x] = 0;
      if (x < run && i0 + x < c.items) {
        int32_t sp;
        cnt[x] = units_of(c, span_of(q[x], q[x + 1], c.n, &bad), span_of(k[x], k[x + 1], c.m, &bad), &sp);
      }
      if (x < run) mine += cnt[x];
    }
    int64_t incl = mine;
    if (first + warp * 32 * run < c.items) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
    }
    if (lane == 31) s_warp[warp] = incl;
    if (bad && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(err, kErrRange);
    __syncthreads();
    // the sums of the warps before this one, and of all
    int64_t before = 0, all = 0;
    const int busy = (left + 32 * run - 1) / (32 * run) < kWarps ? (left + 32 * run - 1) / (32 * run) : kWarps;
    for (int w = 0; w < busy; ++w) {
      const int64_t v = s_warp[w];
      all += v;
      if (w < warp) before += v;
    }
    int64_t at = done + before + incl - mine;
    if (u >= at && u < at + mine) {
#pragma unroll
      for (int x = 0; x < kRun; ++x) {
        if (x < run && u >= at && u < at + cnt[x]) {
          const Span sq = span_of(q[x], q[x + 1], c.n, &bad), sk = span_of(k[x], k[x + 1], c.m, &bad);
          int32_t sp;
          units_of(c, sq, sk, &sp);
          const int32_t r = static_cast<int32_t>(u - at);
          *out = {i0 + x, r / sp, r % sp, sp, sq, sk};
        }
        at += cnt[x];
      }
    }
    done += all;
    __syncthreads();
    // block 0 looks at every item, for the error word
    if (u < done && (blockIdx.x != 0 || blockIdx.y != 0)) break;
  }
}

}  // namespace smc
