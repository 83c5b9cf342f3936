// Device helpers of the token-wise layers (layer norm, rotary positions,
// attention): element conversion, 16-byte chunks of a row, and the search for
// a block's share of the items' rows.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace smc {

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

// Rows [begin, begin + count) of one item, cut to [0, n): whatever the offsets
// hold, no row outside the buffers is touched.
struct Span {
  int32_t begin, count;
};

__device__ __forceinline__ Span item_span(const int32_t* offsets, int item, int64_t n, bool* bad) {
  const int64_t a = __ldg(offsets + item), b = __ldg(offsets + item + 1);
  const int64_t lo = a < 0 ? 0 : (a > n ? n : a);
  const int64_t hi = b < lo ? lo : (b > n ? n : b);
  if (a < 0 || b < a || b > n) *bad = true;
  return {static_cast<int32_t>(lo), static_cast<int32_t>(hi - lo)};
}

// A block's share: tile `tile` of item `item`'s rows, over the keys of its
// split (split 0 of 1: all of them).  item < 0: nothing to do.
struct Unit {
  int32_t item, tile, split, splits;
  Span q, k;
};

// Units of an item: (tiles of `per_tile` rows) x (splits of `chunk` keys,
// chunk 0: one split).  tile_k: the tiles cut the keys instead of the queries.
__device__ __forceinline__ int32_t units_of(Span q, Span k, int per_tile, int chunk, bool tile_k, int32_t* splits) {
  const int32_t rows = tile_k ? k.count : q.count;
  const int32_t sp = chunk > 0 && k.count > chunk ? (k.count + chunk - 1) / chunk : 1;
  *splits = sp;
  return (rows / per_tile + (rows % per_tile ? 1 : 0)) * sp;
}

// Finds unit `u` (every thread of the block calls this; the answer is in
// shared memory).  Each thread adds up the units of a run of items, a block
// scan numbers the runs, and the thread whose run holds u walks it: one pass
// over the offsets, about a microsecond for up to a few thousand items, so the
// host needs no lengths and no table is built.
template <int kThreads>
__device__ __forceinline__ void find_unit(const int32_t* q_off, const int32_t* k_off, int items, int64_t n, int64_t m,
                                          int per_tile, int chunk, bool tile_k, int64_t u, Unit* out, uint32_t* err) {
  static_assert(kThreads % 32 == 0, "whole warps");
  __shared__ int64_t s_warp[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (items + kThreads - 1) / kThreads;
  const int i0 = tid * run < items ? tid * run : items, i1 = i0 + run < items ? i0 + run : items;
  if (tid == 0) out->item = -1;
  int64_t mine = 0;
  int32_t sp;
  bool bad = false;
  for (int i = i0; i < i1; ++i)
    mine += units_of(item_span(q_off, i, n, &bad), item_span(k_off, i, m, &bad), per_tile, chunk, tile_k, &sp);
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int64_t before = incl - mine;
  for (int w = 0; w < warp; ++w) before += s_warp[w];
  if (bad && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(err, kErrRange);
  if (u >= before && u < before + mine) {
    int64_t at = before;
    for (int i = i0; i < i1; ++i) {
      const Span q = item_span(q_off, i, n, &bad), k = item_span(k_off, i, m, &bad);
      const int32_t cnt = units_of(q, k, per_tile, chunk, tile_k, &sp);
      if (u < at + cnt) {
        const int32_t r = static_cast<int32_t>(u - at);
        *out = {i, r / sp, r % sp, sp, q, k};
        break;
      }
      at += cnt;
    }
  }
  __syncthreads();
}

}  // namespace smc
