// Rotary positions: pairs of a head's channels turned by angles that grow with
// the row's position along one or more axes (rope phases from voxel
// coordinates: Pixal3D commit log and shared sparse-core commit log,
// "rope_phases_from_coords").
//
//   angle(n, a, f) = positions[n, a] * freqs[a, f],  pair p = a * F + f
//   (u, v) -> scale * (u cos - v sin, u sin + v cos)
//
// over pairs (2p, 2p + 1) (interleaved) or (p, P + p) (half) of the first 2P
// channels, P = axes * F; the channels behind them pass through.  The inverse
// turns by -angle with the same scale: the gradient of the forward turn.
//
// Angles: positions reach millions of steps, where an fp32 product is off by
// whole radians, so the product, the division by 2 pi and the reduction to
// half a turn are in fp64; only the reduced angle is rounded to fp32, and
// sincospif takes it from there.  One thread serves one chunk of channels of
// a row (16 bytes, or one pair where strides or sizes do not allow that) for
// a run of heads, so the angles are paid once per run.  The bytes (82 MB) take HBM
// 12.5 us for 20,011 x 16 x 64 bf16 over three axes, the kernel 19 us, 4.4 TB/s:
// latency, of the angles (fp64, then a sine and cosine) and of the loads, which are
// issued ahead of them (21 us behind them); HBM is at 27%, the FMA pipe at 18%, the
// special-function unit at 10% of their peaks.  Half layout with pairs that are not
// whole 16-byte chunks takes 22 us for a dense x in L2 (interleaved 16 us).  The run of
// heads is as long as the number of rows allows with the machine full.
#include "kernels.h"
#include "tokens.cuh"

namespace smc {

namespace {

constexpr int kThreads = 256;

template <typename T>
struct RotArgs {
  const T* x;
  T* out;
  const int32_t* pos;
  const double* freqs;
  int64_t n, xs_row, xs_head, os_row, os_head, ps_row, ps_axis;
  int heads, dim, axes, nfreq, runs;  // runs: threads that share a chunk's heads
  float scale;
  bool inverse;
};

// cos and sin of pair p of row `row`, times scale.
template <typename T>
__device__ __forceinline__ float2 turn_of(const RotArgs<T>& a, int64_t row, int p) {
  const int axis = a.axes == 1 ? 0 : p / a.nfreq;
  const double t = static_cast<double>(a.pos[row * a.ps_row + axis * a.ps_axis]) * __ldg(a.freqs + p);
  double turns = t * 0.15915494309189533577;  // 1 / (2 pi)
  turns -= rint(turns);
  float s, c;
  sincospif(static_cast<float>(2.0 * turns), &s, &c);
  return make_float2(c * a.scale, (a.inverse ? -s : s) * a.scale);
}

// One unit: chunk `ch` of a row for the heads h0, h0 + runs, h0 + 2 runs, ...
// kHalf: EPC pairs (a chunk and its partner P channels on), or a chunk behind
// the pairs.  Otherwise: EPC / 2 pairs of one chunk (EPC = 1: two channels).
template <typename T, int EPC, bool kHalf>
__global__ void __launch_bounds__(kThreads) k_rotary(const RotArgs<T> a) {
  constexpr int kElems = EPC == 1 && !kHalf ? 2 : EPC;  // channels of a chunk
  constexpr int kPairs = kHalf ? EPC : kElems / 2;
  using C = Chunk<T, EPC>;
  const int pairs = a.axes * a.nfreq;
  const int paired = kHalf ? pairs / EPC : 0;  // units that hold two chunks
  const int per_row = kHalf ? paired + (a.dim - 2 * pairs + EPC - 1) / EPC : (a.dim + kElems - 1) / kElems;
  const int runs = a.runs;
  const int64_t total = a.n * per_row * runs;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; u < total;
       u += static_cast<int64_t>(gridDim.x) * kThreads) {
    int64_t rest, row;
    if (total < (int64_t{1} << 31)) {  // a 64-bit division takes longer than the turn of a chunk
      rest = static_cast<uint32_t>(u) / static_cast<uint32_t>(per_row);
      row = static_cast<uint32_t>(rest) / static_cast<uint32_t>(runs);
    } else {
      rest = u / per_row;
      row = rest / runs;
    }
    // The heads of a run are `runs` apart, so that neighbouring threads touch
    // neighbouring heads.
    const int ch = static_cast<int>(u - rest * per_row), h0 = static_cast<int>(rest - row * runs);
    const int count = (a.heads - 1 - h0) / runs + 1;
    const T* x = a.x + row * a.xs_row + h0 * a.xs_head;
    T* y = a.out + row * a.os_row + h0 * a.os_head;
    const int64_t xs = a.xs_head * runs, ys = a.os_head * runs;
    float2 cs[kPairs];
    if constexpr (kHalf) {
      constexpr int kBatch = 2;
      const bool two = ch < paired;
      const int lo = two ? ch * EPC : 2 * pairs + (ch - paired) * EPC, second = two ? pairs : 0;
      x += lo;
      y += lo;
      C cu[kBatch], cv[kBatch];
      auto fetch = [&](int h) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b, x += xs)
          if (h + b < count) {
            cu[b] = *reinterpret_cast<const C*>(x);
            cv[b] = *reinterpret_cast<const C*>(x + second);
          }
      };
      fetch(0);
      if (two) {
#pragma unroll
        for (int i = 0; i < EPC; ++i) cs[i] = turn_of(a, row, lo + i);
      }
      for (int h = 0; h < count; h += kBatch) {
        if (h > 0) fetch(h);
#pragma unroll
        for (int b = 0; b < kBatch; ++b, y += ys) {
          if (h + b >= count) break;
          if (!two) {
            *reinterpret_cast<C*>(y) = cu[b];
            continue;
          }
          float fu[EPC], fv[EPC], ru[EPC], rv[EPC];
          unpack(cu[b], fu);
          unpack(cv[b], fv);
#pragma unroll
          for (int i = 0; i < EPC; ++i) {
            ru[i] = fu[i] * cs[i].x - fv[i] * cs[i].y;
            rv[i] = fu[i] * cs[i].y + fv[i] * cs[i].x;
          }
          *reinterpret_cast<C*>(y) = pack<T, EPC>(ru);
          *reinterpret_cast<C*>(y + pairs) = pack<T, EPC>(rv);
        }
      }
    } else if constexpr (EPC == 1) {
      const int lo = ch * kElems;
      const bool two = lo / 2 < pairs, both = lo + 1 < a.dim;
      if (two) cs[0] = turn_of(a, row, lo / 2);
      for (int h = 0; h < count; ++h, x += xs, y += ys) {
        const T u0 = x[lo], v0 = both ? x[lo + 1] : u0;
        const float fu = to_f(u0), fv = to_f(v0);
        y[lo] = two ? from_f<T>(fu * cs[0].x - fv * cs[0].y) : u0;
        if (both) y[lo + 1] = two ? from_f<T>(fu * cs[0].y + fv * cs[0].x) : v0;
      }
    } else {
      constexpr int kBatch = 4;
      const int lo = ch * kElems;
      x += lo;
      y += lo;
      C c[kBatch];
      auto fetch = [&](int h) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b, x += xs)
          if (h + b < count) c[b] = *reinterpret_cast<const C*>(x);
      };
      fetch(0);
#pragma unroll
      for (int i = 0; i < kPairs; ++i)
        cs[i] = lo / 2 + i < pairs ? turn_of(a, row, lo / 2 + i) : make_float2(1.f, 0.f);
      for (int h = 0; h < count; h += kBatch) {
        if (h > 0) fetch(h);
#pragma unroll
        for (int b = 0; b < kBatch; ++b, y += ys) {
          if (h + b >= count) break;
          float f[EPC], r[EPC];
          unpack(c[b], f);
#pragma unroll
          for (int i = 0; i < EPC / 2; ++i) {
            r[2 * i] = f[2 * i] * cs[i].x - f[2 * i + 1] * cs[i].y;
            r[2 * i + 1] = f[2 * i] * cs[i].y + f[2 * i + 1] * cs[i].x;
          }
          C o = pack<T, EPC>(r);
          if (lo / 2 + EPC / 2 > pairs) {  // channels behind the pairs keep their bits
#pragma unroll
            for (int i = 0; i < EPC; ++i)
              if (lo / 2 + i / 2 >= pairs) o.v[i] = c[b].v[i];
          }
          *reinterpret_cast<C*>(y) = o;
        }
      }
    }
  }
}

template <typename T>
cudaError_t launch_typed(const RotaryArgs& b, int sms, cudaStream_t s) {
  constexpr int kWide = 16 / sizeof(T);
  RotArgs<T> a;
  a.x = static_cast<const T*>(b.x);
  a.out = static_cast<T*>(b.out);
  a.pos = b.positions;
  a.freqs = b.freqs;
  a.n = b.n;
  a.xs_row = b.x_stride[0];
  a.xs_head = b.x_stride[1];
  a.os_row = b.out_stride[0];
  a.os_head = b.out_stride[1];
  a.ps_row = b.pos_stride[0];
  a.ps_axis = b.pos_stride[1];
  a.heads = b.heads;
  a.dim = b.dim;
  a.axes = b.axes;
  a.nfreq = b.nfreq;
  a.scale = b.scale;
  a.inverse = b.inverse;
  const int pairs = a.axes * a.nfreq;
  auto whole = [&](int64_t v) { return v % kWide == 0; };
  // Where one pair and head to a thread does not fill the machine, the angles
  // (fp64, about 5 us for the eight of a 16-byte chunk) are what takes the time:
  // one to a thread then.
  const bool few = a.n * a.heads * a.dim <= static_cast<int64_t>(sms) * 1024;
  const bool vec = !few && ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out)) & 15u) == 0 &&
                   whole(a.xs_row) && whole(a.xs_head) && whole(a.os_row) && whole(a.os_head) && whole(a.dim) &&
                   (!b.half || whole(pairs));
  const int elems = vec ? kWide : (b.half ? 1 : 2);
  const int64_t per_row = b.half ? pairs / elems + (a.dim - 2 * pairs + elems - 1) / elems : (a.dim + elems - 1) / elems;
  // A run of heads as long as leaves a thousand threads on each SM (20011 x 16 x
  // 64 bf16 over three axes: 1024, 2048, 4096, 8192 threads took 21, 22, 26, 35 us).
  const int64_t fill = static_cast<int64_t>(sms) * 1024;
  int64_t run = a.n * per_row * a.heads / fill;
  run = run < 1 ? 1 : (run > a.heads ? a.heads : run);
  a.runs = static_cast<int>((a.heads + run - 1) / run);
  const int64_t total = a.n * per_row * a.runs;
  const int64_t want = (total + kThreads - 1) / kThreads, cap = static_cast<int64_t>(sms) * 64;
  const unsigned blocks = static_cast<unsigned>(want < cap ? want : cap);
  if (b.half) {
    if (vec) k_rotary<T, kWide, true><<<blocks, kThreads, 0, s>>>(a);
    else k_rotary<T, 1, true><<<blocks, kThreads, 0, s>>>(a);
  } else {
    if (vec) k_rotary<T, kWide, false><<<blocks, kThreads, 0, s>>>(a);
    else k_rotary<T, 1, false><<<blocks, kThreads, 0, s>>>(a);
  }
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int sms, cudaStream_t s) {
  if (a.dtype == kF32) return launch_typed<float>(a, sms, s);
  if (a.dtype == kBF16) return launch_typed<__nv_bfloat16>(a, sms, s);
  return launch_typed<__half>(a, sms, s);
}

}  // namespace smc
