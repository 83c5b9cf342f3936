// Attention over runs of keys: when to split the keys between blocks, and the
// kernel that joins the blocks' partial results.
#pragma once

#include <cstdint>

#include "kernels.h"
#include "tokens.cuh"

namespace smc {
namespace attn {

// Keys of a run, or 0 for no split: when tiles of `per` queries leave half of the
// machine's `slots` for blocks idle and there are `least` keys, runs of about
// (keys x tiles) / slots, at least 256 keys; within: as short as keep all blocks, the
// items' last runs among them, within the slots.  Items of one run are written as
// they are; the join passes over them.  (Half: single queries, 16 heads of 128 over 4,
// 296 slots.  37 of them, just past it, over 8000 keys each take 141 us whole and 149
// split, over 1000 to 32,768 keys 488 and 310 us; 64 of them 159 and 277, 528 and
// 544 us: unequal lengths would gain from runs a little further on.)
inline int split_keys(const AttnArgs& a, int per, int64_t slots, int64_t least, bool within) {
  const int64_t tiles = a.n / per + a.items;  // upper bound
  if (2 * tiles * a.kv_heads > slots || a.m < least) return 0;
  int64_t chunk = a.m * (a.n / per + 1) / (slots / a.kv_heads - (within ? tiles : 0));
  chunk = (chunk < 256 ? 256 : chunk + 127) / 128 * 128;
  return a.m <= chunk ? 0 : static_cast<int>(chunk);  // no item is longer than one run
}

// fp32 words of the partial results: [splits, n, heads, dim] and (maximum in
// units of log2, sum), [splits, n, heads, 2].
inline int64_t split_words(const AttnArgs& a, int chunk) {
  return chunk ? ((a.m - 1) / chunk + 1) * a.n * a.heads * (a.dim + 2) : 0;
}

struct JoinParams {
  Cut tiles;  // of queries, no splits
  int chunk, heads, dim, group;
  const float *part_o, *part_ml;
  void* out;
  float* lse;
  uint32_t* err;
};

// Joins the splits of a tile's rows, in order: O = sum 2^(top_s - top) O_s / sum ...
// One warp to a row; lane s holds the weight of split s (32 at a time), so that
// the loads of the splits' rows depend on nothing.
template <typename T>
__global__ void __launch_bounds__(256) k_attn_join(const JoinParams p) {
  __shared__ Unit s_unit;
  find_unit<256>(p.tiles, blockIdx.x, &s_unit, p.err);
  const Unit u = s_unit;
  grid_wait();
  if (u.item < 0) return;
  const int hk = blockIdx.y, lane = threadIdx.x & 31;
  const int32_t per = static_cast<int32_t>(p.tiles.per_tile.d), q0 = u.tile * per;
  const int32_t queries = u.q.count - q0 < per ? u.q.count - q0 : per;
  if (u.k.count <= p.chunk) return;  // one run
  const int splits = (u.k.count - 1) / p.chunk + 1;
  const int64_t step = static_cast<int64_t>(p.tiles.n) * p.heads;
  for (int r = blockIdx.z * 8 + (threadIdx.x >> 5); r < queries * p.group; r += gridDim.z * 8) {
    const int64_t at = static_cast<int64_t>(u.q.begin + q0 + r / p.group) * p.heads + hk * p.group + r % p.group;
    float top = -INFINITY;
    for (int s = lane; s < splits; s += 32) top = fmaxf(top, p.part_ml[2 * (at + s * step)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    const bool mine = 4 * lane < p.dim;
    for (int s0 = 0; s0 < splits; s0 += 32) {
      const int many = splits - s0 < 32 ? splits - s0 : 32;
      float w = 0.f, l = 0.f;
      if (lane < many) {
        const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * (at + (s0 + lane) * step));
        w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - top);  // -inf: the split's keys are hidden from the row
        l = w * ml.y;
      }
      sum += group_sum<32>(l);
      const float* from = p.part_o + (at + s0 * step) * p.dim + 4 * lane;
#pragma unroll 8
      for (int s = 0; s < many; ++s) {
        const float ws = __shfl_sync(0xffffffffu, w, s);
        if (mine) {
          const float4 v = *reinterpret_cast<const float4*>(from + s * step * p.dim);
          o[0] += ws * v.x, o[1] += ws * v.y, o[2] += ws * v.z, o[3] += ws * v.w;
        }
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const float r4[4] = {o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv};
    if (mine) *reinterpret_cast<Chunk<T, 4>*>(static_cast<T*>(p.out) + at * p.dim + 4 * lane) = pack<T, 4>(r4);
    if (lane == 0 && p.lse) p.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
  }
}

template <typename T>
cudaError_t launch_join(const AttnArgs& a, Cut cut, const float* part_o, const float* part_ml, cudaStream_t s) {
  JoinParams p = {};
  p.chunk = cut.chunk;
  cut.chunk = 0;
  p.tiles = cut;
  p.heads = a.heads;
  p.dim = a.dim;
  p.group = a.heads / a.kv_heads;
  p.part_o = part_o;
  p.part_ml = part_ml;
  p.out = a.out_w;
  p.lse = a.lse_w;
  p.err = a.err;
  // a row takes a warp a microsecond, most of it latency: one or two rows to a warp
  const unsigned rows = cut.per_tile.d * p.group, parts = rows < 16 ? 1 : rows / 16;
  return launch_after(k_attn_join<T>, dim3(static_cast<unsigned>(a.n / cut.per_tile.d + a.items), a.kv_heads, parts), 256,
                      0, s, p);
}

}  // namespace attn
}  // namespace smc
