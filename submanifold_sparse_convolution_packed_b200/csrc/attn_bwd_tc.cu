// Gradients of attention within each item on the tensor cores (bf16 / fp16,
// sm_100a), with P recomputed from the saved lse:
//
//   P = exp2(S log2e - lse log2e),  dS = P * (dP - delta),  dP = dO V^T
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO
//
// Two launches of one kernel.  A CTA keeps 128 rows of two operands in shared
// memory (queries: Q and dO, for dQ; keys: K and V, for dK and dV) and passes
// 64 rows of the other two through a ring, so every sum over the passing rows
// stays in one TMEM accumulator: no atomics, no fp32 copy of dQ in memory, and
// the same bits every time, at the price of computing S and dP twice (7
// products instead of 5).  The scores of the dK / dV launch are computed
// transposed (keys are the rows), so that P^T and dS^T, written to TMEM by the
// threads that hold their rows, are the A operands of the products as they
// lie; Q, dO, K are read a second time from the same shared memory, MN-major.
//   warp 9     TMA: the resident tiles once, then the passing ones, with the
//              lse and delta of their rows (dK / dV);
//   warp 8     tcgen05.mma: S and dP of step j + 1 are issued before the
//              products of step j, into the other of two TMEM buffers;
//   warps 0-3, 4-7  P and dS of even and odd steps, one thread per row.
// fp16: P carries a factor 2^14 and dS a power of two taken from the largest
// norms of dO and V rows (|dP|, |delta| <= |dO| |V|), undone on the fp32
// accumulators, so that the P of a long context do not fall below fp16's
// range and dS cannot leave it.
#include <type_traits>

#include "attn_tc.cuh"

namespace smc {

namespace {

using namespace attn;

constexpr int kThreads = 320;
constexpr int kStep = 64;                       // passing rows of a step
constexpr uint32_t kStepPanel = kStep * 128;

struct BwdParams {
  const int32_t *q_off, *k_off;
  int64_t n, m;
  int items, heads, kv_heads, dim, group;
  int qpt, qps;  // queries of a resident tile, of a step
  float scale;
  bool causal;
  const float *lse, *delta;
  const uint32_t* norms;  // fp16: bits of max |dO|^2, max |V|^2
  void *d1, *d2;          // dQ, -- or dK, dV
  int64_t s1[2], s2[2];
  uint32_t* err;
  uint64_t wait_ns;
};

template <int DP> struct BwdLayout {
  static constexpr uint32_t kResident = DP / 64 * kPanel, kPass = DP / 64 * kStepPanel;
  static constexpr int kSlots = DP == 64 ? 6 : 4;
  static constexpr uint32_t kA = 0, kB = 2 * kResident, kRowVals = kB + kSlots * 2 * kPass;
  static constexpr uint32_t kBar = kRowVals + kSlots * 2 * kStep * 4;
  // barriers: resident, full[kSlots], empty[kSlots], s[2], p[2], out, tail
  static constexpr uint32_t kMisc = kBar + 8 * (2 * kSlots + 7), kTotal = kMisc + 32 + 1024;
};

// The power of two that dS carries in fp16.
__device__ __forceinline__ float ds_factor(const uint32_t* norms) {
  if (!norms) return 1.f;
  const float bound = 2.f * sqrtf(__uint_as_float(norms[0])) * sqrtf(__uint_as_float(norms[1]));
  if (!(bound > 0.f) || !(bound < 1e37f)) return 1.f;
  int e = 15 - (ilogbf(bound) + 1);  // |dS| <= bound, so |dS| 2^e <= 2^15
  e = e < -60 ? -60 : (e > 60 ? 60 : e);
  return exp2f(static_cast<float>(e));
}

template <typename T, int DP, bool kDQ>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_bwd_tc(const __grid_constant__ CUtensorMap a1map, const __grid_constant__ CUtensorMap a2map,
                  const __grid_constant__ CUtensorMap b1map, const __grid_constant__ CUtensorMap b2map,
                  const BwdParams p) {
  using L = BwdLayout<DP>;
  constexpr int kSlots = L::kSlots, kPanels = DP / 64;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr float kShift = kBf16 || kDQ ? 0.f : 14.f;  // P carries 2^kShift
  extern __shared__ uint8_t smem_raw[];
  __shared__ Unit s_unit;
  const uint32_t raw = smem_u32(smem_raw), sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  volatile uint32_t* s_misc = reinterpret_cast<volatile uint32_t*>(smem + L::kMisc);  // [0] tmem, [1] abort
  const uint32_t bar_a = sbase + L::kBar, bar_full = bar_a + 8, bar_empty = bar_full + 8 * kSlots;
  const uint32_t bar_s = bar_empty + 8 * kSlots, bar_p = bar_s + 16, bar_o = bar_p + 16, bar_tail = bar_o + 8;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // causal: the tiles with the most work (the last queries, the first keys) start first
  const int64_t ux = kDQ && p.causal ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
  find_unit<kThreads>(p.q_off, p.k_off, p.items, p.n, p.m, kDQ ? p.qpt : kRows, 0, !kDQ, ux, &s_unit, p.err);
  if (s_unit.item < 0) return;
  const Unit u = s_unit;
  const int hk = blockIdx.y;
  // resident rows [r0, r0 + count) (queries or keys), passing rows [b_lo, b_hi)
  const int32_t r0 = u.tile * (kDQ ? p.qpt : kRows);
  const int32_t have = (kDQ ? u.q.count : u.k.count) - r0, most = kDQ ? p.qpt : kRows;
  const int32_t count = have < most ? have : most;
  int32_t b_lo = 0, b_hi;
  const int32_t per_step = kDQ ? kStep : p.qps;
  if (kDQ) {
    b_hi = keys_seen(u, r0 + count - 1, p.causal);
  } else {
    b_hi = u.q.count;
    if (p.causal) {  // the first query that sees key r0
      const int64_t f = static_cast<int64_t>(r0) + u.q.count - u.k.count;
      b_lo = f < 0 ? 0 : (f < b_hi ? static_cast<int32_t>(f) : b_hi);
    }
  }
  const int nsteps = b_hi > b_lo ? (b_hi - b_lo + per_step - 1) / per_step : 0;

  if (tid == 0) {
    prefetch_tmap(&a1map);
    prefetch_tmap(&a2map);
    prefetch_tmap(&b1map);
    prefetch_tmap(&b2map);
    mbar_init(bar_a, 1);
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(bar_full + 8 * s, kDQ ? 1 : 2);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar_s + 8 * t, 1);
      mbar_init(bar_p + 8 * t, 4);
    }
    mbar_init(bar_o, 1);
    mbar_init(bar_tail, 1);
    s_misc[1] = 0;
    fence_mbarrier_init();
  }
  const int rows_step = kDQ ? kStep : p.qps * p.group;  // rows of a step that the TMA writes
  if (rows_step < kStep) {  // the others must not hold NaN bits: zero, once
    for (int s = 0; s < kSlots * 2 * kPanels; ++s) {
      uint4* base = reinterpret_cast<uint4*>(smem + L::kB + s * kStepPanel);
      for (int j = rows_step * 8 + tid; j < kStep * 8; j += kThreads) base[j] = make_uint4(0, 0, 0, 0);
    }
  }
  fence_proxy_async_smem();
  if (warp == 8) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(&s_misc[0])), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_misc[0];

  if (warp == 9) {
    // ------------------------------------------------------------- TMA loads
    if (nsteps > 0) {
      const float f = kDQ ? 1.f : ds_factor(p.norms) * exp2f(-kShift);
      if (elect_one()) {
        const uint32_t rows = kDQ ? p.group * p.qpt : kRows;
        mbar_arrive_expect_tx(bar_a, 2 * kPanels * rows * 128u);
        const int head = kDQ ? hk * p.group : hk, row = (kDQ ? u.q.begin : u.k.begin) + r0;
        for (int c = 0; c < kPanels; ++c) {
          tma_load_3d(sbase + L::kA + c * kPanel, &a1map, bar_a, c * 64, head, row);
          tma_load_3d(sbase + L::kA + L::kResident + c * kPanel, &a2map, bar_a, c * 64, head, row);
        }
      }
      __syncwarp();
      // lse and delta of the step's rows, fetched a step ahead
      float l[2], e[2];
      auto fetch = [&](int j) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = lane + 32 * h, qi = b_lo + j * per_step + r / p.group;
          l[h] = INFINITY;  // exp2(s - inf) = 0: rows that are not there, or saw no key
          e[h] = 0.f;
          if (r < rows_step && qi < b_hi) {
            const int64_t at = static_cast<int64_t>(u.q.begin + qi) * p.heads + hk * p.group + r % p.group;
            const float v = __ldg(p.lse + at);
            if (v != -INFINITY) {
              l[h] = v * kLog2e - kShift;
              e[h] = p.delta[at] * f;
            }
          }
        }
      };
      if (!kDQ) fetch(0);
      for (int j = 0; j < nsteps; ++j) {
        const int slot = j % kSlots;
        int ok = 1;
        if (lane == 0)
          ok = mbar_wait_bounded(bar_empty + 8 * slot, ((j / kSlots) & 1) ^ 1, p.err, p.wait_ns) && !s_misc[1];
        if (!__shfl_sync(0xffffffffu, ok, 0)) {
          if (lane == 0) s_misc[1] = 1;
          break;
        }
        const int32_t b0 = b_lo + j * per_step;
        const int rows = (b_hi - b0 < per_step ? b_hi - b0 : per_step) * (kDQ ? 1 : p.group);
        // in the dQ launch b_hi may be the causal limit: rows behind it are the item's own, but not seen
        const bool tail = rows < rows_step;
        const uint32_t dst = sbase + L::kB + slot * 2 * L::kPass, bar = tail ? bar_tail : bar_full + 8 * slot;
        if (elect_one()) {
          mbar_arrive_expect_tx(bar, 2 * kPanels * static_cast<uint32_t>(rows_step) * 128u);
          const int head = kDQ ? hk : hk * p.group, row = (kDQ ? u.k.begin : u.q.begin) + b0;
          for (int c = 0; c < kPanels; ++c) {
            tma_load_3d(dst + c * kStepPanel, &b1map, bar, c * 64, head, row);
            tma_load_3d(dst + L::kPass + c * kStepPanel, &b2map, bar, c * 64, head, row);
          }
        }
        __syncwarp();
        if (!kDQ) {
          float* vals = reinterpret_cast<float*>(smem + L::kRowVals) + slot * 2 * kStep;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            vals[lane + 32 * h] = l[h];
            vals[kStep + lane + 32 * h] = e[h];
          }
          if (j + 1 < nsteps) fetch(j + 1);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_full + 8 * slot);
        }
        if (tail) {  // once, at the last step: rows that are not the item's may hold NaN
          ok = mbar_wait_bounded(bar_tail, 0, p.err, p.wait_ns);
          if (!__all_sync(0xffffffffu, ok)) {
            if (lane == 0) s_misc[1] = 1;
            break;
          }
          for (int c = 0; c < 2 * kPanels; ++c) {
            uint4* base = reinterpret_cast<uint4*>(smem + L::kB + slot * 2 * L::kPass + c * kStepPanel);
            for (int i = rows * 8 + lane; i < rows_step * 8; i += 32) base[i] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_full + 8 * slot);
        }
      }
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------- MMA issue
    const uint32_t ab = kBf16 ? 1u : 0u;
    const int ks = (p.dim + 15) / 16;
    const uint32_t idesc_s = idesc_f16(ab, kStep), idesc_o = idesc_f16(ab, static_cast<uint32_t>(ks * 16)) | kIdescBMn;
    bool ok = nsteps > 0;
    auto wait = [&](uint32_t bar, uint32_t parity) {
      const bool w = mbar_wait_bounded(bar, parity, p.err, p.wait_ns);
      if (!__all_sync(0xffffffffu, w && !s_misc[1])) {
        if (lane == 0) s_misc[1] = 1;
        ok = false;
      }
      tc_fence_after();
    };
    auto scores = [&](int j) {  // S and dP of step j
      const uint32_t b = sbase + L::kB + (j % kSlots) * 2 * L::kPass, d = tmem + (j & 1) * 2 * kStep;
#pragma unroll
      for (int x = 0; x < 2; ++x)
        for (int k = 0; k < ks; ++k) {
          const uint64_t off = 2 * (k & 3);
          umma_f16_elect(d + x * kStep, kmajor_desc(sbase + L::kA + x * L::kResident + (k >> 2) * kPanel, 128) + off,
                         kmajor_desc(b + x * L::kPass + (k >> 2) * kStepPanel, 128) + off, idesc_s, k > 0);
        }
      umma_commit_elect(bar_s + 8 * (j & 1));
    };
    if (ok) wait(bar_a, 0);
    if (ok) wait(bar_full, 0);
    if (ok) scores(0);
    for (int j = 0; j < nsteps && ok; ++j) {
      const int slot = j % kSlots;
      if (j + 1 < nsteps) {
        wait(bar_full + 8 * ((j + 1) % kSlots), ((j + 1) / kSlots) & 1);
        if (!ok) break;
        scores(j + 1);
      }
      wait(bar_p + 8 * (j & 1), (j >> 1) & 1);
      if (!ok) break;
      const uint32_t b = sbase + L::kB + slot * 2 * L::kPass, d = tmem + (j & 1) * 2 * kStep;
      if (!kDQ) {
#pragma unroll
        for (int k = 0; k < kStep / 16; ++k)
          umma_f16_ts_elect(tmem + 4 * kStep + DP, d + 8 * k, mnmajor_desc(b + L::kPass, kStepPanel) + 128 * k, idesc_o,
                            j > 0 || k > 0);
      }
#pragma unroll
      for (int k = 0; k < kStep / 16; ++k)
        umma_f16_ts_elect(tmem + 4 * kStep, d + kStep + 8 * k, mnmajor_desc(b, kStepPanel) + 128 * k, idesc_o,
                          j > 0 || k > 0);
      if (j + kSlots < nsteps) umma_commit_elect(bar_empty + 8 * slot);
    }
    if (ok) umma_commit_elect(bar_o);
  } else {
    // ---------------------------------------------------------------- P, dS
    const int w = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t buf = tmem + lanes + w * 2 * kStep;
    const float c = p.scale * kLog2e, factor = ds_factor(p.norms), f = factor * exp2f(-kShift);
    const int32_t qi = kDQ ? r / p.group : 0;
    const bool row = kDQ ? qi < count : r < count;
    float l = INFINITY, e = 0.f;  // dQ: of this thread's query
    int32_t lim = 0;              // dQ: keys [0, lim) are seen; dK / dV: packed query rows [lim, ..) of the item see the key
    if (kDQ) {
      if (row) {
        const int64_t at = static_cast<int64_t>(u.q.begin + r0 + qi) * p.heads + hk * p.group + r % p.group;
        const float v = __ldg(p.lse + at);
        if (v != -INFINITY) {
          l = v * kLog2e;
          e = p.delta[at] * f;
        }
        lim = keys_seen(u, r0 + qi, p.causal);
      }
    } else if (p.causal) {
      const int64_t first = static_cast<int64_t>(r0) + r + u.q.count - u.k.count;  // the first query that sees this key
      lim = first < 0 ? 0 : static_cast<int32_t>(first < u.q.count ? first : u.q.count) * p.group;
    }
    bool ok = true;
    for (int j = w; j < nsteps; j += 2) {
      const int slot = j % kSlots;
      if (!kDQ) ok = mbar_wait_bounded(bar_full + 8 * slot, (j / kSlots) & 1, p.err, p.wait_ns);  // the row values
      ok = ok && mbar_wait_bounded(bar_s + 8 * w, (j >> 1) & 1, p.err, p.wait_ns);
      if (!__all_sync(0xffffffffu, ok && !s_misc[1])) {
        s_misc[1] = 1;
        ok = false;
        break;
      }
      tc_fence_after();
      float s[kStep], d[kStep];
      tmem_ld(buf, s);
      tmem_ld(buf + kStep, d);
      uint32_t wp[kStep / 2], ws[kStep / 2];
      const int32_t b0 = b_lo + j * per_step;
      // columns [from, to) of this row count
      const int from = kDQ ? 0 : lim - b0 * p.group, to = kDQ ? lim - b0 : kStep;
      const bool whole = __all_sync(0xffffffffu, from <= 0 && to >= kStep);
      const float4* vl = reinterpret_cast<const float4*>(smem + L::kRowVals) + slot * 2 * (kStep / 4);
#pragma unroll
      for (int i = 0; i < kStep; i += 4) {
        float4 l4 = make_float4(l, l, l, l), e4 = make_float4(e, e, e, e);
        if (!kDQ) {
          l4 = vl[i / 4];
          e4 = vl[kStep / 4 + i / 4];
        }
        float pv[4], dv[4];
        pv[0] = exp2_fast(fmaf(s[i], c, -l4.x));
        pv[1] = exp2_fast(fmaf(s[i + 1], c, -l4.y));
        pv[2] = exp2_fast(fmaf(s[i + 2], c, -l4.z));
        pv[3] = exp2_fast(fmaf(s[i + 3], c, -l4.w));
        dv[0] = pv[0] * fmaf(d[i], f, -e4.x);
        dv[1] = pv[1] * fmaf(d[i + 1], f, -e4.y);
        dv[2] = pv[2] * fmaf(d[i + 2], f, -e4.z);
        dv[3] = pv[3] * fmaf(d[i + 3], f, -e4.w);
        if (!whole) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const bool see = i + x >= from && i + x < to;
            pv[x] = see ? pv[x] : 0.f;
            dv[x] = see ? dv[x] : 0.f;
          }
        }
        if (!kDQ) {
          wp[i / 2] = pack2<T>(pv[0], pv[1]);
          wp[i / 2 + 1] = pack2<T>(pv[2], pv[3]);
        }
        ws[i / 2] = pack2<T>(dv[0], dv[1]);
        ws[i / 2 + 1] = pack2<T>(dv[2], dv[3]);
      }
      if (!kDQ) tmem_st(buf, wp);
      tmem_st(buf + kStep, ws);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_p + 8 * w);
    }
    // --------------------------------------------------------------- results
    if (ok && nsteps > 0) {
      ok = mbar_wait_bounded(bar_o, 0, p.err, p.wait_ns);
      ok = __all_sync(0xffffffffu, ok && !s_misc[1]);
      tc_fence_after();
    }
    if (ok) {
      // dQ: the warps of the two halves take half of the columns each; dK / dV: one of the two each
      const int c_lo = kDQ ? w * (DP / 2) : 0, c_hi = kDQ ? c_lo + DP / 2 : DP;
      const bool second = !kDQ && w == 1;
      const uint32_t acc = tmem + lanes + 4 * kStep + (second ? DP : 0);
      const float mul = second ? exp2f(-kShift) : p.scale / factor;
      const int64_t out_row = kDQ ? static_cast<int64_t>(u.q.begin) + r0 + qi : static_cast<int64_t>(u.k.begin) + r0 + r;
      const int head = kDQ ? hk * p.group + r % p.group : hk;
      T* to = static_cast<T*>(second ? p.d2 : p.d1) + out_row * (second ? p.s2[0] : p.s1[0]) +
              head * (second ? p.s2[1] : p.s1[1]);
#pragma unroll 1
      for (int c0 = c_lo; c0 < c_hi; c0 += 32) {
        if (c0 >= p.dim) break;
        float o[32];
        if (nsteps > 0) {
          tmem_ld(acc + c0, o);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.f;
        }
        if (!row) continue;
        uint4* d = reinterpret_cast<uint4*>(to + c0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c0 + 8 * i < p.dim)
            d[i] = make_uint4(pack2<T>(o[8 * i] * mul, o[8 * i + 1] * mul), pack2<T>(o[8 * i + 2] * mul, o[8 * i + 3] * mul),
                              pack2<T>(o[8 * i + 4] * mul, o[8 * i + 5] * mul),
                              pack2<T>(o[8 * i + 6] * mul, o[8 * i + 7] * mul));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, 512);
}

// delta[row, head] = sum of dO * O; fp16: also the largest squared norms of
// the rows of dO and of V that belong to items (as bits: they are not
// negative).  LPR lanes hold a row of up to 8 LPR channels.
template <typename T, int LPR>
__global__ void __launch_bounds__(256) k_attn_delta_tc(const AttnArgs a, uint32_t* norms) {
  using C = Chunk<T, 8>;
  const int l = threadIdx.x % LPR;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (256 / LPR), first = static_cast<int64_t>(blockIdx.x) * (256 / LPR);
  const bool in = 8 * l < a.dim;
  auto bounds = [](const int32_t* off, int items, int64_t n, int64_t& lo, int64_t& hi) {
    lo = __ldg(off);
    hi = __ldg(off + items);
    lo = lo < 0 ? 0 : (lo > n ? n : lo);
    hi = hi < lo ? lo : (hi > n ? n : hi);
  };
  int64_t lo, hi;
  bounds(a.q_off, a.items, a.n, lo, hi);
  float top = 0.f, vtop = 0.f;
  const T* O = static_cast<const T*>(a.out);
  const T* D = static_cast<const T*>(a.dout);
  for (int64_t b = lo * a.heads + first; b < hi * a.heads; b += stride) {
    const int64_t i = b + threadIdx.x / LPR, row = i / a.heads;
    const bool there = i < hi * a.heads;
    float s = 0.f, q = 0.f;
    if (there && in) {
      float o[8], d[8];
      unpack(*reinterpret_cast<const C*>(O + i * a.dim + 8 * l), o);
      unpack(*reinterpret_cast<const C*>(D + row * a.dout_stride[0] + (i - row * a.heads) * a.dout_stride[1] + 8 * l), d);
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        s += o[x] * d[x];
        q += d[x] * d[x];
      }
    }
    s = group_sum<LPR>(s);
    if (there && l == 0) a.delta[i] = s;
    if (norms) top = fmaxf(top, group_sum<LPR>(q));
  }
  if (!norms) return;
  bounds(a.k_off, a.items, a.m, lo, hi);
  const T* V = static_cast<const T*>(a.v);
  for (int64_t b = lo * a.kv_heads + first; b < hi * a.kv_heads; b += stride) {
    const int64_t i = b + threadIdx.x / LPR, row = i / a.kv_heads;
    float q = 0.f;
    if (i < hi * a.kv_heads && in) {
      float v[8];
      unpack(*reinterpret_cast<const C*>(V + row * a.v_stride[0] + (i - row * a.kv_heads) * a.v_stride[1] + 8 * l), v);
#pragma unroll
      for (int x = 0; x < 8; ++x) q += v[x] * v[x];
    }
    vtop = fmaxf(vtop, group_sum<LPR>(q));
  }
  __shared__ uint32_t s_top[2];
  if (threadIdx.x < 2) s_top[threadIdx.x] = 0;
  __syncthreads();
  atomicMax(&s_top[0], __float_as_uint(top));
  atomicMax(&s_top[1], __float_as_uint(vtop));
  __syncthreads();
  if (threadIdx.x < 2) atomicMax(norms + threadIdx.x, s_top[threadIdx.x]);
}

template <typename T, int DP>
cudaError_t launch_typed(const AttnArgs& a, BwdParams p, const CUtensorMap* maps, int sms, uint32_t* norms,
                         cudaStream_t st) {
  const int64_t rows = a.n * a.heads, per = DP == 64 ? 32 : 16;
  int64_t blocks = (rows + per - 1) / per;
  blocks = blocks < 8ll * sms ? (blocks < 1 ? 1 : blocks) : 8ll * sms;
  if (norms) {
    const cudaError_t e = cudaMemsetAsync(norms, 0, 2 * sizeof(uint32_t), st);
    if (e != cudaSuccess) return e;
  }
  k_attn_delta_tc<T, DP / 8><<<static_cast<unsigned>(blocks), 256, 0, st>>>(a, norms);
  constexpr int kSmem = static_cast<int>(BwdLayout<DP>::kTotal);
  auto kq = k_attn_bwd_tc<T, DP, true>;
  auto kk = k_attn_bwd_tc<T, DP, false>;
  cudaError_t e = cudaFuncSetAttribute(kq, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kk, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  p.d1 = a.dq;
  for (int i = 0; i < 2; ++i) p.s1[i] = a.dq_stride[i];
  kq<<<dim3(static_cast<unsigned>(a.n / p.qpt + a.items), a.kv_heads), kThreads, kSmem, st>>>(maps[0], maps[1], maps[2],
                                                                                             maps[3], p);
  p.d1 = a.dk;
  p.d2 = a.dv;
  for (int i = 0; i < 2; ++i) {
    p.s1[i] = a.dk_stride[i];
    p.s2[i] = a.dv_stride[i];
  }
  kk<<<dim3(static_cast<unsigned>(a.m / kRows + a.items), a.kv_heads), kThreads, kSmem, st>>>(maps[4], maps[5], maps[6],
                                                                                              maps[7], p);
  count_launches(3);
  return cudaGetLastError();
}

bool out_fits(const void* p, const int64_t st[2]) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && st[0] % 8 == 0 && st[1] % 8 == 0;
}

}  // namespace

bool attn_bwd_tc_supported(const AttnArgs& a) {
  return a.dtype != kF32 && a.dim % 8 == 0 && a.n > 0 && a.m > 0 && map_fits(a.q, a.q_stride) &&
         map_fits(a.k, a.k_stride) && map_fits(a.v, a.v_stride) && map_fits(a.dout, a.dout_stride) &&
         out_fits(a.dq, a.dq_stride) && out_fits(a.dk, a.dk_stride) && out_fits(a.dv, a.dv_stride) &&
         (reinterpret_cast<uintptr_t>(a.out) & 15u) == 0 && encode_fn() != nullptr;
}

cudaError_t launch_attn_bwd_tc(const AttnArgs& a, uint32_t* norms, int sms, cudaStream_t st) {
  const int group = a.heads / a.kv_heads;
  BwdParams p = {};
  p.qpt = kRows / group;
  p.qps = kStep / group;
  CUtensorMap maps[8];
  auto queries = [&](CUtensorMap* m, const void* t, const int64_t s[2], int per) {
    return make_map(m, t, a.dtype, a.n, a.heads, a.dim, s, group, per);
  };
  auto keys = [&](CUtensorMap* m, const void* t, const int64_t s[2], int per) {
    return make_map(m, t, a.dtype, a.m, a.kv_heads, a.dim, s, 1, per);
  };
  if (!queries(&maps[0], a.q, a.q_stride, p.qpt) || !queries(&maps[1], a.dout, a.dout_stride, p.qpt) ||
      !keys(&maps[2], a.k, a.k_stride, kStep) || !keys(&maps[3], a.v, a.v_stride, kStep) ||
      !keys(&maps[4], a.k, a.k_stride, kRows) || !keys(&maps[5], a.v, a.v_stride, kRows) ||
      !queries(&maps[6], a.q, a.q_stride, p.qps) || !queries(&maps[7], a.dout, a.dout_stride, p.qps))
    return cudaErrorInvalidValue;
  p.q_off = a.q_off;
  p.k_off = a.k_off;
  p.n = a.n;
  p.m = a.m;
  p.items = a.items;
  p.heads = a.heads;
  p.kv_heads = a.kv_heads;
  p.dim = a.dim;
  p.group = group;
  p.scale = a.scale;
  p.causal = a.causal;
  p.lse = a.lse;
  p.delta = a.delta;
  if (a.dtype != kF16) norms = nullptr;
  p.norms = norms;
  p.err = a.err;
  // never below 100 ms, so that no CTA leaves with its loads in flight
  p.wait_ns = scan_wait_limit_ns() > 100000000ull ? scan_wait_limit_ns() : 100000000ull;
  if (a.dtype == kBF16)
    return a.dim <= 64 ? launch_typed<__nv_bfloat16, 64>(a, p, maps, sms, norms, st)
                       : launch_typed<__nv_bfloat16, 128>(a, p, maps, sms, norms, st);
  return a.dim <= 64 ? launch_typed<__half, 64>(a, p, maps, sms, norms, st)
                     : launch_typed<__half, 128>(a, p, maps, sms, norms, st);
}

}  // namespace smc
