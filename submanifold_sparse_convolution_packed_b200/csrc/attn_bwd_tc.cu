// Gradients of attention within each item on the tensor cores (bf16 / fp16,
// sm_100a), with P recomputed from the saved lse:
//
//   P = exp2(S log2e - lse log2e),  dS = P * (dP - delta),  dP = dO V^T
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO
//
// Two kinds of blocks in one grid.  A CTA keeps 128 rows of two operands in TMEM (or
// shared memory; queries: Q and dO, for dQ; keys: K and V, for dK and dV) and
// passes 64 rows of the other two through a ring in shared memory, so every sum
// over the passing rows stays in one TMEM accumulator: no atomics, no fp32 copy
// of dQ in memory, and the same bits every time, at the price of computing S and
// dP twice (7 products instead of 5).  The scores of the dK / dV blocks are computed
// transposed (keys are the rows), so that P^T and dS^T, written to TMEM by the
// threads that hold their rows, are the A operands of the products as they
// lie; Q, dO, K are read a second time from the same shared memory, MN-major.
//   warp 17    TMA: the resident tiles once, then the passing ones, with the
//              lse and delta of their rows (dK / dV, cp.async);
//   warp 16    tcgen05.mma: behind the products of step j, S and dP of the step
//              that takes over its TMEM buffer (two or three steps ahead), as
//              one batch: this warp's waits are what there is to save;
//   warps 0-15 P and dS, one thread per row and 16 of the step's 64 columns.
// fp16: P carries a factor 2^14 and dS a power of two, undone on the fp32
// accumulators, so that the P of a long context do not fall below fp16's range
// and dS cannot leave it.  The power of two is each accumulator row's own, from
// |dS| <= |dO| |V| + |delta|: for dQ the query's |dO| and delta and the largest |V|
// of the keys it passes, for dK the key's |V| and the largest |dO| and delta of the
// queries that pass.  So neither another item, nor another head, nor (dQ) another
// query sets the precision of a row; a key's dK is held to 2^-39 of what the largest
// dO among its block's queries could make it.
//
// What bounds it: the chain of a step (products, scores of the step that takes
// its buffer, TMEM to registers, exponentials, back to TMEM); the tensor cores work
// about half of the time.  Measured, whole calls: 9,973 and 8,111 rows, 8 heads of
// 64, bf16: 1.39 ms, 610 TFLOP/s of the five products; 6,007 rows, causal, 8 heads of
// 128 over 2, fp16: 0.28 ms, 670 TFLOP/s.
#include <type_traits>

#include "attn_tc.cuh"

namespace smc {

namespace {

using namespace attn;

constexpr int kThreads = 576;
constexpr int kStep = 64;                       // passing rows of a step
constexpr uint32_t kStepPanel = kStep * 128;

struct BwdParams {
  Cut cut;
  int heads, kv_heads, dim, group;
  int qpt, qps;  // queries of a resident tile, of a step
  float scale;
  bool causal;
  const float *lse, *delta;  // as k_attn_delta_tc leaves them: -lse log2e (-inf for a row that saw no key), -delta
  const float2* qbound;  // fp16: (|dO|^2, |delta|), [heads, n]
  const float* vbound;   // fp16: |V|^2, [kv_heads, m]
  const void *a1, *a2;    // the resident operands: Q, dO or K, V
  int64_t a1s[2], a2s[2];
  void *d1, *d2;          // dQ, -- or dK, dV
  int64_t s1[2], s2[2];
  float* part;  // dK / dV of splits: [splits, m, kv_heads, 2, dim], or null
  uint32_t* err;
  uint64_t wait_ns;
};

template <int DP, bool kDQ> struct BwdLayout {
  static constexpr uint32_t kResident = DP / 64 * kPanel, kPass = DP / 64 * kStepPanel;
  static constexpr int kSlots = DP == 64 ? 6 : 4;
  // TMEM: buffers of S and dP (64 columns each), the accumulators and, where
  // there is room, the resident operands as 16-bit pairs.  From TMEM they cost
  // no shared-memory reads: with 64-column products those reads alone took 48
  // clocks an MMA where the MMA takes 32, and more beside the other traffic.
  static constexpr bool kTmemA = kDQ || DP == 64;  // else K and V in shared memory
  static constexpr int kBufs = kDQ && DP == 64 ? 3 : 2;
  static constexpr uint32_t kAcc = kBufs * 2 * kStep, kAt = kAcc + (kDQ ? 1 : 2) * DP;
  static_assert(kAt + (kTmemA ? DP : 0) <= 512, "TMEM columns");
  static_assert(kBufs < kSlots, "the first steps' loads need no waiting for slots");
  static constexpr uint32_t kA = 0, kB = kTmemA ? 0 : 2 * kResident, kRowVals = kB + kSlots * 2 * kPass;
  static constexpr uint32_t kBar = kRowVals + kSlots * 2 * kStep * 4;
  // barriers: resident, full[kSlots], empty[kSlots], s[kBufs], p[kBufs], out, tail
  static constexpr uint32_t kMisc = kBar + 8 * (2 * kSlots + 2 * kBufs + 3), kTotal = kMisc + 32 + 1024;
};

// The power of two that a row's dS carry in fp16, |dS| <= bound.
__device__ __forceinline__ float ds_factor(float bound) {
  if (!(bound > 0.f) || !(bound < 1e37f)) return 1.f;
  int e = 15 - (ilogbf(bound) + 1);  // |dS| <= bound, so |dS| 2^e <= 2^15
  e = e < -60 ? -60 : (e > 60 ? 60 : e);
  return exp2f(static_cast<float>(e));
}

// Maps of the passing operands and, where the resident ones are read from
// shared memory, of those.
struct BwdMaps {
  CUtensorMap b1, b2, a1, a2;
};

// Unit `ux` of the dQ (kDQ) or of the dK / dV blocks.
template <typename T, int DP, bool kDQ>
__device__ __forceinline__ void gradients(const BwdMaps& maps, const BwdParams& p, int64_t ux) {
  using L = BwdLayout<DP, kDQ>;
  constexpr int kSlots = L::kSlots, kPanels = DP / 64, kBufs = L::kBufs;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr float kShift = kBf16 || kDQ ? 0.f : 14.f;  // P carries 2^kShift
  extern __shared__ uint8_t smem_raw[];
  __shared__ Unit s_unit;
  __shared__ uint32_t s_bound[2];  // fp16: bits of the largest passing |V|^2, or |dO|^2 and |delta|
  const uint32_t raw = smem_u32(smem_raw), sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  volatile uint32_t* s_misc = reinterpret_cast<volatile uint32_t*>(smem + L::kMisc);  // [0] tmem
  const uint32_t bar_a = sbase + L::kBar, bar_full = bar_a + 8, bar_empty = bar_full + 8 * kSlots;
  const uint32_t bar_s = bar_empty + 8 * kSlots, bar_p = bar_s + 8 * kBufs, bar_o = bar_p + 8 * kBufs, bar_tail = bar_o + 8;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  find_unit<kThreads>(p.cut, ux, &s_unit, p.err);
  if (s_unit.item < 0) {
    grid_wait();  // a grid is complete only behind the one before it
    return;
  }
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
    if (u.splits > 1) {
      b_lo = u.split * p.cut.chunk;
      if (b_hi - b_lo > p.cut.chunk) b_hi = b_lo + p.cut.chunk;
    }
    if (p.causal) {  // the first query that sees key r0
      const int64_t f = static_cast<int64_t>(r0) + u.q.count - u.k.count;
      if (f > b_lo) b_lo = f < b_hi ? static_cast<int32_t>(f) : b_hi;
    }
  }
  const int nsteps = b_hi > b_lo ? (b_hi - b_lo + per_step - 1) / per_step : 0;
  if (tid == 0) {
    prefetch_tmap(&maps.b1);
    prefetch_tmap(&maps.b2);
    mbar_init(bar_a, L::kTmemA ? 16 : 1);
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(bar_full + 8 * s, kDQ ? 1 : 33);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int t = 0; t < kBufs; ++t) {
      mbar_init(bar_s + 8 * t, 1);
      mbar_init(bar_p + 8 * t, 16);
    }
    mbar_init(bar_o, 1);
    mbar_init(bar_tail, 1);
    s_bound[0] = s_bound[1] = 0;
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
  if (warp == 16) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(&s_misc[0])), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_misc[0];
  grid_wait();  // for delta, lse2 and the norms

  // Every wait is bounded; a role that gives up leaves its loop, and the others
  // then run out of their own waits.
  if (warp == 17) {
    // ------------------------------------------------------------- TMA loads
    if (nsteps > 0) {
      if (!L::kTmemA && lane == 0) {  // K and V
        mbar_arrive_expect_tx(bar_a, 2 * L::kResident);
        for (int c = 0; c < kPanels; ++c) {
          tma_load_3d(sbase + L::kA + c * kPanel, &maps.a1, bar_a, c * 64, hk, u.k.begin + r0);
          tma_load_3d(sbase + L::kA + L::kResident + c * kPanel, &maps.a2, bar_a, c * 64, hk, u.k.begin + r0);
        }
      }
      __syncwarp();
      int slot = 0;
      uint32_t parity = 1;
      const int head = kDQ ? hk : hk * p.group, base_row = kDQ ? u.k.begin : u.q.begin;
      for (int j = 0; j < nsteps; ++j) {
        if (!mbar_wait_warp(bar_empty + 8 * slot, parity, p.err, p.wait_ns)) break;
        const int32_t b0 = b_lo + j * per_step;
        const int rows = (b_hi - b0 < per_step ? b_hi - b0 : per_step) * (kDQ ? 1 : p.group);
        // for dQ b_hi may be the causal limit: rows behind it are the item's own, but not seen
        const bool tail = rows < rows_step;
        const uint32_t dst = sbase + L::kB + slot * 2 * L::kPass, bar = tail ? bar_tail : bar_full + 8 * slot;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, 2 * kPanels * static_cast<uint32_t>(rows_step) * 128u);
          for (int c = 0; c < kPanels; ++c) {
            tma_load_3d(dst + c * kStepPanel, &maps.b1, bar, c * 64, head, base_row + b0);
            tma_load_3d(dst + L::kPass + c * kStepPanel, &maps.b2, bar, c * 64, head, base_row + b0);
          }
        }
        if (!kDQ) {  // rows that are not there get 0: their S, dP and dO are 0 too, so they add nothing
          const uint32_t vals = sbase + L::kRowVals + slot * 8 * kStep;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = lane + 32 * h;
            const bool there = r < rows;
            const int64_t at =
                there ? static_cast<int64_t>(base_row + b0 + r / p.group) * p.heads + head + r % p.group : 0;
            cp_async4(vals + 4 * r, p.lse + at, there);
            cp_async4(vals + 4 * (kStep + r), p.delta + at, there);
          }
          cp_async_arrive(bar_full + 8 * slot);
        }
        if (tail) {  // once, at the last step: rows that are not the item's may hold NaN
          if (!mbar_wait_warp(bar_tail, 0, p.err, p.wait_ns)) break;
          for (int c = 0; c < 2 * kPanels; ++c) {
            uint4* base = reinterpret_cast<uint4*>(smem + L::kB + slot * 2 * L::kPass + c * kStepPanel);
            for (int i = rows * 8 + lane; i < rows_step * 8; i += 32) base[i] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_full + 8 * slot);
        }
        if (++slot == kSlots) {
          slot = 0;
          parity ^= 1;
        }
      }
    }
  } else if (warp == 16) {
    // ------------------------------------------------------------- MMA issue
    // The whole warp runs the loop; one elected lane issues each batch, with
    // the descriptors advanced by additions only (computing them anew made
    // each MMA cost about 120 clocks of this warp's time, and a step twice as
    // long).
    const uint32_t ab = kBf16 ? 1u : 0u;
    const int ks = (p.dim + 15) / 16;
    const uint32_t idesc_s = idesc_f16(ab, kStep), idesc_o = idesc_f16(ab, static_cast<uint32_t>(ks * 16)) | kIdescBMn;
    const uint64_t a1 = kmajor_desc(sbase + L::kA, 128);
    const uint64_t b1 = kmajor_desc(sbase + L::kB, 128), n1 = mnmajor_desc(sbase + L::kB, kStepPanel);
    constexpr uint64_t kSecondA = L::kResident >> 4, kSecond = L::kPass >> 4, kSlot = 2 * kSecond;
    auto wait2 = [&](uint32_t bar, uint32_t parity, uint32_t bar2, uint32_t parity2) {
      const bool w = mbar_wait_warp(bar, parity, p.err, p.wait_ns) && mbar_wait_warp(bar2, parity2, p.err, p.wait_ns);
      tc_fence_after();
      return w;
    };
    auto scores = [&](uint32_t d, uint64_t b, uint32_t bar) {  // S and dP of a step, in the elected lane
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int k = 0; k < DP / 16; ++k)
          if (k < ks) {
            const uint64_t bk = b + x * kSecond + (k >> 2) * (kStepPanel >> 4) + 2 * (k & 3);
            if (L::kTmemA)
              umma_f16_ts(d + x * kStep, tmem + L::kAt + x * (DP / 2) + 8 * k, bk, idesc_s, k > 0);
            else
              umma_f16(d + x * kStep, a1 + x * kSecondA + (k >> 2) * (kPanel >> 4) + 2 * (k & 3), bk, idesc_s, k > 0);
          }
      umma_commit(bar);
    };
    bool ok = nsteps > 0;
    // step j + kBufs (aslot) takes over the buffer of step j (slot, buf)
    int slot = 0, buf = 0, aslot = 0;
    uint32_t pparity = 0, aparity = 0;
    for (int j = 0; j < kBufs && j < nsteps && ok; ++j) {
      ok = wait2(bar_full + 8 * aslot, 0, bar_a, 0);
      if (ok && elect_one()) scores(tmem + j * 2 * kStep, b1 + aslot * kSlot, bar_s + 8 * j);
      __syncwarp();
      ++aslot;
    }
    for (int j = 0; j < nsteps && ok; ++j) {
      const bool more = j + kBufs < nsteps;
      ok = wait2(bar_p + 8 * buf, pparity, more ? bar_full + 8 * aslot : bar_a, more ? aparity : 0);
      const uint32_t d = tmem + buf * 2 * kStep;
      const uint64_t at = n1 + slot * kSlot;
      if (ok && elect_one()) {
        if (!kDQ) {
#pragma unroll
          for (int k = 0; k < kStep / 16; ++k)
            umma_f16_ts(tmem + L::kAcc + DP, d + 16 * k, at + kSecond + 128 * k, idesc_o, j > 0 || k > 0);
        }
#pragma unroll
        for (int k = 0; k < kStep / 16; ++k)
          umma_f16_ts(tmem + L::kAcc, d + kStep + 16 * k, at + 128 * k, idesc_o, j > 0 || k > 0);
        if (j + kSlots < nsteps) umma_commit(bar_empty + 8 * slot);
        if (more) scores(d, b1 + aslot * kSlot, bar_s + 8 * buf);
        if (j + 1 == nsteps) umma_commit(bar_o);
      }
      __syncwarp();
      if (++slot == kSlots) slot = 0;
      if (++aslot == kSlots) {
        aslot = 0;
        aparity ^= 1;
      }
      if (++buf == kBufs) {
        buf = 0;
        pparity ^= 1;
      }
    }
  } else {
    // ---------------------------------------------------------------- P, dS
    // columns 16 w .. 16 w + 15 of every step; par, half: of the results
    const int w = warp >> 2, r = (warp & 3) * 32 + lane, par = w & 1, half = w >> 1;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float2 c2 = make_float2(p.scale * kLog2e, p.scale * kLog2e);
    const int32_t qi = kDQ ? r / p.group : 0;
    const bool row = kDQ ? qi < count : r < count;
    float l = -INFINITY, e = 0.f;  // dQ: of this thread's query; exp2(s - inf) = 0
    int32_t lim = 0;               // dQ: keys [0, lim) are seen; dK / dV: packed query rows [lim, ..) of the item see the key
    if (kDQ) {
      if (row) {
        const int64_t at = static_cast<int64_t>(u.q.begin + r0 + qi) * p.heads + hk * p.group + r % p.group;
        l = p.lse[at];
        e = p.delta[at];
        lim = keys_seen(u, r0 + qi, p.causal);
      }
    } else if (p.causal) {
      const int64_t first = static_cast<int64_t>(r0) + r + u.q.count - u.k.count;  // the first query that sees this key
      lim = first < 0 ? 0 : static_cast<int32_t>(first < u.q.count ? first : u.q.count) * p.group;
    }
    float factor = 1.f, own = 0.f;  // fp16: of this thread's row
    if (!kBf16 && row)
      own = kDQ ? p.qbound[static_cast<int64_t>(hk * p.group + r % p.group) * p.cut.n + u.q.begin + r0 + qi].x
                : p.vbound[static_cast<int64_t>(hk) * p.cut.m + u.k.begin + r0 + r];
    if (L::kTmemA) {  // this thread's row of the resident operands: 32 words for each of the DP / 32 groups
      if (w < DP / 32) {
        constexpr int kPer = DP / 64;  // groups to an operand
        const bool second = w / kPer == 1;
        const int c0 = (w % kPer) * 64;
        const int64_t* st = second ? p.a2s : p.a1s;
        const int64_t at = kDQ ? (static_cast<int64_t>(u.q.begin) + r0 + qi) * st[0] + (hk * p.group + r % p.group) * st[1]
                               : (static_cast<int64_t>(u.k.begin) + r0 + r) * st[0] + hk * st[1];
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(second ? p.a2 : p.a1) + (row ? at + c0 : 0));
        uint32_t v[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 x = row && c0 + 8 * i < p.dim ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
          v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
        }
        __syncwarp();
        tmem_st(tmem + lanes + L::kAt + (second ? DP / 2 : 0) + c0 / 2, v);
        tmem_st_wait();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_a);
      __syncwarp();
    }
    if (!kBf16) {  // while the first scores are on their way
      float top = 0.f, top2 = 0.f;  // a NaN is passed over: its row's gradients are NaN under any factor
      if (kDQ) {
        const float* v2 = p.vbound + static_cast<int64_t>(hk) * p.cut.m + u.k.begin;
#pragma unroll 4
        for (int32_t i = tid; i < b_hi; i += 512) top = fmaxf(top, v2[i]);
      } else {
        for (int g = 0; g < p.group; ++g) {
          const float2* d2 = p.qbound + static_cast<int64_t>(hk * p.group + g) * p.cut.n + u.q.begin;
#pragma unroll 4
          for (int32_t i = b_lo + tid; i < b_hi; i += 512) {
            const float2 x = d2[i];
            top = fmaxf(top, x.x);
            top2 = fmaxf(top2, x.y);
          }
        }
      }
      // not negative: ordered as their bits
      const uint32_t t1 = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
      const uint32_t t2 = __reduce_max_sync(0xffffffffu, __float_as_uint(top2));
      if (lane == 0) {
        atomicMax(&s_bound[0], t1);
        atomicMax(&s_bound[1], t2);
      }
      asm volatile("bar.sync 1, 512;" ::: "memory");  // these 16 warps
      if (row)
        factor = ds_factor(sqrtf(own) * sqrtf(__uint_as_float(s_bound[0])) + (kDQ ? fabsf(e) : __uint_as_float(s_bound[1])));
    }
    const float2 f2 = make_float2(factor * exp2f(-kShift), factor * exp2f(-kShift));
    int slot = 0, b = 0;
    uint32_t fparity = 0, sparity = 0;
    bool ok = true, ready = false;  // ready: this step's scores were there before the last step's were worked on
    for (int j = 0; j < nsteps; ++j) {
      if (!__all_sync(0xffffffffu, ready)) {
        if (!kDQ) ok = mbar_wait_warp(bar_full + 8 * slot, fparity, p.err, p.wait_ns);  // the rows' values
        ok = ok && mbar_wait_warp(bar_s + 8 * b, sparity, p.err, p.wait_ns);
        if (!ok) break;
      }
      tc_fence_after();
      const uint32_t buf = tmem + lanes + b * 2 * kStep, bar = bar_p + 8 * b;
      const float4* vl = reinterpret_cast<const float4*>(smem + L::kRowVals + slot * 8 * kStep) + 4 * w;
      const int32_t b0 = b_lo + j * per_step;
      // columns [from, to) of this thread's 16 count
      const int from = kDQ ? 0 : lim - b0 * p.group - 16 * w, to = kDQ ? lim - b0 - 16 * w : 16;
      const bool whole = __all_sync(0xffffffffu, from <= 0 && to >= 16);
      float s[16], d[16];
      tmem_ld2(buf + 16 * w, s, buf + kStep + 16 * w, d);
      // Look for the next step's now: the answer arrives while these are worked on
      // (a wait costs this loop about 200 clocks even on a complete barrier).
      if (++b == kBufs) {
        b = 0;
        sparity ^= 1;
      }
      if (++slot == kSlots) {
        slot = 0;
        fparity ^= 1;
      }
      ready = mbar_test(bar_s + 8 * b, sparity);
      if (!kDQ) ready = ready && mbar_test(bar_full + 8 * slot, fparity);
      uint32_t wp[8], ws[8];
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        float4 l4 = make_float4(l, l, l, l), e4 = make_float4(e, e, e, e);
        if (!kDQ) {
          l4 = vl[i / 4];
          e4 = vl[kStep / 4 + i / 4];
          if (kShift != 0.f) l4 = make_float4(l4.x + kShift, l4.y + kShift, l4.z + kShift, l4.w + kShift);
        }
        const float2 x0 = fma2(make_float2(s[i], s[i + 1]), c2, make_float2(l4.x, l4.y));
        const float2 x1 = fma2(make_float2(s[i + 2], s[i + 3]), c2, make_float2(l4.z, l4.w));
        float2 p0 = make_float2(exp2_fast(x0.x), exp2_fast(x0.y)), p1 = make_float2(exp2_fast(x1.x), exp2_fast(x1.y));
        float2 d0 = add2(make_float2(d[i], d[i + 1]), make_float2(e4.x, e4.y));
        float2 d1 = add2(make_float2(d[i + 2], d[i + 3]), make_float2(e4.z, e4.w));
        if (!kBf16) {  // exact: a power of two
          d0 = mul2(d0, f2);
          d1 = mul2(d1, f2);
        }
        d0 = mul2(p0, d0);
        d1 = mul2(p1, d1);
        if (!whole) {
          auto keep = [&](int x, float v) { return i + x >= from && i + x < to ? v : 0.f; };
          p0 = make_float2(keep(0, p0.x), keep(1, p0.y));
          p1 = make_float2(keep(2, p1.x), keep(3, p1.y));
          d0 = make_float2(keep(0, d0.x), keep(1, d0.y));
          d1 = make_float2(keep(2, d1.x), keep(3, d1.y));
        }
        if (!kDQ) {
          wp[i / 2] = pack2<T>(p0.x, p0.y);
          wp[i / 2 + 1] = pack2<T>(p1.x, p1.y);
        }
        ws[i / 2] = pack2<T>(d0.x, d0.y);
        ws[i / 2 + 1] = pack2<T>(d1.x, d1.y);
      }
      // over this thread's own scores: the others' may not be read yet
      if (!kDQ) tmem_st(buf + 16 * w, wp);
      tmem_st(buf + kStep + 16 * w, ws);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
      __syncwarp();
    }
    // --------------------------------------------------------------- results
    if (ok && nsteps > 0) {
      ok = mbar_wait_warp(bar_o, 0, p.err, p.wait_ns);
      tc_fence_after();
    }
    const bool split = !kDQ && u.splits > 1;
    if (ok && (!split || nsteps > 0)) {  // (k_attn_bwd_join leaves out the splits without a step)
      // dQ: 32 columns each (64 channels: the first two groups); dK: groups 0
      // and 2, dV: 1 and 3, half of the columns each
      const int c_lo = kDQ ? 32 * w : half * (DP / 2), c_hi = kDQ ? (c_lo + 32 < DP ? c_lo + 32 : DP) : c_lo + DP / 2;
      const bool second = !kDQ && par == 1;
      const uint32_t acc = tmem + lanes + L::kAcc + (second ? DP : 0);
      const float mul = second ? exp2f(-kShift) : p.scale / factor;
      const int64_t out_row = kDQ ? static_cast<int64_t>(u.q.begin) + r0 + qi : static_cast<int64_t>(u.k.begin) + r0 + r;
      const int head = kDQ ? hk * p.group + r % p.group : hk;
      T* to = static_cast<T*>(second ? p.d2 : p.d1);
      const int64_t at = out_row * (second ? p.s2[0] : p.s1[0]) + head * (second ? p.s2[1] : p.s1[1]);
      // the resident tiles are no longer needed: every product is done
      uint8_t* stage = smem + L::kA + warp * 2048;
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
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] *= mul;
        if (split) {  // k_attn_bwd_join adds them up
          if (row) {
            float4* d = reinterpret_cast<float4*>(
                p.part + (((static_cast<int64_t>(u.split) * p.cut.m + out_row) * p.kv_heads + hk) * 2 + (second ? 1 : 0)) * p.dim + c0);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (c0 + 4 * i < p.dim) d[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
          __syncwarp();
          continue;
        }
        store_rows<T>(stage, o, to, row ? at : -1, c0, p.dim);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 16) tmem_dealloc(tmem, 512);
}

// The dK / dV blocks first, which take longer, then those of dQ (causal: from the
// tiles with the most keys down): one grid, so that neither waits for the other's
// last blocks.
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_bwd_tc(const __grid_constant__ BwdMaps kmaps, const __grid_constant__ BwdParams pk, uint32_t kunits,
                  const __grid_constant__ BwdMaps qmaps, const __grid_constant__ BwdParams pq) {
  if (blockIdx.x < kunits)
    gradients<T, DP, false>(kmaps, pk, blockIdx.x);
  else
    gradients<T, DP, true>(qmaps, pq, pq.causal ? gridDim.x - 1 - blockIdx.x : blockIdx.x - kunits);
}

// Adds up the splits of a tile's dK and dV, in order; kJoinParts blocks to a tile.
constexpr int kJoinParts = 8;

template <typename T>
__global__ void __launch_bounds__(256) k_attn_bwd_join(const BwdParams p, const Cut tiles) {
  __shared__ Unit s_unit;
  find_unit<256>(tiles, blockIdx.x, &s_unit, p.err);
  const Unit u = s_unit;
  grid_wait();
  if (u.item < 0) return;
  const int hk = blockIdx.y, r0 = u.tile * kRows, quads = p.dim / 4;
  const int rows = u.k.count - r0 < kRows ? u.k.count - r0 : kRows;
  if (u.q.count <= p.cut.chunk) return;  // one split, written as it is
  const int splits = (u.q.count - 1) / p.cut.chunk + 1;
  // splits without a step have written nothing: those before the first query
  // that sees a key of the tile
  int s0 = 0;
  if (p.causal) {
    const int64_t f = static_cast<int64_t>(r0) + u.q.count - u.k.count;
    if (f > 0) s0 = f >= u.q.count ? splits : static_cast<int>(f / p.cut.chunk);
  }
  const int64_t step = static_cast<int64_t>(p.cut.m) * p.kv_heads * 2 * p.dim;
  constexpr int kPer = kRows / kJoinParts;  // rows of this block
  const int i0 = blockIdx.z * kPer * 2 * quads, i1 = i0 + kPer * 2 * quads;
  for (int i = i0 + threadIdx.x; i < i1 && i < rows * 2 * quads; i += 256) {
    const int r = i / (2 * quads), rest = i - r * 2 * quads, second = rest / quads, c = (rest - second * quads) * 4;
    const int64_t row = static_cast<int64_t>(u.k.begin) + r0 + r;
    const float* from = p.part + ((row * p.kv_heads + hk) * 2 + second) * p.dim + c;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = s0; s < splits; ++s) {
      const float4 v = *reinterpret_cast<const float4*>(from + s * step);
      t.x += v.x, t.y += v.y, t.z += v.z, t.w += v.w;
    }
    T* to = static_cast<T*>(second ? p.d2 : p.d1) + row * (second ? p.s2[0] : p.s1[0]) + hk * (second ? p.s2[1] : p.s1[1]) + c;
    *reinterpret_cast<uint2*>(to) = make_uint2(pack2<T>(t.x, t.y), pack2<T>(t.z, t.w));
  }
}

// delta[row, head] = -sum of dO * O, and lse2 = -lse log2e, or -infinity for a
// row that saw no key, whose P = exp2(S + lse2) is then 0; fp16: also what bounds dS,
// (|dO|^2, |delta|) and |V|^2 of the rows that belong to items, by head, so that a
// block reads its rows' as runs.  LPR lanes hold a row of up to 8 LPR channels.  Bound
// by HBM: one read of O and dO (and V).
template <typename T, int LPR>
__global__ void __launch_bounds__(256) k_attn_delta_tc(const AttnArgs a, float* lse2, float2* qbound, float* vbound) {
  using C = Chunk<T, 8>;
  allow_next();
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
    if (qbound) q = group_sum<LPR>(q);
    if (there && l == 0) {
      a.delta[i] = -s;
      lse2[i] = a.lse[i] == -INFINITY ? -INFINITY : a.lse[i] * -kLog2e;
      if (qbound) qbound[(i - row * a.heads) * a.n + row] = make_float2(q, fabsf(s));
    }
  }
  if (!qbound) return;
  bounds(a.k_off, a.items, a.m, lo, hi);
  const T* V = static_cast<const T*>(a.v);
  for (int64_t b = lo * a.kv_heads + first; b < hi * a.kv_heads; b += stride) {
    const int64_t i = b + threadIdx.x / LPR, row = i / a.kv_heads;
    const bool there = i < hi * a.kv_heads;
    float q = 0.f;
    if (there && in) {
      float v[8];
      unpack(*reinterpret_cast<const C*>(V + row * a.v_stride[0] + (i - row * a.kv_heads) * a.v_stride[1] + 8 * l), v);
#pragma unroll
      for (int x = 0; x < 8; ++x) q += v[x] * v[x];
    }
    q = group_sum<LPR>(q);
    if (there && l == 0) vbound[(i - row * a.kv_heads) * a.m + row] = q;
  }
}

// Where the tiles of keys do not fill the machine (shared heads: the heads of a
// group are rows of one tile; causal: the first keys have all the work), the
// queries in runs, for one CTA to an SM, or one and a half where the mask leaves
// them unequal, each of at least 1024 packed rows.  (One, one and a half, two and
// a half CTAs: 6,000 rows, 2 heads of 128 over 1, took 156, 191, 199 us; 6,007
// causal rows, 8 heads of 128 over 2, 318, 287, 287 us.  Runs of 512 rows: 700 rows,
// 4 heads of 64, 31 us, whole 25 us.)
struct BwdPlan {
  int64_t units;
  int chunk;  // queries of a run, 0: all
};

BwdPlan bwd_plan(const AttnArgs& a, int sms) {
  const int group = a.heads / a.kv_heads;
  const int64_t tiles = a.m / kRows + a.items, blocks = tiles * a.kv_heads;
  BwdPlan b = {tiles, 0};
  const int64_t runs = ((a.causal ? 3ll * sms / 2 : sms) + blocks - 1) / blocks;
  int64_t chunk = a.n / runs;
  if (chunk < 1024 / group) chunk = 1024 / group;
  if (runs < 2 || a.n <= chunk) return b;
  b.chunk = static_cast<int>(chunk);
  b.units = tiles + (a.m / kRows + 1) * (a.n / chunk);
  return b;
}

template <typename T, int DP>
cudaError_t launch_typed(const AttnArgs& a, BwdParams p, const BwdMaps* maps, int sms, const BwdScratch& x, cudaStream_t st) {
  const BwdPlan plan = bwd_plan(a, sms);
  const int64_t rows = a.n * a.heads, per = DP == 64 ? 32 : 16;
  int64_t blocks = (rows + per - 1) / per;
  blocks = blocks < 8ll * sms ? (blocks < 1 ? 1 : blocks) : 8ll * sms;
  k_attn_delta_tc<T, DP / 8><<<static_cast<unsigned>(blocks), 256, 0, st>>>(a, x.lse2, x.qbound, x.vbound);
  constexpr uint32_t kSmemQ = BwdLayout<DP, true>::kTotal, kSmemK = BwdLayout<DP, false>::kTotal;
  constexpr int kSmem = static_cast<int>(kSmemQ > kSmemK ? kSmemQ : kSmemK);
  auto kern = k_attn_bwd_tc<T, DP>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  BwdParams k = p;
  auto resident = [](BwdParams& t, const void* x, const int64_t xs[2], const void* y, const int64_t ys[2]) {
    t.a1 = x;
    t.a2 = y;
    for (int i = 0; i < 2; ++i) {
      t.a1s[i] = xs[i];
      t.a2s[i] = ys[i];
    }
  };
  resident(p, a.q, a.q_stride, a.dout, a.dout_stride);
  p.d1 = a.dq;
  for (int i = 0; i < 2; ++i) p.s1[i] = a.dq_stride[i];
  resident(k, a.k, a.k_stride, a.v, a.v_stride);
  k.cut.per_tile = divisor(kRows);
  k.cut.by_keys = true;
  k.cut.chunk = plan.chunk;
  k.part = plan.chunk ? x.part : nullptr;
  k.d1 = a.dk;
  k.d2 = a.dv;
  for (int i = 0; i < 2; ++i) {
    k.s1[i] = a.dk_stride[i];
    k.s2[i] = a.dv_stride[i];
  }
  const int64_t qunits = a.n / p.qpt + a.items;
  e = launch_after(kern, dim3(static_cast<unsigned>(plan.units + qunits), a.kv_heads), kThreads, kSmem, st, maps[1], k,
                   static_cast<uint32_t>(plan.units), maps[0], p);
  if (e != cudaSuccess) return e;
  if (plan.chunk) {
    Cut tiles = k.cut;
    tiles.chunk = 0;
    e = launch_after(k_attn_bwd_join<T>, dim3(static_cast<unsigned>(a.m / kRows + a.items), a.kv_heads, kJoinParts), 256, 0,
                     st, k, tiles);
    if (e != cudaSuccess) return e;
  }
  count_launches(plan.chunk ? 3 : 2);
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

int64_t attn_bwd_tc_scratch(const AttnArgs& a, int sms) {
  const BwdPlan b = bwd_plan(a, sms);
  return b.chunk ? ((a.n - 1) / b.chunk + 1) * a.m * a.kv_heads * 2 * a.dim : 0;
}

cudaError_t launch_attn_bwd_tc(const AttnArgs& a, const BwdScratch& x, int sms, cudaStream_t st) {
  const int group = a.heads / a.kv_heads;
  BwdParams p = {};
  p.qpt = kRows / group;
  p.qps = kStep / group;
  BwdMaps maps[2] = {};  // dQ; dK and dV
  auto queries = [&](CUtensorMap* m, const void* t, const int64_t s[2], int per) {
    return make_map(m, t, a.dtype, a.n, a.heads, a.dim, s, group, per);
  };
  auto keys = [&](CUtensorMap* m, const void* t, const int64_t s[2], int per) {
    return make_map(m, t, a.dtype, a.m, a.kv_heads, a.dim, s, 1, per);
  };
  bool ok = keys(&maps[0].b1, a.k, a.k_stride, kStep) && keys(&maps[0].b2, a.v, a.v_stride, kStep) &&
            queries(&maps[1].b1, a.q, a.q_stride, p.qps) && queries(&maps[1].b2, a.dout, a.dout_stride, p.qps);
  if (ok && !BwdLayout<128, false>::kTmemA && a.dim > 64)
    ok = keys(&maps[1].a1, a.k, a.k_stride, kRows) && keys(&maps[1].a2, a.v, a.v_stride, kRows);
  if (!ok) return cudaErrorInvalidValue;
  p.cut = {a.q_off, a.k_off, static_cast<int32_t>(a.n), static_cast<int32_t>(a.m), a.items, 0, divisor(p.qpt), false};
  p.heads = a.heads;
  p.kv_heads = a.kv_heads;
  p.dim = a.dim;
  p.group = group;
  p.scale = a.scale;
  p.causal = a.causal;
  p.lse = x.lse2;
  p.delta = a.delta;
  p.qbound = x.qbound;
  p.vbound = x.vbound;
  p.err = a.err;
  // never below 100 ms, so that no CTA leaves with its loads in flight
  p.wait_ns = scan_wait_limit_ns() > 100000000ull ? scan_wait_limit_ns() : 100000000ull;
  if (a.dtype == kBF16)
    return a.dim <= 64 ? launch_typed<__nv_bfloat16, 64>(a, p, maps, sms, x, st)
                       : launch_typed<__nv_bfloat16, 128>(a, p, maps, sms, x, st);
  return a.dim <= 64 ? launch_typed<__half, 64>(a, p, maps, sms, x, st)
                     : launch_typed<__half, 128>(a, p, maps, sms, x, st);
}

}  // namespace smc
