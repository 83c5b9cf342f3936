// Attention within each item on the tensor cores (bf16 / fp16, sm_100a).
//
//   S = scale Q K^T,  P = exp2(S log2e - top),  O = sum P V / sum P
//
// One CTA holds kTiles (1 or 2) tiles of 128 packed rows (row = query * G +
// head of the group, so the heads that share keys share the tile) of one
// key/value head against a run of the item's keys, 128 (or 64) at a time.  Its
// warps:
//   softmax    four for each tile and, with two tiles of up to 64 channels, for
//              each half of a step's columns: one thread per row, its scores in
//              registers, running maximum and sum in fp32, P rounded to the input
//              type into the TMEM columns its scores came from;
//   MMA        one for each tile: S = Q K^T (both from shared memory), then
//              O += P V with P in TMEM and V read MN-major as it lies;
//   TMA        the Q tiles once, then K and V tiles into a ring.
// Each tile's half is a chain of its own, S -> softmax -> product -> next S,
// with its own maxima, sums and accumulator (TMEM has the room), so a row's two
// threads meet only at the end, and while one chain waits for the tensor cores
// the others keep the special-function unit busy (up to 64 channels an SM runs
// four chains: two tiles with two halves, or four one-tile CTAs).
// An accumulator is rescaled in TMEM only when a row's maximum has grown by
// more than 2^8; the sums use the unrounded P.  In fp16 P carries 2^7 besides: it
// stays below 2^15, and a key counts down to 2^-32 of its row's largest (without, down
// to 2^-25: 40,000 equal keys 17.5 below one other were lost, 1e-3 of the output).  A
// P below 2^-21 of the largest is rounded in steps of 2^-31 of it.  Keys behind the item's end are masked, and V rows there are
// zeroed in shared memory, since P = 0 does not undo a NaN.
// With few queries over many keys the keys are split between CTAs; each writes
// its unnormalised fp32 O, maximum and sum, and k_attn_join adds them up in
// order.
//
// What bounds it: at 64 channels the exponentials (16 a clock and SM: 0.71 ms of
// the first figure), not the products (0.50 ms); a chain's own latency for the rest.
// Measured: 20,011 rows, 8 heads of 64, bf16: 1.09 ms, 750 TFLOP/s, 8 heads of 128:
// 1.62 to 1.74 ms, 940 to 1010 TFLOP/s (causal 0.90 to 0.96 ms); 512 items of 1 to
// 512 rows, fp16: 0.26 ms; 8 single queries over 1,000 to 32,768 keys, 16 heads of
// 128 over 4: 53 us, 4.5 TB/s.  Registers are short: at 128 channels a thread spills
// 68 bytes (one tile 44) and reads 148 (108) of them again, at 64 channels 20 (36) and
// 24 (56).
#include <type_traits>

#include "attn_join.cuh"
#include "attn_tc.cuh"

namespace smc {

namespace {

using namespace attn;

constexpr int kShortItem = 512;  // packed rows

struct FwdParams {
  Cut cut;                                // per_tile: queries of a CTA; chunk: keys of a split
  int heads, kv_heads, dim, group, qpt;   // qpt: queries of a tile
  float c;                                       // scale * log2 e
  bool causal;
  void* out;
  float* lse;
  float *part_o, *part_ml;  // of splits: [splits, n, heads, dim] and [.., 2], or null
  uint32_t* err;
  uint64_t wait_ns;
};

// Two tiles: one CTA to an SM.  One tile: CTAs share an SM, two of up to 128
// channels, or four of up to 64 with steps of 64 keys.
template <int DP, int kTiles> struct FwdLayout {
  static constexpr bool kSmall = kTiles == 1 && DP == 64;
  static constexpr int kKeys = kSmall ? 64 : 128;  // keys of a step
  static constexpr int kBlocks = kTiles == 2 ? 1 : kSmall ? 4 : 2;
  static constexpr uint32_t kQBytes = DP / 64 * kPanel;                                   // a tile of Q
  static constexpr uint32_t kKvPanel = kKeys * 128, kKvBytes = DP / 64 * kKvPanel;        // a step of K or V
  static constexpr int kSlots = kTiles == 2 ? (DP == 64 ? 8 : 4) : kSmall ? 4 : 2;
  static constexpr int kHalves = kTiles == 2 && DP == 64 ? 2 : 1, kGroups = kTiles * kHalves;
  static constexpr int kThreads = 128 * kGroups + 32 * (kTiles + 1);
  static constexpr uint32_t kQ = 0, kKv = kTiles * kQBytes, kBar = kKv + kSlots * kKvBytes;
  // barriers: q, kv full[kSlots], kv empty[kSlots], s full[kGroups], p ready[kGroups], o done[kTiles], tail, q free
  static constexpr uint32_t kMisc = kBar + 8 * (2 * kSlots + kTiles + 2 * kGroups + 3);
  static constexpr uint32_t kMl = (kMisc + 16 + 15) / 16 * 16;  // (maximum, sum) of each row and half
  static constexpr uint32_t kTotal = kMl + (kHalves == 2 ? kGroups * kRows * 8 : 0) + 1024;
  // TMEM columns: S of the tiles, then O of the tiles' halves
  static constexpr uint32_t kO = kTiles * kKeys, kColumns = 512 / kBlocks;
  static_assert(kO + kGroups * DP <= kColumns, "accumulators fit");
};

template <typename T, int DP, int kTiles>
__global__ void __launch_bounds__(FwdLayout<DP, kTiles>::kThreads, FwdLayout<DP, kTiles>::kBlocks)
    k_attn_fwd_tc(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const FwdParams p) {
  using L = FwdLayout<DP, kTiles>;
  constexpr int kSlots = L::kSlots, kPanels = DP / 64, kHalves = L::kHalves, kKeys = L::kKeys, kCols = kKeys / kHalves;
  constexpr int kMmaWarp = 4 * L::kGroups, kTmaWarp = kMmaWarp + kTiles;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr float kShift = kBf16 ? 0.f : 7.f;  // P carries 2^kShift: it cancels in O / sum and is part of top
  extern __shared__ uint8_t smem_raw[];
  __shared__ Unit s_unit;
  const uint32_t raw = smem_u32(smem_raw), sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  volatile uint32_t* s_misc = reinterpret_cast<volatile uint32_t*>(smem + L::kMisc);  // [0] tmem
  const uint32_t bar_q = sbase + L::kBar, bar_full = bar_q + 8, bar_empty = bar_full + 8 * kSlots;
  const uint32_t bar_s = bar_empty + 8 * kSlots, bar_p = bar_s + 8 * L::kGroups, bar_o = bar_p + 8 * L::kGroups;
  const uint32_t bar_tail = bar_o + 8 * kTiles, bar_qfree = bar_tail + 8;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    prefetch_tmap(&qmap);
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
    mbar_init(bar_q, 1);
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, kTiles);
    }
    for (int t = 0; t < kTiles; ++t) mbar_init(bar_o + 8 * t, 1);
    for (int g = 0; g < L::kGroups; ++g) {
      mbar_init(bar_s + 8 * g, 1);
      mbar_init(bar_p + 8 * g, 4);
    }
    mbar_init(bar_tail, 1);
    mbar_init(bar_qfree, kTiles);
    fence_mbarrier_init();
    fence_proxy_async_smem();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(&s_misc[0])), L::kColumns);
    tmem_relinquish();
  }
  tc_fence_before();
  // causal: the tiles with the most keys come last in an item and start first
  const int64_t ux = p.causal ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
  find_unit<L::kThreads>(p.cut, ux, &s_unit, p.err);
  tc_fence_after();
  const uint32_t tmem = s_misc[0];
  if (s_unit.item < 0) {
    if (warp == kMmaWarp) tmem_dealloc(tmem, L::kColumns);
    return;
  }
  const Unit u = s_unit;
  // this block's key/value heads: blockIdx.y, + gridDim.y, ...
  const int nheads = (p.kv_heads - 1 - static_cast<int>(blockIdx.y)) / static_cast<int>(gridDim.y) + 1;
  const int32_t q0 = u.tile * kTiles * p.qpt;
  const int32_t left = u.q.count - q0;
  const int32_t k_lo = u.split * p.cut.chunk;
  const int32_t k_hi = u.splits > 1 && u.k.count - k_lo > p.cut.chunk ? k_lo + p.cut.chunk : u.k.count;
  int queries[kTiles], steps[kTiles];
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    const int32_t rest = left - t * p.qpt;
    queries[t] = rest < 0 ? 0 : (rest < p.qpt ? rest : p.qpt);
    const int32_t seen = queries[t] > 0 ? keys_seen(u, q0 + t * p.qpt + queries[t] - 1, p.causal) : 0;
    const int32_t hi = seen < k_hi ? seen : k_hi;
    steps[t] = hi > k_lo ? (hi - k_lo + kKeys - 1) / kKeys : 0;
  }
  const int nsteps = kTiles == 2 && steps[kTiles - 1] > steps[0] ? steps[kTiles - 1] : steps[0];

  if (warp == kTmaWarp) {
    // ------------------------------------------------------------- TMA loads
    // 2 * nsteps tiles in the order they are used: K0 V0 K1 V1 ...
    int slot = 0;
    uint32_t parity = 1;
    bool ok = nsteps > 0;
    for (int i = 0; i < nheads && ok; ++i) {
      const int hk = blockIdx.y + i * gridDim.y;
      ok = mbar_wait_warp(bar_qfree, (i & 1) ^ 1, p.err, p.wait_ns);  // the head before has no scores left to do
      if (ok && elect_one()) {
        const int tiles = kTiles == 2 && queries[kTiles - 1] > 0 ? 2 : 1;
        mbar_arrive_expect_tx(bar_q, static_cast<uint32_t>(tiles * kPanels * p.group * p.qpt) * 128u);
        for (int t = 0; t < tiles; ++t)
          for (int c = 0; c < kPanels; ++c)
            tma_load_3d(sbase + L::kQ + t * L::kQBytes + c * kPanel, &qmap, bar_q, c * 64, hk * p.group,
                        u.q.begin + q0 + t * p.qpt);
      }
      __syncwarp();
      for (int j = 0; j < 2 * nsteps && ok; ++j) {
        ok = mbar_wait_warp(bar_empty + 8 * slot, parity, p.err, p.wait_ns);
        if (!ok) break;
        const int32_t key = k_lo + (j >> 1) * kKeys;
        const int rows = u.k.count - key;  // V rows behind the item's end are zeroed below
        const bool tail = (j & 1) && rows < kKeys;
        const uint32_t dst = sbase + L::kKv + slot * L::kKvBytes, bar = tail ? bar_tail : bar_full + 8 * slot;
        if (elect_one()) {
          mbar_arrive_expect_tx(bar, L::kKvBytes);
          for (int c = 0; c < kPanels; ++c)
            tma_load_3d(dst + c * L::kKvPanel, (j & 1) ? &vmap : &kmap, bar, c * 64, hk, u.k.begin + key);
        }
        __syncwarp();
        if (tail) {  // once for each head, at the last step
          ok = mbar_wait_warp(bar_tail, i & 1, p.err, p.wait_ns);
          if (!ok) break;
          uint4* base = reinterpret_cast<uint4*>(smem + L::kKv + slot * L::kKvBytes);
          for (int c = 0; c < kPanels; ++c)
            for (int z = rows * 8 + lane; z < kKeys * 8; z += 32) base[c * (L::kKvPanel / 16) + z] = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_full + 8 * slot);
          __syncwarp();
        }
        if (++slot == kSlots) {
          slot = 0;
          parity ^= 1;
        }
      }
    }
  } else if (warp >= kMmaWarp) {
    // ------------------------------------------------------------- MMA issue
    // A warp for each tile; one elected lane issues each batch, with the
    // descriptors advanced by additions only (computing them anew made each
    // MMA cost about 120 clocks of the warp's time).
    const int t = warp - kMmaWarp, mine = steps[t];
    const uint32_t ab = kBf16 ? 1u : 0u;
    const int ks = (p.dim + 15) / 16;
    const uint32_t idesc_s = idesc_f16(ab, kCols), idesc_o = idesc_f16(ab, static_cast<uint32_t>(ks * 16)) | kIdescBMn;
    constexpr uint64_t kTile = L::kKvBytes >> 4;
    const uint64_t q = kmajor_desc(sbase + L::kQ, 128) + t * (L::kQBytes >> 4), kd = kmajor_desc(sbase + L::kKv, 128);
    const uint64_t vd = mnmajor_desc(sbase + L::kKv, L::kKvPanel);
    auto wait = [&](uint32_t bar, uint32_t parity) {
      const bool w = mbar_wait_warp(bar, parity, p.err, p.wait_ns);
      tc_fence_after();
      return w;
    };
    auto scores = [&](int h, uint64_t k0) {  // in the elected lane
#pragma unroll
      for (int k = 0; k < DP / 16; ++k)
        if (k < ks)
          umma_f16(tmem + t * kKeys + h * kCols, q + (k >> 2) * (kPanel >> 4) + 2 * (k & 3),
                   k0 + h * (kCols * 8) + (k >> 2) * (L::kKvPanel >> 4) + 2 * (k & 3), idesc_s, k > 0);
      umma_commit(bar_s + 8 * (t * kHalves + h));
    };
    // A slot is free once every tile's warp has let go of it: behind the products
    // that read it, or at once where the tile has none.  Only slots that are
    // loaded again: no arrival is left under way at the end.
    auto release = [&](int slot, int index, bool read) {  // in the elected lane; index: of all this block's loads
      if (index + kSlots >= 2 * nsteps * nheads) return;
      if (read) umma_commit(bar_empty + 8 * slot);
      else mbar_arrive(bar_empty + 8 * slot);
    };
    // Slots and phases run on over the heads: the loads are one sequence K V K V.
    int sk = 0, sv = 1;
    uint32_t pk = 0, pv = 0, pp = 0;
    bool ok = nsteps > 0;
    auto next_k = [&]() {
      if ((sk += 2) >= kSlots) {
        sk -= kSlots;
        pk ^= 1;
      }
    };
    for (int i = 0; i < nheads && ok; ++i) {
      const int load0 = 2 * nsteps * i;
      // the first scores; with one step they are the last that read this Q
      ok = wait(bar_q, i & 1) && wait(bar_full + 8 * sk, pk);
      if (ok && elect_one()) {
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
          if (mine > 0) scores(h, kd + sk * kTile);
        release(sk, load0, mine > 0);
        if (nsteps == 1 && i + 1 < nheads) umma_commit(bar_qfree);
      }
      __syncwarp();
      next_k();
      for (int j = 0; j < nsteps && ok; ++j) {
        const uint64_t v0 = vd + sv * kTile, k0 = kd + sk * kTile;
        const bool last = j + 1 == mine, more = j + 1 < nsteps, qdone = j + 2 == nsteps && i + 1 < nheads;
        ok = wait(bar_full + 8 * sv, pv);
        // with two slots, K of the next step may still be on its way when P is ready
        constexpr bool kEarly = kSlots > 2;
        if (kEarly && ok && more) ok = wait(bar_full + 8 * sk, pk);
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
          const int g = t * kHalves + h;
          if (ok && j < mine) ok = wait(bar_p + 8 * g, pp);
          if (ok && elect_one()) {
            if (j < mine) {
#pragma unroll
              for (int k = 0; k < kCols / 16; ++k)
                umma_f16_ts(tmem + L::kO + g * DP, tmem + t * kKeys + h * kCols + k * 8, v0 + 128 * (h * kCols / 16 + k),
                            idesc_o, j > 0 || k > 0);
            }
            if (kEarly && j + 1 < mine) scores(h, k0);
            if (h + 1 == kHalves) {
              if (last) umma_commit(bar_o + 8 * t);
              release(sv, load0 + 2 * j + 1, j < mine);
              if (kEarly && more) release(sk, load0 + 2 * j + 2, j + 1 < mine);
              if (kEarly && qdone) umma_commit(bar_qfree);
            }
          }
          __syncwarp();
        }
        if (j < mine) pp ^= 1;
        if (!kEarly && ok && more) {
          ok = wait(bar_full + 8 * sk, pk);
          if (ok && elect_one()) {
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
              if (j + 1 < mine) scores(h, k0);
            release(sk, load0 + 2 * j + 2, j + 1 < mine);
            if (qdone) umma_commit(bar_qfree);
          }
          __syncwarp();
        }
        if ((sv += 2) >= kSlots) {
          sv -= kSlots;
          pv ^= 1;
        }
        if (more) next_k();
      }
    }
  } else {
    // --------------------------------------------------------------- softmax
    const int g = warp >> 2, t = g / kHalves, h = g % kHalves, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + t * kKeys + h * kCols, to = tmem + lanes + L::kO + g * DP;
    const int32_t qi = r / p.group;  // query in the tile
    const bool row = qi < queries[t];
    const bool used = __any_sync(0xffffffffu, row);  // a warp without rows only keeps step
    int32_t lim = row ? keys_seen(u, q0 + t * p.qpt + qi, p.causal) : 0;  // keys [0, lim) are seen
    lim = (lim < k_hi ? lim : k_hi) - k_lo - h * kCols;
    bool ok = true;
    uint32_t ps = 0;
    for (int head = 0; head < nheads && ok; ++head) {
      const int hk = blockIdx.y + head * gridDim.y;
      // top: the exponent that the sums refer to, a row's rounded largest score times c, less kShift
      float top = -INFINITY, sum = 0.f;
      for (int j = 0; j < steps[t]; ++j) {
        ok = mbar_wait_warp(bar_s + 8 * g, ps, p.err, p.wait_ns);
        ps ^= 1;
        if (!ok) break;
        tc_fence_after();
        if (used) {
          // The scores in registers: all of this thread's, or (four CTAs to an SM)
          // 32 at a time, read from TMEM twice.
          constexpr int kPart = L::kSmall ? 32 : kCols, kParts = kCols / kPart;
          const int32_t seen = lim - j * kKeys;
          const bool whole = __all_sync(0xffffffffu, seen >= kCols);
          float x[kPart];
          float m0 = -INFINITY, m1 = m0, m2 = m0, m3 = m0;
          auto load = [&](int q) {
            tmem_ld(ts + q * kPart, x);
            if (!whole) {
#pragma unroll
              for (int i = 0; i < kPart; ++i)
                if (q * kPart + i >= seen) x[i] = -INFINITY;
            }
          };
#pragma unroll
          for (int q = 0; q < kParts; ++q) {
            load(q);
#pragma unroll
            for (int i = 0; i < kPart; i += 8) {
              m0 = max3(m0, x[i], x[i + 1]);
              m1 = max3(m1, x[i + 2], x[i + 3]);
              m2 = max3(m2, x[i + 4], x[i + 5]);
              m3 = max3(m3, x[i + 6], x[i + 7]);
            }
          }
          const float m = __fmul_rn(fmaxf(max3(m0, m1, m2), m3), p.c);
          const bool grown = m > top + (8.f + kShift) || (top == -INFINITY && m > -INFINITY);
          if (__any_sync(0xffffffffu, grown)) {
            const float next = m - kShift, keep = grown ? exp2_fast(top - next) : 1.f;
            if (grown) {
              sum *= keep;
              top = next;
            }
            if (j > 0) {  // the products so far are complete: these scores came after them
#pragma unroll 1
              for (int c0 = 0; c0 < DP; c0 += 16) {
                float o[16];
                uint32_t b[16];
                tmem_ld(to + c0, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) b[i] = __float_as_uint(o[i] * keep);
                tmem_st(to + c0, b);
              }
            }
          }
          const float base = top == -INFINITY ? 0.f : top;
          float2 sa = make_float2(0.f, 0.f), sb = sa;
          const float2 c2 = make_float2(p.c, p.c), b2 = make_float2(-base, -base);
#pragma unroll
          for (int q = 0; q < kParts; ++q) {
            if (kParts > 1) load(q);
            constexpr int kWords = kPart >= 64 ? 32 : 16;
#pragma unroll
            for (int z = 0; z < kPart / (2 * kWords); ++z) {
              uint32_t w[kWords];
#pragma unroll
              for (int i = 0; i < kWords; i += 2) {
                const int e = z * 2 * kWords + 2 * i;
                const float2 y0 = fma2(make_float2(x[e], x[e + 1]), c2, b2), y1 = fma2(make_float2(x[e + 2], x[e + 3]), c2, b2);
                const float2 e0 = make_float2(exp2_fast(y0.x), exp2_fast(y0.y)), e1 = make_float2(exp2_fast(y1.x), exp2_fast(y1.y));
                sa = add2(sa, e0);
                sb = add2(sb, e1);
                w[i] = pack2<T>(e0.x, e0.y);
                w[i + 1] = pack2<T>(e1.x, e1.y);
              }
              // over scores that are in registers, or used up
              tmem_st(ts + (q * kPart / 2 + z * kWords), w);
            }
          }
          sum += (sa.x + sa.y) + (sb.x + sb.y);
          tmem_st_wait();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_p + 8 * g);
        __syncwarp();
      }
      // --------------------------------------------------------------- results
      float2* s_ml = reinterpret_cast<float2*>(smem + L::kMl);
      float weight = 1.f, weight2 = 0.f;  // of this half's accumulator, and the other's
      if (kHalves == 2) {
        s_ml[g * kRows + r] = make_float2(top, sum);
        asm volatile("bar.sync %0, 256;" ::"r"(1 + t) : "memory");  // the tile's two groups
        const float2 other = s_ml[(g ^ 1) * kRows + r];
        const float m = fmaxf(top, other.x);
        weight = top == -INFINITY ? 0.f : exp2_fast(top - m);
        weight2 = other.x == -INFINITY ? 0.f : exp2_fast(other.x - m);
        sum = sum * weight + other.y * weight2;
        top = m;
      }
      if (ok && steps[t] > 0) {
        ok = mbar_wait_warp(bar_o + 8 * t, head & 1, p.err, p.wait_ns);
        tc_fence_after();
      }
      if (ok && used) {
        const int64_t at = static_cast<int64_t>(u.q.begin + q0 + t * p.qpt + qi) * p.heads + hk * p.group + r % p.group;
        const bool split = u.splits > 1;
        const int64_t slot = static_cast<int64_t>(u.split) * p.cut.n * p.heads + at;
        const float inv = sum == 0.f ? 0.f : 1.f / sum, f1 = split ? weight : weight * inv, f2 = split ? weight2 : weight2 * inv;
        const uint32_t to2 = tmem + lanes + L::kO + (g ^ 1) * DP;
#pragma unroll 1
        for (int c0 = h * (DP / kHalves); c0 < (h + 1) * (DP / kHalves); c0 += 32) {
          if (c0 >= p.dim) break;
          float o[32];
          if (steps[t] > 0) {
            tmem_ld(to + c0, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= f1;
            if (kHalves == 2) {
              float o2[32];
              tmem_ld(to2 + c0, o2);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = fmaf(o2[i], f2, o[i]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0.f;
          }
          if (row && split) {
            float4* d = reinterpret_cast<float4*>(p.part_o + slot * p.dim + c0);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (c0 + 4 * i < p.dim) d[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          } else if (row) {
            uint4* d = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + at * p.dim + c0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (c0 + 8 * i < p.dim)
                d[i] = make_uint4(pack2<T>(o[8 * i], o[8 * i + 1]), pack2<T>(o[8 * i + 2], o[8 * i + 3]),
                                  pack2<T>(o[8 * i + 4], o[8 * i + 5]), pack2<T>(o[8 * i + 6], o[8 * i + 7]));
          }
          __syncwarp();
        }
        if (row && h == 0) {
          if (split) *reinterpret_cast<float2*>(p.part_ml + 2 * slot) = make_float2(top, sum);
          else if (p.lse) p.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
        }
        __syncwarp();
        tc_fence_before();  // the next head's products may overwrite O once P of its first step is there
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, L::kColumns);
}

struct FwdPlan {
  int tiles;      // tiles of a CTA
  int64_t units;  // blocks along x
  int chunk;      // keys of a split, 0: all
  int heads;      // key/value heads of a CTA
};

// One tile to a CTA where items are short on average: such a CTA's start and
// end are most of its life, and the others on its SM fill them.  (51,200 rows in
// items of 256, 512, 1024, 2048, 5000 rows, 8 heads, one tile / two: of 64 channels
// 76 / 145, 103 / 160, 175 / 210, 304 / 324, 713 / 690 us, of 128 channels 127 / 192,
// 165 / 228, 255 / 317, 453 / 491, 1095 / 1049 us: the border could lie at 2048 rows.
// The average misjudges one item of 8000 rows beside 1000 of one row: 551 / 557 and
// 884 / 720 us.)
FwdPlan fwd_plan(const AttnArgs& a, int sms) {
  const int group = a.heads / a.kv_heads, qpt = kRows / group;
  FwdPlan s = {};
  s.tiles = a.n <= a.items * static_cast<int64_t>(kShortItem / kRows * qpt) ? 1 : 2;
  const int blocks = s.tiles == 2 ? 1 : a.dim <= 64 ? FwdLayout<64, 1>::kBlocks : FwdLayout<128, 1>::kBlocks;
  const int per = s.tiles * qpt;
  const int64_t tiles = a.n / per + a.items, slots = static_cast<int64_t>(sms) * blocks;
  s.units = tiles;
  // Short items: several heads to a CTA, as long as three waves of CTAs remain,
  // since finding the block's share and the first loads' way are a third of a
  // CTA's life there.  (Two, three, four, eight waves: 512 items of 1 to 512 rows, 8
  // heads of 64: 275, 259, 260, 274 us; 1000 of 1 to 216, 8 of 32: 167, 166, 175, 189.)  (Two-tile CTAs read each other's halves at the end, and
  // their items are long.)
  s.heads = 1;
  if (s.tiles == 1) {
    const int64_t most = tiles * a.kv_heads / (3 * slots);
    s.heads = static_cast<int>(most < 1 ? 1 : most < a.kv_heads ? most : a.kv_heads);
  }
  // The join and its scratch cost 8 us of the device: one query of 8 heads of 64
  // took 21 us split and 14, 21, 27 us whole over 300, 600, 1000 keys, 300 queries
  // 25 to 29 us split and 17, 18, 25, 30 us whole over 300, 600, 1000, 1500 keys.
  // All in one wave: 8 queries over 8 contexts of 116,166 keys in all, a grid of 308
  // on 296 slots, took 61 us, within the slots 53 us.
  s.chunk = split_keys(a, per, slots, 1024, true);
  if (s.chunk) s.units += (a.n / per + 1) * (a.m / s.chunk);
  return s;
}

template <typename T, int DP, int kTiles>
cudaError_t launch_tiles(const AttnArgs& a, const FwdParams& p, const FwdPlan& s, const CUtensorMap* maps,
                         cudaStream_t st) {
  using L = FwdLayout<DP, kTiles>;
  auto kern = k_attn_fwd_tc<T, DP, kTiles>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(L::kTotal));
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(s.units), static_cast<unsigned>((a.kv_heads + s.heads - 1) / s.heads));
  kern<<<grid, L::kThreads, L::kTotal, st>>>(maps[0], maps[1], maps[2], p);
  count_launches(s.chunk ? 2 : 1);
  e = cudaGetLastError();
  return s.chunk && e == cudaSuccess ? launch_join<T>(a, p.cut, p.part_o, p.part_ml, st) : e;
}

template <typename T>
cudaError_t launch_fwd(const AttnArgs& a, const FwdParams& p, const FwdPlan& s, const CUtensorMap* maps,
                       cudaStream_t st) {
  if (a.dim <= 64) return s.tiles == 1 ? launch_tiles<T, 64, 1>(a, p, s, maps, st) : launch_tiles<T, 64, 2>(a, p, s, maps, st);
  return s.tiles == 1 ? launch_tiles<T, 128, 1>(a, p, s, maps, st) : launch_tiles<T, 128, 2>(a, p, s, maps, st);
}

}  // namespace

bool attn_tc_supported(const AttnArgs& a) {
  return a.dtype != kF32 && a.dim % 8 == 0 && a.m > 0 && map_fits(a.q, a.q_stride) && map_fits(a.k, a.k_stride) &&
         map_fits(a.v, a.v_stride) && (reinterpret_cast<uintptr_t>(a.out_w) & 15u) == 0 && encode_fn() != nullptr;
}

int64_t attn_tc_scratch(const AttnArgs& a, int sms) {
  const FwdPlan s = fwd_plan(a, sms);
  return split_words(a, s.chunk) * static_cast<int64_t>(sizeof(float));
}

cudaError_t launch_attn_tc(const AttnArgs& a, void* scratch, int sms, cudaStream_t st) {
  const int group = a.heads / a.kv_heads, qpt = kRows / group;
  const FwdPlan s = fwd_plan(a, sms);
  const int keys = s.tiles == 1 && a.dim <= 64 ? FwdLayout<64, 1>::kKeys : kRows;
  CUtensorMap maps[3];
  if (!make_map(&maps[0], a.q, a.dtype, a.n, a.heads, a.dim, a.q_stride, group, qpt) ||
      !make_map(&maps[1], a.k, a.dtype, a.m, a.kv_heads, a.dim, a.k_stride, 1, keys) ||
      !make_map(&maps[2], a.v, a.dtype, a.m, a.kv_heads, a.dim, a.v_stride, 1, keys))
    return cudaErrorInvalidValue;
  FwdParams p = {};
  p.cut = {a.q_off, a.k_off, static_cast<int32_t>(a.n), static_cast<int32_t>(a.m), a.items, s.chunk,
           divisor(s.tiles * qpt), false};
  p.heads = a.heads;
  p.kv_heads = a.kv_heads;
  p.dim = a.dim;
  p.group = group;
  p.qpt = qpt;
  p.c = a.scale * kLog2e;
  p.causal = a.causal;
  p.out = a.out_w;
  p.lse = a.lse_w;
  if (s.chunk) {
    p.part_o = static_cast<float*>(scratch);
    p.part_ml = p.part_o + ((a.m - 1) / s.chunk + 1) * a.n * a.heads * a.dim;
  }
  p.err = a.err;
  // never below 100 ms, so that no CTA leaves with its loads in flight
  p.wait_ns = scan_wait_limit_ns() > 100000000ull ? scan_wait_limit_ns() : 100000000ull;
  return a.dtype == kBF16 ? launch_fwd<__nv_bfloat16>(a, p, s, maps, st) : launch_fwd<__half>(a, p, s, maps, st);
}

}  // namespace smc
