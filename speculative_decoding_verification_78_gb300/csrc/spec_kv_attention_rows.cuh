// spec_kv_attention_rows.cuh -- attention of many query rows (more than 32 for a key head: candidate
// trees, pieces of prompts, chains with many query heads) over the paged e4m3 cache, on the
// 5th-generation tensor cores.
//
// The same mathematics as the kernel for few rows: with y = scale log2(e) ks (q . kb) + log2 vs and a
// reference m, weights p = 2^(y - m) multiply the e4m3 bytes vb and p / vs adds to the denominator.
//
// Here the query rows lie along the MMA's 128 rows and the tokens along its columns: S = Q K^T (Q as
// 2 or 3 e4m3 terms, K's bytes as TMA lands them), O = P V. A softmax thread owns a query row, so
// its reference, its sum and its query's unit are registers; what differs by token, the page scales,
// is constant over 16 columns (pages hold at least 16 tokens). P is written back to tensor memory,
// over the scores it came from, as the fp16 operand of the second MMA: nothing of the softmax passes
// through shared memory, which the operands of the MMAs already load. V is widened to fp16 by four
// warps of their own, once for all rows of the CTA.
//
// Two groups of eight softmax warps (two for each 32 rows, half of the tile's tokens each) work half a
// step apart, so that the tensor cores have one group's MMAs while the other group exponentiates: with
// more than 128 rows each group has 128 rows of its own and both take every tile; with fewer, the groups
// take the tiles in turn and are joined at the end of the item. Unit u of a segment belongs to group
// u & 1; values(u) and then scores(u + 2) are issued as soon as its weights are there.
//
// What bounds it (D = 128, measured with clock counters): a 256-row tile of 128 tokens costs 2100 clocks
// of MMA (two e4m3 terms cost what one 16-bit operand would: 2048 at the nominal rate; the operands of
// both MMAs, V's widening and the copies want about 2400 clocks of shared-memory bandwidth) and 1380 of
// weights (345 clocks a warp for 64 scores of 32 rows: ex2 256 of them). A group's turn is longer than
// either, about 3500: its weights (1340, the other group's beside them), the store, a hand-over to the
// MMA warp, its MMAs (1050) behind the other group's, a hand-over back; an item's start and end cost
// another 20000. 32 trees of 64 nodes, four query heads a key head, 8192 tokens: 234 us with the join,
// 1100 TFLOP/s (233 in the form these clocks were taken of, see the registers below); with a window of 2048 and 64
// sinks 100 us, 710 TFLOP/s, two items of 17 tiles a CTA; at the steps before
// it with full rows per thread 367 us, with one MMA warp waiting for each hand-over in turn
// 294 us, with spills in the epilogue 251, with the MMA warp asking for the keys after the weights and
// issuing values and scores apart 244. No one part bounds it: dropping the second e4m3 term, half of the
// value MMAs or the widening (wrong results, for timing only) gained 3 to 10 % each.
// Tried and not kept (us against what was there then): three stages of K and V for 256 rows (265 for 262),
// scores and values issued by two warps (294 for 262), the next item's queries posted before the
// accumulators are read (262 for 250), tiles widened by two lots of four warps (267 for 262), all 64
// scores of a thread loaded at once (276 for 262) or 32 (263 for 245), the next item's queries asked for
// in L2 some tiles ahead (253 for 251), results turned round in shared memory to store whole lines (no
// change), with up to 64 rows the second group on the warps of the other 64 lanes (149 for 155 at best,
// before what joining its accumulators would cost).
#pragma once

#include "spec_kv_attn.h"

namespace specv {

using namespace attn;

namespace {

constexpr int kGroupWarps = 8;                        // two for each 32 rows: half of the tokens each
constexpr int kSoftWarps = 2 * kGroupWarps;
constexpr int kSoftThreads = 32 * kSoftWarps;
constexpr int kWidenWarp = kSoftWarps, kWidenWarps = 4;   // warps that widen V
constexpr int kWidenThreads = 32 * kWidenWarps;
constexpr int kCopyK = kWidenWarp + kWidenWarps, kMma = kCopyK + 1, kCopyV = kCopyK + 2,
              kConsts = kCopyK + 3;
// 24 warps of 80 registers, all that an SM has. Moving registers from the other roles to the softmax warps
// (setmaxnreg) is not open to them: the copying, constants and MMA warps make up one warpgroup, whose four
// warps have to execute the same instruction, and with one instruction before their branches the compiler
// spills 460 bytes for 50. In a graph, us (64 chains of 6 / 32 trees / the same over 8192 tokens / two
// prompts): 49 / 165 / 240 / 246; eight widening warps, 72 registers a thread: 52 / 167 / 249 / 255; those
// with an instruction in each role's branch, which is undefined: 48 / 152 / 233 / 237.
constexpr int kRowsThreads = 32 * (kConsts + 1);
constexpr int kEdge = 1 << 31;      // (with a window) beside a page's first slot: the tile needs masks
constexpr float kBias = 8.f;        // a new reference puts the row's largest weight at 2^8 ...
constexpr float kTrigger = 15.f;    // ... and is taken when one exceeds 2^15 (fp16 ends at 2^16)

__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc));
}
// barrier of the two warps that share rows: true in both if `p` was in any of their threads
__device__ __forceinline__ bool pair_any(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(p)), "r"(id)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void rows_sync() {   // the softmax threads
  asm volatile("bar.sync 1, %0;" ::"n"(kSoftThreads) : "memory");
}
__device__ __forceinline__ void widen_sync() {
  asm volatile("bar.sync 2, %0;" ::"n"(kWidenThreads) : "memory");
}

// RTC: row tiles of 128 a CTA works on at once; S: stages of K and V; kWin: with a window
template <typename T_, int D_, int RTC_, int S_, bool kWin_>
struct RowsCfg {
  using T = T_;
  static constexpr int D = D_, RTC = RTC_, S = S_, NT = 128 * RTC;
  static constexpr bool kWin = kWin_;
  static constexpr int kTerms = __is_same(T, __half) ? 3 : 2;
  static constexpr int kSideBytes = kTile * D;
  static constexpr int kVfBytes = kTile * D * 2;
  static constexpr int kQBytes = 128 * D;                // one term of a row tile
  static constexpr int kOffV16 = S * 2 * kSideBytes;
  static constexpr int kOffQ = kOffV16 + 2 * kVfBytes;
  static constexpr int kOffSmall = kOffQ + RTC * kTerms * kQBytes;
  // A tile's page constants give way to those of kPages tiles later, which are written when the
  // scores of the tile S before those are done, so after the values of at least two tiles more.
  static constexpr int kPages = RTC == 2 ? 4 : 8;
  // Shares of whole items may be this much longer (see search_line). 256 rows: 32 trees of 64 nodes with a window of
  // 2048 99 us (6) for 123, 24 97 (14) for 106, 5 50 (14) for 48, 3 48 (16) for 45; 2 x 1500 tokens of 8 rows with 1000
  // 47 (7) for 58. 128 rows: trees of 24 nodes, 3 with 2048 29 (16) for 31, 8 with 4096 46 (20) for 45.
  static constexpr int kWholeTiles = RTC == 2 ? 15 : 18;
  // And whole items of up to this many tiles where there is at most one a CTA (128 rows: less than two, for the groups
  // take tiles in turn): one tree of 64 nodes with a window of 512 25.1 us (6 tiles) for 25.8, of 768 28.4 for 27.0, of
  // 2048 45 for 33; two with 1152 (170 tiles) 37 for 43. Of 24 nodes, two with 1536 24.5 (14) for 24.1, with 2048 28.2
  // for 24.1.
  static constexpr int kFewTiles = RTC == 2 ? 6 : 16, kFewLoad = RTC == 2 ? 8 : 15;
  static_assert(S + (RTC == 2 ? 2 : 3) <= kPages, "page constants are read by then");
  static constexpr uint32_t kColS = 0, kColO = 256;      // tensor memory: S of each group, O of each
};

struct __align__(16) RowsSmall {
  uint64_t full[4], empty[4];    // stages
  uint64_t vfull[2], vfree[2];   // widened V
  uint64_t cfull[8], room[8];    // page constants; the keys' warp has room for the tile
  uint64_t sfull[2], pfull[2], ofull[2];   // by group
  uint64_t qfull, done;
  uint32_t vnan[2][4];           // tokens whose values hold NaN (tiles with new tokens)
  uint32_t tmem;
};
// + by tile and 16 tokens the page constants (scale log2(e) ks, log2 vs, 1 / vs) of the last kPages tiles;
// + the queries' units, which, once read, leave their place to the row maxima [group][half][row]
template <class F> constexpr int rows_smem() {
  return F::kOffSmall + static_cast<int>(sizeof(RowsSmall)) + 512 * 4 + F::kPages * 8 * 16;
}

// Bits of the 32 slots from number `j0` among the new tokens on (negative: the cached ones, which
// every row sees) that row (b, i) sees; `n` new tokens.
__device__ __forceinline__ uint32_t seen_bits(const AttnArgs &p, int b, int i, int j0, int n) {
  const int lim = p.a.mask ? n : min(n, i + 1);
  if (j0 >= lim) return 0;
  uint32_t r = 0xffffffffu;
  if (p.a.mask && j0 > -32) {
    const uint32_t *m = p.a.mask + (static_cast<long long>(b) * p.a.N + i) * p.a.W;
    if (j0 < 0) {
      r = (ld_given(m) << -j0) | ((1u << -j0) - 1u);
    } else {
      const int w = j0 >> 5;
      const uint32_t lo = ld_given(m + w), hi = w + 1 < p.a.W ? ld_given(m + w + 1) : 0u;
      r = __funnelshift_r(lo, hi, j0 & 31);
    }
  }
  if (lim - j0 < 32) r &= (1u << (lim - j0)) - 1u;
  return r;
}

// Bits of the 32 slots from `slot` on that a row whose window begins at `lo` sees, sinks among them.
__device__ __forceinline__ uint32_t window_bits(int slot, int lo, int sinks) {
  const int from = lo - slot, early = sinks - slot;
  const uint32_t w = from <= 0 ? ~0u : from < 32 ? ~0u << from : 0u;
  return w | (early >= 32 ? ~0u : early > 0 ? (1u << early) - 1u : 0u);
}

// Half a row of the tile: weights against -nm, as fp16 pairs in h, and their sum over the value scales;
// returns the largest exponent. The next 16 scores are on their way while these are worked on.
template <bool kMasked>
__device__ __forceinline__ float row_weights(uint32_t ts, const float4 *page, float qs, float nm,
                                             const uint32_t (&see)[2], uint32_t (&h)[32],
                                             float &sum) {
  float big = -INFINITY;
  sum = 0.f;
  uint32_t s[2][16];
  tmem_ld(ts, s[0]);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t(&v)[16] = s[c & 1];
    const float4 pg = page[c];
    const float k = pg.x * qs, d = pg.y + nm;
    const f32x2 k2 = pk2(k, k), d2 = pk2(d, d);
    tmem_wait(v);
    if (c < 3) tmem_ld(ts + 16 * (c + 1), s[(c + 1) & 1]);
    f32x2 acc = pk2(0.f, 0.f);
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      float y0, y1;
      up2(fma2(pk2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), k2, d2), y0, y1);
      if (kMasked) {
        const int at = 16 * c + e;
        if (!(see[at >> 5] >> (at & 31) & 1u)) y0 = -INFINITY;
        if (!(see[at >> 5] >> (at & 31) & 2u)) y1 = -INFINITY;
      }
      big = fmaxf(big, fmaxf(y0, y1));
      const float p0 = ex2(y0), p1 = ex2(y1);
      acc = add2(acc, pk2(p0, p1));
      h[8 * c + e / 2] = pack_pair(p0, p1, __half());
    }
    float a0, a1;
    up2(acc, a0, a1);
    sum = __fmaf_rn(a0 + a1, pg.z, sum);
  }
  return big;
}
// The largest y of the half row, without the reference.
template <bool kMasked>
__device__ __forceinline__ float row_maximum(uint32_t ts, const float4 *page, float qs,
                                             const uint32_t (&see)[2]) {
  float big = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t v[16];
    tmem_ld(ts + 16 * c, v);
    const float4 pg = page[c];
    tmem_wait(v);
    const float k = pg.x * qs;
    const uint32_t bits = kMasked ? (c < 2 ? see[0] : see[1]) >> (16 * (c & 1)) : 0xffffu;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float y = __fmaf_rn(__uint_as_float(v[e]), k, pg.y);
      if (!kMasked || (bits >> e & 1u)) big = fmaxf(big, y);
    }
  }
  return big;
}

template <class F>
__global__ void __launch_bounds__(kRowsThreads, 1)
    kv_attention_rows_kernel(const __grid_constant__ CUtensorMap map_k,
                             const __grid_constant__ CUtensorMap map_v,
                             const __grid_constant__ AttnArgs p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  RowsSmall &sm = *reinterpret_cast<RowsSmall *>(smem + F::kOffSmall);
  float4 *pages = reinterpret_cast<float4 *>(smem + F::kOffSmall + sizeof(RowsSmall));
  float *qs = reinterpret_cast<float *>(pages + F::kPages * 8);
  constexpr int NT = F::NT, D = F::D;
  constexpr bool kWin = F::kWin;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // warps of 32 MMA rows that any item uses; the softmax warps of the others take no part in the tiles
  const int quads = F::RTC == 2 ? 4 : static_cast<int>((static_cast<unsigned>(p.a.N) * p.G + 31) / 32);
  if (tid == 0) {
    for (int s = 0; s < F::S; ++s) {
      tc::mbar_init(&sm.full[s], 2);          // the keys' and the values' byte counts
      tc::mbar_init(&sm.empty[s], 1 + kWidenWarps);   // the score MMAs; the widening warps
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm.vfull[i], kWidenWarps);
      tc::mbar_init(&sm.vfree[i], 1);
      tc::mbar_init(&sm.sfull[i], 1);
      tc::mbar_init(&sm.pfull[i], 2 * quads);
      tc::mbar_init(&sm.ofull[i], 1);
    }
    for (int i = 0; i < F::kPages; ++i) tc::mbar_init(&sm.cfull[i], 1);
    for (int i = 0; i < 8; ++i) tc::mbar_init(&sm.room[i], 1);
    tc::mbar_init(&sm.qfull, 1);
    tc::mbar_init(&sm.done, 1);
    tc::mbar_fence_init();
  }
  if (warp == kMma) tmem_alloc(&sm.tmem, 512);
  asm volatile("griddepcontrol.wait;" ::: "memory");   // what is above may run under the kernel before
  int t0 = 0, t1 = 0, total = 0, skip = 0;
  Item<kWin> x{};
  tc::fence_before_sync();
  locate<NT, kRowsThreads, kWin, false, F::kWholeTiles, F::kFewTiles, F::kFewLoad>(p, *reinterpret_cast<LocateScratch<kWin> *>(smem + F::kOffQ), t0, t1, total, x, skip);
  tc::fence_after_sync();
  const uint32_t tmem = sm.tmem;
  // (by a lane of another warp than softmax's first: what one lane of that does here sets it apart from its warp
  // until the first item's end, 18000 clocks for the queries instead of 7000)
  if (tid == 32 * kConsts) publish_range(p, x, skip, t0, t1, total);
  bool ok = true;   // false after a wait gave up: no further waits, and no further work is issued
  // A lane's wait; after one that gave up its lane waits no more but keeps step with its warp, whose
  // loops end by their counts (an `ok` agreed on by vote cost each hand-over about 60 clocks).
  auto wait = [&](uint64_t *bar, int parity) {
    if (!tc::mbar_try(bar, parity) && ok) ok = wait_for(bar, parity);
  };
  if (warp == kCopyK || warp == kCopyV) {
    // One warp copies the keys' pages, one the values', a third works out the page constants. One warp for
    // all of it took 2290 clocks a tile of 16-token pages (the copies 1250 of them), more than the rest
    // of the tile: 58.5 us for 52.3 (64 chains of 6, 16 query heads on 2, 4000 tokens). Where pages are
    // larger or rows more, the copies wait for room and it makes no difference.
    const bool keys = warp == kCopyK;
    const CUtensorMap *map = keys ? &map_k : &map_v;
    const int per_tile = kTile >> p.a.page_shift;
    const uint32_t lane_dst =
        tc::saddr(smem) + (keys ? 0 : F::kSideBytes) + (lane << p.a.page_shift) * D;
    int it = 0;
    for (int t = t0; t < t1 && ok;) {
      const int cnt = min(x.tiles - skip, t1 - t);
      // this lane's page of the next tile: its number, on its way while the tile before waits for room
      const int32_t *table = p.a.page_table + static_cast<long long>(x.b) * p.a.pps;
      const int pages_end = (x.end + p.a.page - 1) >> p.a.page_shift;
      auto place = [&](int k) {   // in the table, of this lane's page in tile k of the segment
        return slot_of<kWin>(x, (skip + k) * kTile + (lane << p.a.page_shift)) >> p.a.page_shift;
      };
      int at = place(0);
      auto wanted = [&]() {
        return lane < per_tile && at < pages_end &&
               span_seen<kWin>(p, x, at << p.a.page_shift, p.a.page);
      };
      auto page_of = [&]() { return wanted() ? ld_given(table + at) : -1; };
      int next = page_of();
      for (int k = 0; k < cnt; ++k, ++it) {
        const int s = it % F::S, page = next;
        const bool want = wanted();
        at = kWin ? place(k + 1) : at + per_tile;
        next = page_of();
        const bool good = page >= 0 && page < p.a.num_pages;
        if (want && !good) set_status(p.a.status, SPEC_ERR_PAGE);
        const uint32_t goods = __ballot_sync(0xffffffffu, good);
        wait(&sm.empty[s], ((it / F::S) & 1) ^ 1);
        if (!__all_sync(0xffffffffu, ok)) {   // no copy into a place that may be in use
          ok = false;
          break;
        }
        if (lane == 0) {
          tc::mbar_expect_tx(&sm.full[s], __popc(goods) * (D << p.a.page_shift));
          if (keys) mbar_arrive(&sm.room[it & 7]);
        }
        __syncwarp();
        if (good)
          tma_load_2d(lane_dst + s * 2 * F::kSideBytes, map, 0,
                      (page * p.a.Hkv + x.h) << p.a.page_shift, &sm.full[s]);
      }
      t += cnt;
      skip = 0;
      if (t < t1) item_next<NT, kWin>(p, x);
    }
    // the last copies of each stage land before the CTA may end
    for (int k = max(0, it - F::S); k < it; ++k)
      if (!wait_for(&sm.full[k % F::S], (k / F::S) & 1)) ok = false;
  } else if (warp == kConsts) {
    // The page constants of every tile, from scales asked for two tiles before, once the keys' warp has
    // room for the tile (it is at most S tiles ahead: a stage is free only when its tile's constants were
    // read, so the eight `room` barriers are never a round off).
    const int per_tile = kTile >> p.a.page_shift, chunks = 1 << (p.a.page_shift - 4);
    int it = 0;
    for (int t = t0; t < t1;) {
      const int cnt = min(x.tiles - skip, t1 - t);
      const int32_t *table = p.a.page_table + static_cast<long long>(x.b) * p.a.pps;
      const int pages_end = (x.end + p.a.page - 1) >> p.a.page_shift;
      // this lane's place in tile k of the segment
      auto place = [&](int k) {
        return slot_of<kWin>(x, (skip + k) * kTile + (lane << p.a.page_shift)) >> p.a.page_shift;
      };
      auto wanted = [&](int at) {
        return lane < per_tile && at < pages_end && span_seen<kWin>(p, x, at << p.a.page_shift, p.a.page);
      };
      auto page_of = [&](int k) {
        const int at = place(k);
        return k < cnt && wanted(at) ? ld_given(table + at) : -1;
      };
      auto scales_of = [&](int page) {
        const int head = page * p.a.Hkv + x.h;
        return page >= 0 && page < p.a.num_pages
                   ? make_float2(ld_given(p.a.k_scale + head), ld_given(p.a.v_scale + head))
                   : make_float2(NAN, NAN);   // what reads a bad page is NaN
      };
      const int full = seen_by_all<NT, kWin>(p, x);
      const int second = page_of(1);
      int next = page_of(2);
      float2 sc = scales_of(page_of(0)), sc1 = scales_of(second);
      for (int k = 0; k < cnt; ++k, ++it) {
        const float2 now = sc;
        const bool want = wanted(place(k));
        sc = sc1;
        sc1 = scales_of(next);
        next = page_of(k + 3);
        // a NaN scale makes its tokens' scores NaN through log2 vs; 1 / vs multiplies the zero weights of
        // the rows that do not see them too, so it stays finite, as everything past the end
        const float vse = now.y < kMinValueScale ? kMinValueScale : now.y;
        float4 c = want ? make_float4(now.x * p.scale2, __log2f(vse),
                                      now.y == now.y ? __frcp_rn(vse) : 1.f, 0.f)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
        if (kWin)   // the page's first slot, and whether the tile needs masks, for the softmax threads
          c.w = __int_as_float(place(k) << p.a.page_shift | (tile_edge<kWin>(p, x, skip + k, full) ? kEdge : 0));
        wait(&sm.room[it & 7], (it >> 3) & 1);
        if (lane < per_tile)
          for (int e = 0; e < chunks; ++e) {
            pages[it % F::kPages * 8 + lane * chunks + e] = c;
            if (kWin) c.w = __int_as_float(__float_as_int(c.w) + 16);   // by 16 tokens
          }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.cfull[it % F::kPages]);
      }
      t += cnt;
      skip = 0;
      if (t < t1) item_next<NT, kWin>(p, x);
    }
  } else if (warp == kMma) {
    // The whole warp walks the units and one elected lane issues. values(u) is followed at once by
    // scores(u + 2), whose scores go where values(u)'s P lies: MMAs run in the order of their issue,
    // so a group's turn costs one hand-over in each direction.
    constexpr uint32_t id_s = attn_idesc(128, kTile, false);
    constexpr uint32_t id_o = (1u << 4) | (1u << 16) | (static_cast<uint32_t>(D >> 3) << 17) |
                              (static_cast<uint32_t>(128 >> 4) << 24);   // B MN-major
    const uint32_t base = tc::saddr(smem);
    int it = 0, seg = 0;
    uint32_t phase = 0;   // bit g: parity of group g's next unit
    auto tile_of = [&](int u) { return it + (F::RTC == 2 ? u >> 1 : u); };
    auto keys_there = [&](int u) {
      const int tile = tile_of(u);
      if (F::RTC == 1 || !(u & 1)) wait(&sm.full[tile % F::S], (tile / F::S) & 1);
    };
    auto scores = [&](int u) {   // one lane
      const int g = u & 1, tile = tile_of(u);
      const uint64_t da = smem_desc<D>(
          base + F::kOffQ + (F::RTC == 2 ? g * F::kTerms * F::kQBytes : 0), 16, 8 * D);
      const uint64_t db = smem_desc<D>(base + tile % F::S * 2 * F::kSideBytes, 16, 8 * D);
      const uint32_t d = tmem + F::kColS + g * 128;
#pragma unroll
      for (int term = 0; term < F::kTerms; ++term)
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk)   // 32 dims of e4m3: 32 bytes on
          mma_f8(d, da + term * (F::kQBytes / 16) + 2 * kk, db + 2 * kk, id_s, (term | kk) != 0);
      mma_commit(&sm.sfull[g]);
      if (F::RTC == 1 || g) mma_commit(&sm.empty[tile % F::S]);
    };
    auto first_scores = [&](int u) {
      keys_there(u);
      __syncwarp();
      tc::fence_after_sync();
      if (elect_one()) scores(u);
      __syncwarp();
    };
    // everything else is waited for before the weights, as a rule the last to come
    auto values = [&](int u, bool last) {
      const int g = u & 1, tile = tile_of(u);
      if (F::RTC == 1 || !g) wait(&sm.vfull[tile & 1], (tile >> 1) & 1);
      if (!last) keys_there(u + 2);
      wait(&sm.pfull[g], phase >> g & 1);
      __syncwarp();
      phase ^= 1u << g;
      tc::fence_after_sync();
      // (N = D dims: one or two blocks of 64)
      const uint64_t db = smem_desc<128>(base + F::kOffV16 + (tile & 1) * F::kVfBytes,
                                         D > 64 ? kTile * 128 : 0, 1024);
      const uint32_t d = tmem + F::kColO + g * D, a = tmem + F::kColS + g * 128;
      const uint32_t later = u < 2 ? 0u : 1u;   // the group's first unit of the segment starts O
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)   // 16 tokens: 8 columns of pairs
          mma_f16_ts(d, a + 8 * kk, db + kk * (16 * 128 / 16), id_o, kk ? 1u : later);
        if (F::RTC == 1 || g) mma_commit(&sm.vfree[tile & 1]);
        if (F::RTC == 1 || last) mma_commit(&sm.ofull[g]);
        if (!last) scores(u + 2);
      }
      __syncwarp();
    };
    for (int t = t0; t < t1; ++seg) {
      const int cnt = min(x.tiles - skip, t1 - t);
      const int units = F::RTC * cnt;
      wait(&sm.qfull, seg & 1);
      first_scores(0);
      if (units > 1) first_scores(1);
      for (int u = 0; u < units; ++u) {
        values(u, u + 2 >= units);
      }
      it += cnt;
      t += cnt;
      skip = 0;
      if (t < t1) item_next<NT, kWin>(p, x);
    }
    if (elect_one()) mma_commit(&sm.done);   // every MMA issued has completed before the CTA may end
    if (!wait_for(&sm.done, 0)) ok = false;
    __syncwarp();
  } else if (warp >= kWidenWarp) {
    const int wtid = tid - 32 * kWidenWarp;
    int it = 0;
    for (int t = t0; t < t1;) {
      const int cnt = min(x.tiles - skip, t1 - t), full = seen_by_all<NT, kWin>(p, x);
      for (int k = 0; k < cnt; ++k, ++it) {
        const int s = it % F::S, buf = it & 1;
        wait(&sm.full[s], (it / F::S) & 1);
        uint4 w[Widen<D, kWidenThreads>::kSteps];
        const bool edge = tile_edge<kWin>(p, x, skip + k, full);
        fetch_values<D, kWidenThreads, kWin>(p, x, smem + s * 2 * F::kSideBytes + F::kSideBytes, wtid, skip + k,
                                             edge, w);
        wait(&sm.vfree[buf], ((it >> 1) & 1) ^ 1);
        __syncwarp();
        if (edge) {
          if (wtid < 4) sm.vnan[buf][wtid] = 0;
          widen_sync();
          scrub_values<D, kWidenThreads>(
              w, wtid, [&](int at) { atomicOr(&sm.vnan[buf][at >> 5], 1u << (at & 31)); });
        }
        widen<D, kWidenThreads>(w, smem + F::kOffV16 + buf * F::kVfBytes, wtid);
        fence_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.empty[s]);
          mbar_arrive(&sm.vfull[buf]);
        }
      }
      t += cnt;
      skip = 0;
      if (t < t1) item_next<NT, kWin>(p, x);
    }
  } else {
    const int grp = warp / kGroupWarps, half = warp >> 2 & 1, quad = warp & 3;
    const int lrow = quad * 32 + lane;                        // row of the MMA tile
    const int n = F::RTC == 2 ? grp * 128 + lrow : lrow;      // row of the item's tile
    const int pair = 4 + grp * 4 + quad;                      // barrier of the two warps with these rows
    const uint32_t tlane = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t ts = tlane + F::kColS + grp * 128;         // the row's scores
    // what the two halves (and, at the end, the groups) of a row tell each other: [group][half][row].
    // The queries' place is free once every score has been taken.
    float *share = reinterpret_cast<float *>(smem + F::kOffQ);
    float *top = qs + grp * 256;
    int it = 0, use = 0, ends = 0;   // tiles so far; this group's units and commits to `ofull` so far
    for (int t = t0; t < t1;) {
      const int cnt = min(x.tiles - skip, t1 - t);
      const RowMap map = RowMap::of<NT>(p, x.rt);
      // rows in use, up to whole warps; the others hold what they held: nothing reads their scores
      const long long used = x.ok ? static_cast<long long>(x.n) * p.G - static_cast<long long>(x.rt) * NT : 0;
      const int fill = static_cast<int>(max(0LL, min(static_cast<long long>(NT), (used + 31) / 32 * 32)));
      load_queries<typename F::T, D, NT, 128, F::kTerms, kSoftThreads, kWin>(p, x, map, fill, tid,
                                                                       smem + F::kOffQ, qs);
      fence_async();
      rows_sync();
      if (tid == 0) mbar_arrive(&sm.qfull);
      int i, gq;
      map.row(n, i, gq);
      const bool live = i < x.n && x.ok;
      const bool idle = !__any_sync(0xffffffffu, live);   // no row of this warp: nothing to weigh
      const float q = qs[n];
      rows_sync();   // `top` takes its place
      float nm = kNoRef, l = 0.f;
      const int plain = kWin ? 0 : seen_by_all<NT, kWin>(p, x) - kTile;   // tiles from slots past this on need masks
      const int lo = kWin && live ? window_start(p, x, i) : 0;
      const int step = F::RTC == 2 ? 1 : 2;
      const int k0 = F::RTC == 2 ? 0 : grp;
      for (int k = quad < quads ? k0 : cnt; k < cnt; k += step, ++use) {
        const int tile = it + k, buf = tile & 1;
        const float4 *page = pages + (tile % F::kPages * 8 + 4 * half);
        bool edge;
        if constexpr (kWin) {
          wait(&sm.cfull[tile % F::kPages], (tile / F::kPages) & 1);
          edge = __any_sync(0xffffffffu, __float_as_int(page->w) & kEdge);   // (the same in all lanes, and known to be)
        } else {
          edge = (skip + k) * kTile > plain;
        }
        uint32_t see[2] = {~0u, ~0u};
        if (edge)
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const int from = kWin ? __float_as_int(page[2 * w].w) & ~kEdge : (skip + k) * kTile + 64 * half + 32 * w;
            see[w] = live ? seen_bits(p, x.b, i, from - x.len, x.n) : 0u;
            if (kWin) see[w] &= window_bits(from, lo, p.sinks);
          }
        if (!kWin) wait(&sm.cfull[tile % F::kPages], (tile / F::kPages) & 1);
        wait(&sm.sfull[grp], use & 1);
        __syncwarp();
        tc::fence_after_sync();
        if (!idle) {
          uint32_t h[32];
          float sum = 0.f;
          bool fresh = k == k0;   // (a row that sees its first token later asks for it by its weights)
#pragma unroll 1
          for (;;) {
            if (fresh) {   // new references: the larger of the halves' maxima
              const float mine = edge ? row_maximum<true>(ts + 64 * half, page, q, see)
                                      : row_maximum<false>(ts + 64 * half, page, q, see);
              top[half * 128 + lrow] = mine;
              pair_any(pair, false);
              const float m = fmaxf(mine, top[(half ^ 1) * 128 + lrow]);
              const bool grow = m + nm > kTrigger;
              const float now = grow ? kBias - m : nm;
              const float f = grow ? ex2(now - nm) : 1.f;   // 2^(m_old - m_new)
              nm = now;
              l *= f;
              if (k > k0)   // the group's earlier value MMAs completed before these scores
#pragma unroll 1
                for (int c = half * (D / 2); c < half * (D / 2) + D / 2; c += 16) {
                  uint32_t o[16];
                  tmem_ld(tlane + F::kColO + grp * D + c, o);
                  tmem_wait(o);
#pragma unroll
                  for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                  tmem_st(tlane + F::kColO + grp * D + c, o);
                }
            }
            const float big = edge ? row_weights<true>(ts + 64 * half, page, q, nm, see, h, sum)
                                   : row_weights<false>(ts + 64 * half, page, q, nm, see, h, sum);
            // (also: both halves have read their scores, which P is about to overwrite)
            if (!pair_any(pair, !fresh && big > kTrigger)) break;
            fresh = true;
          }
          l += sum;
          if (edge) {   // values with NaN went into the product as zeros: the rows that see them are NaN
            wait(&sm.vfull[buf], (tile >> 1) & 1);
            if ((sm.vnan[buf][2 * half] & see[0]) | (sm.vnan[buf][2 * half + 1] & see[1])) l = NAN;
          }
          tmem_st(ts + 32 * half, h);
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.pfull[grp]);
      }
      it += cnt;
      // The item's (or its part's) result.
      const bool whole = skip == 0 && cnt == x.tiles;
      const long long part = 2LL * blockIdx.x + (skip == 0 ? 1 : 0);
      if (F::RTC == 2 || use > 0) wait(&sm.ofull[grp], F::RTC == 2 ? ends++ & 1 : (use - 1) & 1);
      __syncwarp();
      tc::fence_after_sync();
      rows_sync();   // every MMA of the item has completed: the queries' place is free
      float *mine = share + (grp * 2 + half) * 256;
      mine[lrow] = l;
      mine[128 + lrow] = nm;
      rows_sync();
      auto sum_of = [&](int g) { return share[g * 512 + lrow] + share[g * 512 + 256 + lrow]; };
      float f0 = 0.f, f1 = 0.f;   // what the accumulator(s) are multiplied by
      float lse2;
      if constexpr (F::RTC == 2) {
        const float total = sum_of(grp);
        lse2 = total == 0.f ? -INFINITY : __log2f(total) - nm;
        f0 = total == 0.f ? 0.f : __frcp_rn(total);
      } else {
        const float n0 = share[128 + lrow], n1 = share[512 + 128 + lrow];
        const float l0 = sum_of(0), l1 = sum_of(1);
        const float m = fminf(n0, n1);   // -m of the larger reference
        const float w0 = ex2(m - n0), w1 = ex2(m - n1);
        const float total = l0 * w0 + l1 * w1;
        const float inv = total == 0.f ? 0.f : __frcp_rn(total);
        lse2 = total == 0.f ? -INFINITY : __log2f(total) - m;
        f0 = l0 == 0.f ? 0.f * inv : w0 * inv;   // (0 NaN is NaN)
        f1 = l1 == 0.f ? 0.f * inv : w1 * inv;
      }
      if (!x.ok) lse2 = f0 = NAN;
      if (i < p.a.N && half == 0 && (F::RTC == 2 || grp == 0)) {
        if (!whole)
          p.part_lse[part * NT + n] = lse2;
        else if (p.lse)
          p.lse[(static_cast<long long>(x.b) * p.a.N + i) * p.a.Hq +
                static_cast<long long>(x.h) * p.G + gq] = live || !x.ok ? lse2 * kLn2 : -INFINITY;
      }
      const bool zero = x.ok && !live;   // padding
      // the dims shared out over the warps with these rows: two, or four when the groups share them
      constexpr int kDims = F::RTC == 2 ? D / 2 : D / 4;
      const int d0 = (F::RTC == 2 ? half : grp * 2 + half) * kDims;
      using T = typename F::T;
      T *out = static_cast<T *>(p.out) + ((static_cast<long long>(x.b) * p.a.N + i) * p.a.Hq +
                                          static_cast<long long>(x.h) * p.G + gq) * D;
      float *po = p.part_o + (part * NT + n) * D;
      if (__any_sync(0xffffffffu, i < p.a.N))   // (whole warps)
#pragma unroll
      for (int c = d0; c < d0 + kDims; c += 16) {
        uint32_t o[16], o1[16];
        tmem_ld(tlane + F::kColO + (F::RTC == 2 ? grp * D : 0) + c, o);
        if (F::RTC == 1) tmem_ld(tlane + F::kColO + D + c, o1);
        tmem_wait(o);
        if (F::RTC == 1) tmem_wait(o1);
        if (i < p.a.N && SPEC_CHECK(p.a, n < NT && part < 2LL * gridDim.x && x.b < p.a.B && gq < p.G)) {
          float v[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            // an accumulator that nothing was added to counts 0 whatever it holds
            v[e] = f0 == 0.f ? 0.f : __uint_as_float(o[e]) * f0;
            if (F::RTC == 1) v[e] += f1 == 0.f ? 0.f : __uint_as_float(o1[e]) * f1;
            if (zero) v[e] = 0.f;
          }
          if (!whole) {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<float4 *>(po + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
          } else {
#pragma unroll
            for (int e = 0; e < 16; e += 8)
              *reinterpret_cast<uint4 *>(out + c + e) =
                  make_uint4(pack_pair(v[e], v[e + 1], T()), pack_pair(v[e + 2], v[e + 3], T()),
                             pack_pair(v[e + 4], v[e + 5], T()), pack_pair(v[e + 6], v[e + 7], T()));
          }
        }
      }
      if (!x.ok && tid == 0) set_status(p.a.status, SPEC_ERR_LENGTH);
      tc::fence_before_sync();
      rows_sync();   // every accumulator and `share` are read before the next item writes
      t += cnt;
      skip = 0;
      if (t < t1) item_next<NT, kWin>(p, x);
    }
  }
  if (!ok) set_status(p.a.status, SPEC_ERR_TIMEOUT);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMma) {
    tc::fence_after_sync();
    tmem_free(tmem, 512);
  }
}

template <class F>
cudaError_t launch_cfg(AttnArgs &p, const CUtensorMap &mk, const CUtensorMap &mv, int ctas, char *ws,
                       cudaStream_t stream) {
  static std::atomic<bool> ready[64];
  constexpr int smem = rows_smem<F>();
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  cudaError_t e = allow_smem(kv_attention_rows_kernel<F>, smem, ready);
  if (e != cudaSuccess) return e;
  plan_parts(p, ws, F::NT);
  e = launch_kv(kv_attention_rows_kernel<F>, ctas, kRowsThreads, smem, stream, mk, mv, static_cast<const AttnArgs &>(p));
  return e != cudaSuccess ? e : launch_join<typename F::T, F::D, F::NT>(p, ctas, stream);
}

template <typename T, int D, bool kWin>
cudaError_t launch_rows_of(AttnArgs &p, const CUtensorMap &mk, const CUtensorMap &mv, int ctas,
                           char *ws, cudaStream_t stream) {
  if (kv_row_tile(static_cast<long long>(p.a.N) * p.G) == 256)
    return launch_cfg<RowsCfg<T, D, 2, 2, kWin>>(p, mk, mv, ctas, ws, stream);
  return launch_cfg<RowsCfg<T, D, 1, 3, kWin>>(p, mk, mv, ctas, ws, stream);
}

template <bool kWin>
cudaError_t launch_rows(AttnArgs &p, int dtype, const CUtensorMap &mk, const CUtensorMap &mv, int ctas,
                        char *ws, cudaStream_t stream) {
  if (dtype == SPEC_BF16)
    return p.a.D == 64 ? launch_rows_of<__nv_bfloat16, 64, kWin>(p, mk, mv, ctas, ws, stream)
                       : launch_rows_of<__nv_bfloat16, 128, kWin>(p, mk, mv, ctas, ws, stream);
  return p.a.D == 64 ? launch_rows_of<__half, 64, kWin>(p, mk, mv, ctas, ws, stream)
                     : launch_rows_of<__half, 128, kWin>(p, mk, mv, ctas, ws, stream);
}

}  // namespace

}  // namespace specv
