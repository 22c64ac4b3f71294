// spec_kv_attn.h -- what the two attention kernels share: tensor-core and barrier helpers, the line
// of 128-token tiles and its even cut over the SMs, queries as e4m3 terms, values widened to fp16, and
// the join of the parts of an item that several CTAs worked on.
#pragma once

#include <cudaTypedefs.h>

#include <atomic>

#include "spec_kv.h"
#include "spec_tc.cuh"

namespace specv {
namespace attn {

constexpr int kTile = 128;          // tokens
constexpr int kMaxCtas = 152;       // workspace parts are sized for this many CTAs
constexpr float kNoRef = 1e30f;     // -m of a row that has seen nothing
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kMinValueScale = 8.271806125530277e-25f;   // 2^-80: a zero scale's logarithm

struct AttnArgs {
  KvArgs a;
  const void *q;
  long long q_stride;
  float scale2;        // scale * log2(e)
  void *out;
  float *lse;
  float *part_o;       // [2 G][NT][D]
  float *part_lse;     // [2 G][NT], base 2
  int4 *start;         // [G]: (item's b, h, row tile, first tile) of each CTA's range; then [G]
                       // its tiles
  int G;               // query heads per key head
  int RT;              // row tiles
  int window, sinks;   // (windowed kernels) a query at position p sees slots past p - window, and the first
                       // `sinks`
};

// ------------------------------------------------------------------ tensor-core helpers

__device__ __forceinline__ void mbar_arrive(uint64_t *b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc::saddr(b)) : "memory");
}
// an arrival once this thread's cp.async copies so far have landed (counted at initialisation)
__device__ __forceinline__ void mbar_arrive_copies(uint64_t *b) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::saddr(b))
               : "memory");
}
__device__ __forceinline__ void copy4(void *dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(tc::saddr(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, int c0, int c1,
                                            uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(tc::saddr(bar))
      : "memory");
}
__device__ __forceinline__ void tmem_alloc(uint32_t *slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   tc::saddr(slot)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          tc::saddr(bar))
      : "memory");
}
// 4 / 8 / 16 consecutive fp32 columns of this thread's lane; valid after tmem_wait of the same array
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&v)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}
// the registers pass through, so nothing that uses them is scheduled ahead of the wait
template <int K>
__device__ __forceinline__ void tmem_wait(uint32_t (&v)[K]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < K; ++i) asm volatile("" : "+r"(v[i]));
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, "
      "%10, %11, %12, %13, %14, %15};" ::"r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
      "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, "
      "%10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31};" ::"r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
      "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
      "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
      "r"(v[29]), "r"(v[30]), "r"(v[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// true in one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
// tc::mbar_wait in line: no call, whose registers would be kept free around every wait
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity) {
  if (tc::mbar_try(bar, parity)) return true;
  const unsigned long long t0 = tc::now_ns();
#pragma unroll 1
  while (!tc::mbar_try(bar, parity))
    if (tc::now_ns() - t0 > tc::kWaitNs) return false;
  return true;
}
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Byte offset `at` of a tile whose rows are `kSpan` bytes (32, 64 or 128), swizzled as TMA and the
// MMA do: the 16-byte chunk number exclusive-or the bits from 7 up.
template <int kSpan>
__device__ __forceinline__ uint32_t swz(uint32_t at) {
  constexpr uint32_t m = kSpan == 128 ? 7u : kSpan == 64 ? 3u : 1u;
  return at ^ (((at >> 7) & m) << 4);
}
// Shared-memory matrix descriptor: start, leading and stride byte offsets in units of 16 bytes,
// version 1, swizzle mode (2: 128 bytes, 4: 64, 6: 32). K-major operands: rows of the swizzle span,
// 8-row atoms `sbo` apart. MN-major operands: k rows of the span (8 of them an atom, atoms `sbo`
// apart), spans of consecutive m or n `lbo` apart.
template <int kSpan>
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  constexpr uint64_t mode = kSpan == 128 ? 2 : kSpan == 64 ? 4 : 6;
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) |
         (static_cast<uint64_t>(sbo >> 4) << 32) | (1ull << 46) | (mode << 61);
}
// Instruction descriptor: fp32 accumulator; A and B e4m3 (kind::f8f6f4) or fp16 (kind::f16), both
// format 0; bits 15, 16: A, B are MN-major
__host__ __device__ constexpr uint32_t attn_idesc(int M, int N, bool mn_major) {
  return (1u << 4) | (mn_major ? 3u << 15 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// ------------------------------------------------------------------ the line of tiles

// With a window: the first slot of any row's window, and of the last row's (every row's window has begun by
// then); of the slots from 0 on, `gap` are left out after the first `head` ones, which hold the sinks (both whole
// pages and multiples of 32).
template <bool kWin> struct WindowPart {
  int lo, lo_all, head, gap;
};
template <> struct WindowPart<false> {
  static constexpr int lo = 0, lo_all = 0, head = 0, gap = 0;
};
template <bool kWin> struct Item : WindowPart<kWin> {   // one (sequence, key head, row tile)
  int b, h, rt;
  int len, n;      // tokens before the new ones; new ones
  bool ok;         // lengths fit
  int end;         // first slot that no row sees
  int tiles;       // tiles that some row sees
};

template <int NT>
__device__ __forceinline__ int item_end(const AttnArgs &p, int len, int n, bool ok, int rt) {
  if (!ok || n == 0) return 0;
  if (p.RT == 1 || p.a.mask) return len + n;
  const int first = static_cast<int>(static_cast<unsigned>(rt) * NT / p.G);
  if (first >= n) return 0;   // padding
  const int last = static_cast<int>((static_cast<unsigned>(rt) * NT + NT - 1) / p.G);
  return len + min(last + 1, n);
}
// The slots below it are seen by every row of the item that has a token: what lies past the first
// token's place may be hidden from some.
template <int NT, bool kWin>
__device__ __forceinline__ int seen_by_all(const AttnArgs &p, const Item<kWin> &x) {
  const int first = static_cast<int>(static_cast<unsigned>(x.rt) * NT / p.G);
  return min(x.len + (p.a.mask ? 0 : first + 1), x.end);
}
__device__ __forceinline__ int tiles_for(int end) { return end > kTile ? (end + kTile - 1) / kTile : 1; }

// What a row tile's item is, from its lengths.
template <int NT, bool kWin>
__device__ __forceinline__ void item_span(const AttnArgs &p, Item<kWin> &x) {
  x.end = item_end<NT>(p, x.len, x.n, x.ok, x.rt);
  x.tiles = tiles_for(x.end);
  if constexpr (kWin) {
    x.lo = x.lo_all = x.head = x.gap = 0;
    if (x.end == 0) return;   // (its lengths may be anything)
    // Positions of the item's rows: a chain's are its tokens', a tree's at least the root's and at most as
    // deep as it has nodes. (Numbers of at most 2^30, as is the window: no overflow.)
    const int first = p.a.mask ? 0 : static_cast<int>(static_cast<unsigned>(x.rt) * NT / p.G);
    const int last = p.a.mask ? p.a.N - 1 : x.end - 1 - x.len;
    x.lo = max(0, x.len + first - p.window + 1);
    x.lo_all = max(0, x.len + last - p.window + 1);
    const int grain = max(p.a.page, 32);
    const int low = min(x.lo, x.end - 1) & -grain, early = (min(p.sinks, x.end) + grain - 1) & -grain;
    if (low > early) {
      x.head = early;
      x.gap = low - early;
    }
    x.tiles = tiles_for(x.end - x.gap);
  }
}
// The tokens of an item's tiles are its slots in order, but for the gap: the slot that token v is in.
template <bool kWin>
__device__ __forceinline__ int slot_of(const Item<kWin> &x, int v) {
  return kWin && v >= x.head ? v + x.gap : v;
}
// Whether some row's window, or the sinks, reach into slots [slot, slot + n).
template <bool kWin>
__device__ __forceinline__ bool span_seen(const AttnArgs &p, const Item<kWin> &x, int slot, int n) {
  return !kWin || slot + n > x.lo || slot < p.sinks;
}
// Whether some row does not see all of tile k; slots below `full` are hidden from none but by its window.
template <bool kWin>
__device__ __forceinline__ bool tile_edge(const AttnArgs &p, const Item<kWin> &x, int k, int full) {
  const int v = k * kTile, s = slot_of<kWin>(x, v);
  if (!kWin) return v + kTile > full;
  if (v < x.head && v + kTile > x.head) return true;   // sinks and window
  return s + kTile > full || (s < x.lo_all && s + kTile > p.sinks);
}

// The first slot in the window of new token i, whose position is its slot's, or in a tree its depth's.
template <bool kWin>
__device__ __forceinline__ int window_start(const AttnArgs &p, const Item<kWin> &x, int i) {
  int at = i;
  if (p.a.mask) {
    const uint32_t *m = p.a.mask + (static_cast<long long>(x.b) * p.a.N + i) * p.a.W;
    int bits = 0;
#pragma unroll 1
    for (int w = 0; w < p.a.W; ++w) bits += __popc(ld_given(m + w));
    at = max(bits - 1, 0);
  }
  return x.len + at - p.window + 1;
}

template <int NT, bool kWin>
__device__ __forceinline__ void item_load(const AttnArgs &p, Item<kWin> &x) {
  x.ok = kv_lengths(p.a, x.b, x.len, x.n);
  item_span<NT, kWin>(p, x);
}
template <int NT, bool kWin>
__device__ __forceinline__ void item_next(const AttnArgs &p, Item<kWin> &x) {
  if (++x.rt == p.RT) {
    x.rt = 0;
    if (++x.h == p.a.Hkv) {
      x.h = 0;
      ++x.b;
    }
  }
  if (x.b >= p.a.B) return;
  if (x.h == 0 && x.rt == 0) {   // another sequence
    item_load<NT, kWin>(p, x);
  } else if (p.RT > 1) {
    item_span<NT, kWin>(p, x);
  }
}
// Range c of G of a line of T tiles begins at floor(T c / G), in 32 bits (c <= G <= kMaxCtas); range_of: the range
// that holds tile t.
__device__ __forceinline__ int range_start(int T, int c, int G) {
  const int q = T / G;
  return q * c + (T - q * G) * c / G;
}
__device__ __forceinline__ int range_of(int T, int t, int G) {
  return static_cast<int>((static_cast<unsigned long long>(t + 1) * G + T - 1) / T) - 1;
}

// The CTA's range [t0, t1) of the line and its first item; called by all threads. With one row tile an item each
// thread sums the sequences of its own contiguous share; with more, each warp does, its lanes a row tile each.
// Whoever's share holds an end of the range finds the item there. (One thread that went through the row tiles
// one after another took 94000 clocks for 47 of them.)
//
// Ranges are equal, but for this: where windows make items short, and shares of whole items would be at most
// kWhole tiles longer, the CTAs take those. Then no item has parts that are written, read back and joined,
// which costs more than the tiles. Where there are so few tiles a CTA (up to kFewLoad eighths) that with an even cut
// hardly any begins a second item, that costs less: there whole items are taken up to kFew tiles.
template <bool kWin> struct LocateScratch {
  int warp_sum[32], warp_most[32];
  Item<kWin> x;
  int t0, t1, total, skip;
};
// The sum over the lanes of the tiles of one key head of x.b, 32 row tiles at a time; all lanes.
template <int NT, bool kWin>
__device__ __forceinline__ int warp_head_tiles(const AttnArgs &p, Item<kWin> &x, int lane, int &most,
                                               int &gaps) {
  x.ok = kv_lengths(p.a, x.b, x.len, x.n);
  int s = 0;
#pragma unroll 1
  for (x.rt = lane; x.rt < p.RT; x.rt += 32) {
    item_span<NT, kWin>(p, x);
    s += x.tiles;
    most = max(most, x.tiles);
    gaps |= x.gap;
  }
  return __reduce_add_sync(0xffffffffu, s);
}
template <int NT, int kThreads, bool kWin, int kWhole, int kFew, int kFewLoad>
__device__ __forceinline__ void search_line(const AttnArgs &p, LocateScratch<kWin> &sm) {
  constexpr int kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool one = p.RT == 1;
  const int sharers = one ? kThreads : kWarps, me = one ? tid : warp;
  const int share = (p.a.B + sharers - 1) / sharers;
  const int lo = min(p.a.B, me * share), hi = min(p.a.B, lo + share);
  Item<kWin> y{};
  int mine = 0, most = 0, gaps = 0;
#pragma unroll 1
  for (y.b = lo; y.b < hi; ++y.b) {
    if (one) {
      item_load<NT, kWin>(p, y);
      mine += y.tiles * p.a.Hkv;
      most = max(most, y.tiles);
      gaps |= y.gap;
    } else {
      mine += warp_head_tiles<NT, kWin>(p, y, lane, most, gaps) * p.a.Hkv;
    }
  }
  if (kWin) {   // (a gap: some item is shorter for its window)
    most = __reduce_max_sync(0xffffffffu, most);
    gaps = __any_sync(0xffffffffu, gaps != 0);
  }
  int incl = mine;   // of the thread's share within the warp
  if (one)
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
  if (lane == 31) {
    sm.warp_sum[warp] = incl;
    if (kWin) sm.warp_most[warp] = 2 * most + gaps;
  }
  __syncthreads();
  const int w = lane < kWarps ? sm.warp_sum[lane] : 0;
  int upto = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  const int all = __shfl_sync(0xffffffffu, upto, 31);
  const int G = gridDim.x;
  if constexpr (kWin) {
    const int known = lane < kWarps ? sm.warp_most[lane] : 0;
    most = __reduce_max_sync(0xffffffffu, known) >> 1;
    gaps = __any_sync(0xffffffffu, known & 1);
    const int items = p.a.B * p.a.Hkv * p.RT;
    const int each = (items + G - 1) / G;
    const bool whole = 8LL * all <= kFewLoad * G ? most <= kFew : static_cast<long long>(each) * most <= all / G + kWhole;
    if (gaps && whole) {   // (so the numbers below are small)
      const int i0 = range_start(items, blockIdx.x, G), n = range_start(items, blockIdx.x + 1, G) - i0;
      if (warp == 0) {
        int sum = 0;
        for (int i = lane; i < n; i += 32) {
          y.rt = (i0 + i) % p.RT;
          y.h = (i0 + i) / p.RT % p.a.Hkv;
          y.b = (i0 + i) / p.RT / p.a.Hkv;
          item_load<NT, kWin>(p, y);
          sum += y.tiles;
          if (i == 0) sm.x = y;
        }
        sum = __reduce_add_sync(0xffffffffu, sum);
        if (lane == 0) {
          sm.t0 = sm.skip = 0;
          sm.t1 = sum;
          sm.total = all;
        }
      }
      return;
    }
  }
  int at = __shfl_sync(0xffffffffu, upto - w, warp) + incl - mine;
  const int first = range_start(all, blockIdx.x, G);
  if (tid == 0) {
    sm.t0 = first;
    sm.t1 = range_start(all, blockIdx.x + 1, G);
    sm.total = all;
  }
  if (first >= at && first < at + mine) {
    y.rt = 0;
    int left, per_head;
#pragma unroll 1
    for (y.b = lo;; ++y.b) {
      if (one) {
        item_load<NT, kWin>(p, y);
        per_head = y.tiles;
      } else {
        per_head = warp_head_tiles<NT, kWin>(p, y, lane, most, gaps);
      }
      left = first - at;
      if (left < per_head * p.a.Hkv) break;
      at += per_head * p.a.Hkv;
    }
    y.h = left / per_head;
    left -= y.h * per_head;
    if (one) {
      sm.x = y;
      sm.skip = left;
    } else {
#pragma unroll 1
      for (y.rt = lane;; y.rt += 32) {   // 32 row tiles at a time
        int n = 0;
        if (y.rt < p.RT) {
          item_span<NT, kWin>(p, y);
          n = y.tiles;
        }
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += v;
        }
        if (left >= sum - n && left < sum) {
          sm.x = y;
          sm.skip = left - (sum - n);
        }
        const int chunk = __shfl_sync(0xffffffffu, sum, 31);
        if (left < chunk) break;
        left -= chunk;
      }
    }
  }
}
template <int NT, int kThreads, bool kWin, int kWhole, int kFew, int kFewLoad>
__device__ __noinline__ void search_line_apart(const AttnArgs &p, LocateScratch<kWin> &sm) {
  search_line<NT, kThreads, kWin, kWhole, kFew, kFewLoad>(p, sm);
}
// kApart: by a call, with registers of its own (the kernel for few rows spills less with it, the other more).
template <int NT, int kThreads, bool kWin, bool kApart, int kWhole, int kFew, int kFewLoad>
__device__ __forceinline__ void locate(const AttnArgs &p, LocateScratch<kWin> &sm, int &t0, int &t1,
                                       int &total, Item<kWin> &x, int &skip) {
  if constexpr (kApart)
    search_line_apart<NT, kThreads, kWin, kWhole, kFew, kFewLoad>(p, sm);
  else
    search_line<NT, kThreads, kWin, kWhole, kFew, kFewLoad>(p, sm);
  __syncthreads();
  x = sm.x;
  t0 = sm.t0;
  t1 = sm.t1;
  total = sm.total;
  skip = sm.skip;
  __syncthreads();   // the scratch may be put to other use
}
// What the join needs to know of the CTA's range: its first item and the item's tiles before it,
// the item's tiles, the range, and the length of the line.
template <bool kWin>
__device__ __forceinline__ void publish_range(const AttnArgs &p, const Item<kWin> &x, int skip, int t0,
                                              int t1, int total) {
  if (t0 < t1) p.start[blockIdx.x] = make_int4(x.b, x.h, x.rt, skip);
  p.start[gridDim.x + blockIdx.x] = make_int4(t0 < t1 ? x.tiles : 0, t0, t1, total);
}

// ------------------------------------------------------------------ operands

// The token and query head of row n < 256 of a row tile: one division for the tile, then an exact
// quotient of small numbers ((t + 1/2) / G is 1/2G away from an integer at least, the product's error
// below 2^-8 / G for t < 2^15).
struct RowMap {
  int i0, g0, G;
  float inv;
  template <int NT>
  static __device__ __forceinline__ RowMap of(const AttnArgs &p, int rt) {
    RowMap m;
    const unsigned r = static_cast<unsigned>(rt) * NT;
    m.G = p.G;
    m.i0 = static_cast<int>(r / p.G);
    m.g0 = static_cast<int>(r - static_cast<unsigned>(m.i0) * p.G);
    m.inv = __frcp_rn(static_cast<float>(p.G));
    return m;
  }
  __device__ __forceinline__ void row(int n, int &i, int &g) const {
    const int t = g0 + n;
    const int d = static_cast<int>((static_cast<float>(t) + 0.5f) * inv);
    i = i0 + d;
    g = t - d * G;
  }
};

// Eight dims (number `sub`) of row n as e4m3 terms in shared memory, by the kLanes lanes that have the row, in
// units of a power of two that puts its largest element in [2^7, 2^8); qs[n] undoes it. Two terms hold bf16's 8
// significant bits exactly for elements from 2^-2 on, three fp16's 11 from 2 on; below that they are off by
// at most 2^-10, half the smallest e4m3 value. Blocks of kBlock rows, each term of a block a K-major operand.
template <typename T, int D, int kBlock, int kTerms, int kLanes>
__device__ __forceinline__ void store_query(uint4 raw, int n, int sub, uint8_t *sq, float *qs) {
  float f[8];
  vec_to_floats<T>(raw, f);
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmax_nan(m, fabsf(f[e]));
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  const int e = max(static_cast<int>(__float_as_uint(m) >> 23), 27);   // exponent, at least -100
  const float mul = __uint_as_float(static_cast<uint32_t>(127 + 127 + 7 - e) << 23);
  if (sub == 0)
    qs[n] = m < INFINITY ? __uint_as_float(static_cast<uint32_t>(e - 7) << 23) : NAN;
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] *= mul;
  uint8_t *blk = sq + n / kBlock * (kTerms * kBlock * D);
#pragma unroll
  for (int t = 0; t < kTerms; ++t) {
    const uint2 w = floats_to_e4m3(f, 1.f);
    *reinterpret_cast<uint2 *>(blk + t * (kBlock * D) + swz<D>(n % kBlock * D + sub * 8)) = w;
    if (t + 1 < kTerms) {
      float g8[8];
      e4m3_to_floats(w, g8);
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] -= g8[k];   // exact
    }
  }
}
// The rows 0 .. NT - 1 of an item: of them the first `rows` (a multiple of 16) are written, zero past the item's.
template <typename T, int D, int NT, int kBlock, int kTerms, int kThreads, bool kWin>
__device__ __forceinline__ void load_queries(const AttnArgs &p, const Item<kWin> &x, const RowMap &map,
                                             int rows, int tid, uint8_t *sq, float *qs) {
  constexpr int kLanes = D / 8, kRows = kThreads / kLanes;
  constexpr int kSteps = (NT + kRows - 1) / kRows, kAhead = kSteps < 4 ? kSteps : 4;
  const int sub = tid % kLanes, row0 = tid / kLanes;
  const T *base = static_cast<const T *>(p.q) +
                  static_cast<long long>(x.b) * p.a.N * p.q_stride +
                  static_cast<long long>(x.h) * p.G * D + sub * 8;
#pragma unroll 1
  for (int n0 = row0; n0 < rows; n0 += kAhead * kRows) {   // whole warps: a warp's rows are 2 or 4
    uint4 raw[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int n = n0 + u * kRows;
      int i, g;
      map.row(n, i, g);
      raw[u] = make_uint4(0, 0, 0, 0);
      if (n < rows && i < x.n && x.ok)
        raw[u] = ld_given(reinterpret_cast<const uint4 *>(
            base + static_cast<long long>(i) * p.q_stride + static_cast<long long>(g) * D));
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int n = n0 + u * kRows;
      if (n >= rows) break;
      store_query<T, D, kBlock, kTerms, kLanes>(raw[u], n, sub, sq, qs);
    }
  }
}

// V's bytes of a tile, on their way to fp16: 16 bytes a lane and step, whole rows side by side.
template <int D, int kThreads> struct Widen {
  static constexpr int kLanes = D / 16;             // lanes of a token
  static constexpr int kRows = kThreads / kLanes;   // tokens a step
  static constexpr int kSteps = kTile / kRows;
};
// Tokens of tile k that no row sees count as zeros. (edge: see tile_edge; with a window only such tiles have any.)
template <int D, int kThreads, bool kWin>
__device__ __forceinline__ void fetch_values(const AttnArgs &p, const Item<kWin> &x, const uint8_t *sv, int gtid,
                                             int k, bool edge, uint4 (&w)[Widen<D, kThreads>::kSteps]) {
  using W = Widen<D, kThreads>;
#pragma unroll
  for (int u = 0; u < W::kSteps; ++u) {
    const int t = u * W::kRows + gtid / W::kLanes;
    w[u] = *reinterpret_cast<const uint4 *>(sv + t * D + gtid % W::kLanes * 16);
    if (!kWin && k * kTile + t >= x.end) w[u] = make_uint4(0, 0, 0, 0);
  }
  if (kWin && edge)
#pragma unroll
    for (int u = 0; u < W::kSteps; ++u) {
      const int slot = slot_of<kWin>(x, k * kTile + u * W::kRows + gtid / W::kLanes);
      if (slot >= x.end || !span_seen<kWin>(p, x, slot, 1)) w[u] = make_uint4(0, 0, 0, 0);
    }
}
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {   // bit 7 of each NaN byte
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}
// NaN codes made zero; `mark`(token) is called for each token that had one. Returns whether any had.
// For tiles that not every row sees whole: there the weights of the rows that do see such a token are
// made NaN instead, since a NaN operand would reach the rows that do not (0 NaN is NaN). Where every
// row sees every token the operand may stay NaN.
template <int D, int kThreads, typename Mark>
__device__ __forceinline__ bool scrub_values(uint4 (&w)[Widen<D, kThreads>::kSteps], int gtid,
                                             Mark mark) {
  using W = Widen<D, kThreads>;
  bool any = false;
#pragma unroll
  for (int u = 0; u < W::kSteps; ++u) {
    const uint32_t hx = nan_codes(w[u].x), hy = nan_codes(w[u].y), hz = nan_codes(w[u].z),
                   hw = nan_codes(w[u].w);
    if (hx | hy | hz | hw) {
      w[u].x &= ~((hx >> 7) * 255u);
      w[u].y &= ~((hy >> 7) * 255u);
      w[u].z &= ~((hz >> 7) * 255u);
      w[u].w &= ~((hw >> 7) * 255u);
      mark(u * W::kRows + gtid / W::kLanes);
      any = true;
    }
  }
  return any;
}
// The values as fp16 rows of 64 dims (128 bytes, swizzled): 64 dims (4 lanes) a block of kTile rows;
// the second block's lanes store their halves the other way round, so that eight neighbours never
// meet in a bank.
template <int D, int kThreads>
__device__ __forceinline__ void widen(const uint4 (&w)[Widen<D, kThreads>::kSteps], uint8_t *out,
                                      int gtid) {
  using W = Widen<D, kThreads>;
  const int c = gtid % W::kLanes, row0 = gtid / W::kLanes;
  uint8_t *blk = out + (c >> 2) * (kTile * 128);
  const bool flip = (c >> 2) & 1;
#pragma unroll
  for (int u = 0; u < W::kSteps; ++u) {
    const int t = u * W::kRows + row0;
    const uint4 lo = make_uint4(e4m3_to_half2(w[u].x & 0xffffu), e4m3_to_half2(w[u].x >> 16),
                                e4m3_to_half2(w[u].y & 0xffffu), e4m3_to_half2(w[u].y >> 16));
    const uint4 hi = make_uint4(e4m3_to_half2(w[u].z & 0xffffu), e4m3_to_half2(w[u].z >> 16),
                                e4m3_to_half2(w[u].w & 0xffffu), e4m3_to_half2(w[u].w >> 16));
    const uint32_t a0 = swz<128>(t * 128 + (c & 3) * 32), a1 = swz<128>(t * 128 + (c & 3) * 32 + 16);
    *reinterpret_cast<uint4 *>(blk + (flip ? a1 : a0)) = flip ? hi : lo;
    *reinterpret_cast<uint4 *>(blk + (flip ? a0 : a1)) = flip ? lo : hi;
  }
}

// ------------------------------------------------------------------ the join

// Joins the parts of the items that cross ranges, in the order of the line. Block (c, rows): the item
// that range c begins inside of, if c is the first range to do so; kJoinRows rows a warp, whose loads
// overlap. The ranges are arithmetic, so every load but the first two waits for nothing but those.
constexpr int kJoinRows = 4, kJoinBlockRows = 8 * kJoinRows;

template <typename T, int D, int NT>
__global__ void __launch_bounds__(256) kv_attention_join(const __grid_constant__ AttnArgs p,
                                                         int ctas) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kRows = NT < kJoinBlockRows ? NT / 8 : kJoinRows;   // of a warp
  constexpr int kBlocks = NT / (8 * kRows), E = D / 32;
  const int c = 1 + blockIdx.x / kBlocks;
  const int n0 = (blockIdx.x % kBlocks) * 8 * kRows + (threadIdx.x >> 5) * kRows;
  const int lane = threadIdx.x & 31;
  // (written by other CTAs: read from L2)
  const int4 s = __ldcg(p.start + c);          // its first item: b, h, row tile, tiles before
  const int4 d = __ldcg(p.start + ctas + c);   // that item's tiles, t0, t1, all tiles
  if (d.y >= d.z || s.w == 0) return;
  const int total = d.w, begin = d.y - s.w, end = begin + d.x;   // the item's tiles on the line
  const int first = range_of(total, begin, ctas);
  // with fewer tiles than ranges each part is a tile
  const int parts = total >= ctas ? range_of(total, end - 1, ctas) - first + 1 : d.x;
  auto cta = [&](int k) { return total >= ctas ? first + k : range_of(total, begin + k, ctas); };
  if (c != cta(1)) return;   // another block's
  const unsigned r0 = static_cast<unsigned>(s.z) * NT + n0;
  if (r0 >= static_cast<unsigned>(p.a.N) * p.G) return;
  int len, nn;
  const bool ok = kv_lengths(p.a, s.x, len, nn);
  float m[kRows], sum[kRows], acc[kRows][E];
#pragma unroll
  for (int q = 0; q < kRows; ++q) {
    m[q] = -INFINITY;
    sum[q] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[q][e] = 0.f;
  }
  for (int k0 = 0; k0 < parts; k0 += 32) {   // 32 parts at a time, a lane each for their weights
    const int k = k0 + lane;
    const long long part = k < parts ? (2LL * cta(k) + (k == 0 ? 1 : 0)) * NT + n0 : 0;
    float v[kRows], w[kRows];
#pragma unroll
    for (int q = 0; q < kRows; ++q) v[q] = k < parts ? __ldcg(p.part_lse + part + q) : -INFINITY;
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      float top = v[q];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmax_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
      top = fmax_nan(top, m[q]);
      const float ref = top == -INFINITY ? 0.f : top;
      w[q] = ex2(v[q] - ref);
      const float old = ex2(m[q] - ref);
      m[q] = top;
      float all = w[q];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
      sum[q] = sum[q] * old + all;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[q][e] *= old;
    }
    const int cnt = min(32, parts - k0);
#pragma unroll 2
    for (int j = 0; j < cnt; ++j) {
      const float *o = p.part_o + __shfl_sync(0xffffffffu, part, j) * D + lane * E;
#pragma unroll
      for (int q = 0; q < kRows; ++q) {
        const float wj = __shfl_sync(0xffffffffu, w[q], j);
        if constexpr (E == 4) {
          const float4 x = __ldcg(reinterpret_cast<const float4 *>(o + q * D));
          acc[q][0] = __fmaf_rn(wj, x.x, acc[q][0]);
          acc[q][1] = __fmaf_rn(wj, x.y, acc[q][1]);
          acc[q][2] = __fmaf_rn(wj, x.z, acc[q][2]);
          acc[q][3] = __fmaf_rn(wj, x.w, acc[q][3]);
        } else {
          const float2 x = __ldcg(reinterpret_cast<const float2 *>(o + q * D));
          acc[q][0] = __fmaf_rn(wj, x.x, acc[q][0]);
          acc[q][1] = __fmaf_rn(wj, x.y, acc[q][1]);
        }
      }
    }
  }
#pragma unroll
  for (int q = 0; q < kRows; ++q) {
    const unsigned r = r0 + q;
    const int i = static_cast<int>(r / p.G), g = static_cast<int>(r - static_cast<unsigned>(i) * p.G);
    if (i >= p.a.N) break;
    const bool none = (ok && i >= nn) || m[q] == -INFINITY;   // padding, or nothing seen
    const float f = 1.f / sum[q];
    const long long at = (static_cast<long long>(s.x) * p.a.N + i) * p.a.Hq +
                         static_cast<long long>(s.y) * p.G + g;
    T *o = static_cast<T *>(p.out) + at * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *reinterpret_cast<uint32_t *>(o + e) =
          none ? 0u : pack_pair(acc[q][e] * f, acc[q][e + 1] * f, T());
    if (p.lse && lane == 0) p.lse[at] = none ? -INFINITY : (m[q] + log2f(sum[q])) * kLn2;
  }
}

// ------------------------------------------------------------------ launch


inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 f = fn.load(std::memory_order_acquire);
  if (!f) {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                         cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !ptr)
      return nullptr;
    f = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    fn.store(f, std::memory_order_release);
  }
  return f;
}

// [rows, D] bytes, boxes of one page of one head
inline bool make_map(CUtensorMap *m, const void *base, long long rows, int D, int page, bool swizzle) {
  const auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(D)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(D), static_cast<cuuint32_t>(page)};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             !swizzle ? CU_TENSOR_MAP_SWIZZLE_NONE
                      : D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// `ctas` CTAs' parts of NT rows in the workspace, and the launch that joins them.
inline void plan_parts(AttnArgs &p, char *ws, int NT) {
  p.start = reinterpret_cast<int4 *>(ws);
  p.part_lse = reinterpret_cast<float *>(ws + 2 * kMaxCtas * sizeof(int4));
  p.part_o = p.part_lse + 2 * kMaxCtas * NT;
  const long long rows = static_cast<long long>(p.a.N) * p.G;
  p.RT = static_cast<int>((rows + NT - 1) / NT);
}
template <typename T, int D, int NT>
cudaError_t launch_join(const AttnArgs &p, int ctas, cudaStream_t stream) {
  if (ctas == 1) return cudaSuccess;
  constexpr int kBlocks = NT < kJoinBlockRows ? 1 : NT / kJoinBlockRows;
  return launch_kv(kv_attention_join<T, D, NT>, static_cast<long long>(ctas - 1) * kBlocks, 256, 0,
                   stream, p, ctas);
}
// raises a kernel's shared-memory limit once per device
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<bool> (&ready)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && ready[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) ready[dev].store(true, std::memory_order_release);
  return e;
}

}  // namespace attn

// the kernels for items of up to 32 query rows and of more (each with and without a window)
cudaError_t launch_attention_cols(attn::AttnArgs &p, int dtype, const CUtensorMap &mk,
                                  const CUtensorMap &mv, int ctas, char *ws, cudaStream_t stream);
cudaError_t launch_attention_rows(attn::AttnArgs &p, int dtype, const CUtensorMap &mk,
                                  const CUtensorMap &mv, int ctas, char *ws, cudaStream_t stream);
cudaError_t launch_window_cols(attn::AttnArgs &p, int dtype, const CUtensorMap &mk,
                               const CUtensorMap &mv, int ctas, char *ws, cudaStream_t stream);
cudaError_t launch_window_rows(attn::AttnArgs &p, int dtype, const CUtensorMap &mk,
                               const CUtensorMap &mv, int ctas, char *ws, cudaStream_t stream);

}  // namespace specv
