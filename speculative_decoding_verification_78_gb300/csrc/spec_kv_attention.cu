// spec_kv_attention.cu -- attention of the new tokens over the paged e4m3 cache, on the
// 5th-generation tensor cores.
//
// The mathematics. For the rows r = (token i, query head g) that share a key head, over the slots t
// that the row may see, with page scales ks, vs and e4m3 bytes kb, vb:
//   x[r,t] = scale log2(e) ks[t] (q[r] . kb[t]),   out[r] = sum_t 2^x vs[t] vb[t] / sum_t 2^x
// The value scale goes into the exponent: with y = x + log2 vs[t] and a reference m[r] (a running
// upper estimate of y), p = 2^(y - m) is what multiplies the bytes vb, and p / vs[t] what the
// denominator adds, so bytes of pages with unlike scales meet in one accumulator.
//
// Orientation. Tokens, of which there are always many, lie along the MMA's 128 rows, and the query
// rows (1 to 128 of them, padded to 16) along its columns: S^T = K Q^T, O^T = V^T P^T. Both cost
// tensor time in proportion to the query rows that exist. K's e4m3 bytes are an MMA operand as TMA
// lands them: Q is the sum of 2 (bf16) or 3 (fp16) e4m3 terms, whose products accumulate in the
// same fp32 accumulator (two terms hold bf16's 8 significant bits exactly down to 2^-9 of the
// row's power-of-two unit; three fp16's 11). P is fp16 (11 bits; e4m3 terms would flush weights
// below 2^-18 of the reference, which a long context of small weights adds up), so V's bytes are
// widened to fp16, exactly, on their way through the softmax threads.
//
// One thread of the softmax warps has one token of the tile and half of the columns. Weights are
// taken against m as it stands; only when some y exceeds m by 2^7 in a tile (one barrier with an
// OR, which the tile needs anyway) are the maxima reduced over the tokens, the accumulators
// rescaled and the tile taken again. m starts at -1e30, so a row's first visible token does that.
//
// Work is cut evenly whatever the lengths: the 128-token tiles of all (sequence, key head, row
// tile) items form one line, CTA c of G takes tiles [T c / G, T (c+1) / G). An item inside one
// CTA's range is written directly; the parts of one that crosses ranges go to the workspace (at
// most two per CTA), and a second kernel joins them in order, so results do not depend on timing.
#include <cudaTypedefs.h>

#include <atomic>

#include "spec_kv.cuh"
#include "spec_tc.cuh"

namespace specv {

namespace {

constexpr int kTile = 128;          // tokens
constexpr int kGroupWarps = 8;      // softmax warps of a tile
constexpr int kGroupThreads = 32 * kGroupWarps;
constexpr int kSoftThreads = 2 * kGroupThreads;
constexpr int kProducer = 2 * kGroupWarps, kMma = kProducer + 1;   // warps
constexpr int kAttnThreads = 32 * (kMma + 1);
constexpr int kMaxCtas = 304;       // workspace parts are sized for this many CTAs
constexpr float kBias = 8.f;        // a new reference puts the largest weight at 2^8 ...
constexpr float kTrigger = 15.f;    // ... and is taken when one exceeds 2^15 (fp16 ends at 2^16)
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
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// barrier 1 + group over a group's threads; true in all of them if `p` was in any
__device__ __forceinline__ bool group_any(int group, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %3, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(p)), "n"(kGroupThreads), "r"(1 + group)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void group_sync(int group) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kGroupThreads) : "memory");
}
__device__ __forceinline__ void soft_sync() {   // both groups
  asm volatile("bar.sync 3, %0;" ::"n"(kSoftThreads) : "memory");
}
// true in one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
// tc::mbar_wait whose usual case, a phase that has completed, costs no call
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity) {
  return tc::mbar_try(bar, parity) || tc::mbar_wait(bar, parity);
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

// ------------------------------------------------------------------ configuration

// T: query type; D: head dim; NT: columns (query rows of a tile); S: stages of K and V
template <typename T_, int D_, int NT_, int S_>
struct Cfg {
  using T = T_;
  static constexpr int D = D_, NT = NT_, S = S_;
  static constexpr int kTerms = __is_same(T, __half) ? 3 : 2;
  static constexpr int C = NT / 2;                       // columns of a softmax thread
  static constexpr int CH = 8;                           // columns read at a time
  static constexpr int EC = NT / 4;                      // columns of a thread in the epilogue
  static constexpr int ECH = EC < 16 ? EC : 16;
  static constexpr int kSideBytes = kTile * D;           // K or V of a stage
  static constexpr int kPSpan = NT >= 64 ? 128 : 2 * NT; // bytes of a row of P
  static constexpr int kPBlocks = NT > 64 ? NT / 64 : 1;
  static constexpr int kPBytes = kTile * kPSpan * kPBlocks;
  static constexpr int kVfBytes = kTile * D * 2;
  static constexpr int kQBytes = NT * D;                 // one term
  static constexpr int kOffV16 = S * 2 * kSideBytes;
  static constexpr int kOffP = kOffV16 + 2 * kVfBytes;
  static constexpr int kOffQ = kOffP + 2 * kPBytes;
  static constexpr int kOffSmall = kOffQ + kTerms * kQBytes;
  static constexpr uint32_t kTmem = 4 * NT;              // each group's S and O
};

struct __align__(16) Small {   // the small parts of shared memory; arrays of NT follow
  uint64_t full[4], empty[4], sfull[2], pfull[2], pfree[2], qfull, done;
  float ks[4][8], vs[4][8];
  uint8_t vnan[2][kTile];      // by group: the token's values hold NaN (see widen)
  uint32_t tmem;
  int b0, skip0;
  int warp_sum[kAttnThreads / 32];
};
template <class F> constexpr int smem_bytes() {   // + qs, nm of each group, tok
  return F::kOffSmall + static_cast<int>(sizeof(Small)) + 4 * F::NT * 4;
}

// ------------------------------------------------------------------ the line of tiles

struct Item {   // one (sequence, key head, row tile)
  int b, h, rt;
  int len, n;      // tokens before the new ones; new ones
  bool ok;         // lengths fit
  int end;         // first slot that no row sees
  int tiles;
};

template <int NT>
__device__ __forceinline__ int item_end(const AttnArgs &p, int len, int n, bool ok, int rt) {
  if (!ok || n == 0) return 0;
  if (p.RT == 1 || p.a.mask) return len + n;
  const long long first = static_cast<long long>(rt) * NT / p.G;
  if (first >= n) return 0;   // padding
  const long long last = (static_cast<long long>(rt) * NT + NT - 1) / p.G;
  return len + static_cast<int>(last + 1 < n ? last + 1 : n);
}
__device__ __forceinline__ int tiles_for(int end) { return end > kTile ? (end + kTile - 1) / kTile : 1; }

// tiles of one key head of sequence b
template <int NT>
__device__ __forceinline__ int head_tiles(const AttnArgs &p, int b) {
  int len, n;
  const bool ok = kv_lengths(p.a, b, len, n);
  int s = 0;
  for (int rt = 0; rt < p.RT; ++rt) s += tiles_for(item_end<NT>(p, len, n, ok, rt));
  return s;
}
template <int NT>
__device__ __forceinline__ void item_load(const AttnArgs &p, Item &x) {
  x.ok = kv_lengths(p.a, x.b, x.len, x.n);
  x.end = item_end<NT>(p, x.len, x.n, x.ok, x.rt);
  x.tiles = tiles_for(x.end);
}
template <int NT>
__device__ __forceinline__ void item_next(const AttnArgs &p, Item &x) {
  if (++x.rt == p.RT) {
    x.rt = 0;
    if (++x.h == p.a.Hkv) {
      x.h = 0;
      ++x.b;
    }
  }
  if (x.b < p.a.B) item_load<NT>(p, x);
}
__device__ __forceinline__ int range_start(long long T, int c, int G) {
  return static_cast<int>(T * c / G);
}

// The CTA's range [t0, t1) of the line and its first item; called by all threads. Thread t sums
// the sequences of its own contiguous share; the thread whose share holds t0 finds it there.
template <int NT>
__device__ void locate(const AttnArgs &p, Small &sm, int &t0, int &t1, Item &x, int &skip) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int share = (p.a.B + kAttnThreads - 1) / kAttnThreads;
  const int lo = min(p.a.B, tid * share), hi = min(p.a.B, lo + share);
  int mine = 0;
  for (int b = lo; b < hi; ++b) mine += head_tiles<NT>(p, b) * p.a.Hkv;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sm.warp_sum[warp] = incl;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kAttnThreads / 32; ++w) {
    if (w < warp) before += sm.warp_sum[w];
    total += sm.warp_sum[w];
  }
  t0 = range_start(total, blockIdx.x, gridDim.x);
  t1 = range_start(total, blockIdx.x + 1, gridDim.x);
  int at = before + incl - mine;
  if (t0 >= at && t0 < at + mine) {
    int b = lo;
    for (;; ++b) {
      const int n = head_tiles<NT>(p, b) * p.a.Hkv;
      if (t0 < at + n) break;
      at += n;
    }
    sm.b0 = b;
    sm.skip0 = t0 - at;
  }
  __syncthreads();
  if (t0 >= t1) return;
  x.b = sm.b0;
  x.rt = 0;
  skip = sm.skip0;
  const int per_head = head_tiles<NT>(p, x.b);
  x.h = skip / per_head;
  skip -= x.h * per_head;
  item_load<NT>(p, x);
  while (skip >= x.tiles) {
    skip -= x.tiles;
    ++x.rt;
    item_load<NT>(p, x);
  }
}

// ------------------------------------------------------------------ softmax threads

// Rows of the item's tile as e4m3 terms in shared memory (16 or 8 lanes a row), each in units of a
// power of two that puts its largest element in [2^7, 2^8); qs[n] undoes it. All softmax threads.
template <class F>
__device__ __forceinline__ void load_queries(const AttnArgs &p, const Item &x, uint8_t *sq,
                                             float *qs, float *nm, int *tok) {
  constexpr int kLanes = F::D / 8, kRows = kSoftThreads / kLanes;
  const int sub = threadIdx.x % kLanes, row0 = threadIdx.x / kLanes;
  using T = typename F::T;
#pragma unroll
  for (int n0 = 0; n0 < F::NT; n0 += kRows) {
    const int n = n0 + row0;
    if (n >= F::NT) break;   // whole warps: a warp's rows are 2 or 4
    const long long r = static_cast<long long>(x.rt) * F::NT + n;
    const int i = static_cast<int>(r / p.G), g = static_cast<int>(r - static_cast<long long>(i) * p.G);
    float f[8];
    if (i < x.n && x.ok) {
      const T *src = static_cast<const T *>(p.q) +
                     (static_cast<long long>(x.b) * p.a.N + i) * p.q_stride +
                     (static_cast<long long>(x.h) * p.G + g) * F::D + sub * 8;
      vec_to_floats<T>(__ldg(reinterpret_cast<const uint4 *>(src)), f);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = 0.f;
    }
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmax_nan(m, fabsf(f[e]));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    const int e = max(static_cast<int>(__float_as_uint(m) >> 23), 27);   // exponent, at least -100
    const float mul = __uint_as_float(static_cast<uint32_t>(127 + 127 + 7 - e) << 23);
    if (sub == 0) {
      qs[n] = m < INFINITY ? __uint_as_float(static_cast<uint32_t>(e - 7) << 23) : NAN;
      nm[n] = nm[F::NT + n] = kNoRef;
      tok[n] = min(i, p.a.N - 1);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] *= mul;
#pragma unroll
    for (int t = 0; t < F::kTerms; ++t) {
      const uint2 w = floats_to_e4m3(f, 1.f);
      *reinterpret_cast<uint2 *>(sq + t * F::kQBytes + swz<F::D>(n * F::D + sub * 8)) = w;
      if (t + 1 < F::kTerms) {
        float g8[8];
        e4m3_to_floats(w, g8);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] -= g8[k];   // exact
      }
    }
  }
}

// V's bytes of a tile, on their way to fp16: 16 bytes a lane and step, whole rows side by side.
template <class F> struct Widen {
  static constexpr int kLanes = F::D / 16;               // lanes of a token
  static constexpr int kRows = kGroupThreads / kLanes;   // tokens a step
  static constexpr int kSteps = kTile / kRows;
};
template <class F>
__device__ __forceinline__ void fetch_values(const uint8_t *sv, int gtid, int valid,
                                             uint4 (&w)[Widen<F>::kSteps]) {
#pragma unroll
  for (int u = 0; u < Widen<F>::kSteps; ++u) {
    const int t = u * Widen<F>::kRows + gtid / Widen<F>::kLanes;
    w[u] = *reinterpret_cast<const uint4 *>(sv + t * F::D + gtid % Widen<F>::kLanes * 16);
    if (t >= valid) w[u] = make_uint4(0, 0, 0, 0);
  }
}
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {   // bit 7 of each NaN byte
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}
// The values as fp16 rows of 64 dims (128 bytes, swizzled). NaN codes become zero and mark their
// token: the weights of the rows that see it then turn NaN instead (a NaN operand would reach the
// rows that do not). Returns whether there was one.
template <class F>
__device__ __forceinline__ bool widen(uint4 (&w)[Widen<F>::kSteps], uint8_t *out, int gtid,
                                      uint8_t *vnan) {
  const int c = gtid % Widen<F>::kLanes, row0 = gtid / Widen<F>::kLanes;
  uint32_t any = 0;
#pragma unroll
  for (int u = 0; u < Widen<F>::kSteps; ++u)
    any |= nan_codes(w[u].x) | nan_codes(w[u].y) | nan_codes(w[u].z) | nan_codes(w[u].w);
  if (any) {
#pragma unroll
    for (int u = 0; u < Widen<F>::kSteps; ++u) {
      const uint32_t hx = nan_codes(w[u].x), hy = nan_codes(w[u].y), hz = nan_codes(w[u].z),
                     hw = nan_codes(w[u].w);
      w[u].x &= ~((hx >> 7) * 255u);
      w[u].y &= ~((hy >> 7) * 255u);
      w[u].z &= ~((hz >> 7) * 255u);
      w[u].w &= ~((hw >> 7) * 255u);
      if (hx | hy | hz | hw) vnan[u * Widen<F>::kRows + row0] = 1;
    }
  }
  // 64 dims (4 lanes) a block of kTile rows; the second block's lanes store their halves the other
  // way round, so that eight neighbours never meet in a bank
  uint8_t *blk = out + (c >> 2) * (kTile * 128);
  const bool flip = (c >> 2) & 1;
#pragma unroll
  for (int u = 0; u < Widen<F>::kSteps; ++u) {
    const int t = u * Widen<F>::kRows + row0;
    const uint4 lo = make_uint4(e4m3_to_half2(w[u].x & 0xffffu), e4m3_to_half2(w[u].x >> 16),
                                e4m3_to_half2(w[u].y & 0xffffu), e4m3_to_half2(w[u].y >> 16));
    const uint4 hi = make_uint4(e4m3_to_half2(w[u].z & 0xffffu), e4m3_to_half2(w[u].z >> 16),
                                e4m3_to_half2(w[u].w & 0xffffu), e4m3_to_half2(w[u].w >> 16));
    const uint32_t a0 = swz<128>(t * 128 + (c & 3) * 32), a1 = swz<128>(t * 128 + (c & 3) * 32 + 16);
    *reinterpret_cast<uint4 *>(blk + (flip ? a1 : a0)) = flip ? hi : lo;
    *reinterpret_cast<uint4 *>(blk + (flip ? a0 : a1)) = flip ? lo : hi;
  }
  return any != 0;
}

// Sums (or maxima) over a warp's 32 lanes of C per-lane values, C a power of two up to 32: on
// return lane l holds the total of value l % C in v[0].
template <int C, bool kMax>
__device__ __forceinline__ float reduce_columns(float (&v)[C], int lane) {
#pragma unroll
  for (int w = C / 2; w >= 1; w >>= 1) {
    const bool up = lane & w;
#pragma unroll
    for (int k = 0; k < w; ++k) {
      const float give = up ? v[k] : v[k + w], keep = up ? v[k + w] : v[k];
      const float got = __shfl_xor_sync(0xffffffffu, give, w);
      v[k] = kMax ? fmaxf(keep, got) : keep + got;
    }
  }
#pragma unroll
  for (int o = C; o < 32; o <<= 1) {
    const float got = __shfl_xor_sync(0xffffffffu, v[0], o);
    v[0] = kMax ? fmaxf(v[0], got) : v[0] + got;
  }
  return v[0];
}

// What one softmax thread knows of its token in a tile
struct Token {
  float ks2;       // scale * log2(e) * key scale
  float lvs, ivs;  // log2 of the value scale, and one over it
  int from;        // columns from this one on see it (a mask: all that its bits allow)
  int j;           // number among the new tokens (mask), or -1
};

template <class F>
__device__ __forceinline__ bool sees(const AttnArgs &p, const Item &x, const Token &t, int n,
                                     const int *tok) {
  bool see = n >= t.from;
  if (t.j >= 0 && see)
    see = (__ldg(p.a.mask + (static_cast<long long>(x.b) * p.a.N + tok[n]) * p.a.W + (t.j >> 5)) >>
           (t.j & 31)) & 1u;
  return see;
}

// The weights of the tile against the reference as it stands: fp16 to P, their sums (over the value
// scale) added to l; true if one exceeds what fp16 holds comfortably. The scores of the next
// columns are on their way from tensor memory while these are worked on.
template <class F, bool kMasked>
__device__ __forceinline__ bool weigh(const AttnArgs &p, const Item &x, const Token &t, bool poison,
                                      uint32_t ts, int col0, uint8_t *sp, const float *qs,
                                      const float *nm, const int *tok, int row,
                                      f32x2 (&l)[F::C / 2]) {
  const f32x2 ks2 = pk2(t.ks2, t.ks2), lvs2 = pk2(t.lvs, t.lvs), ivs2 = pk2(t.ivs, t.ivs);
  float big = -INFINITY;
  uint32_t s[2][F::CH];
  tmem_ld(ts, s[0]);
#pragma unroll
  for (int c0 = 0; c0 < F::C; c0 += F::CH) {
    uint32_t(&v)[F::CH] = s[(c0 / F::CH) & 1];
    tmem_wait(v);
    if (c0 + F::CH < F::C) tmem_ld(ts + c0 + F::CH, s[(c0 / F::CH + 1) & 1]);
    uint32_t h[F::CH / 2];
#pragma unroll
    for (int c = 0; c < F::CH; c += 4) {
      const float4 q4 = *reinterpret_cast<const float4 *>(qs + col0 + c0 + c);
      const float4 m4 = *reinterpret_cast<const float4 *>(nm + col0 + c0 + c);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int k = c + 2 * u;
        const f32x2 q2 = u ? pk2(q4.z, q4.w) : pk2(q4.x, q4.y);
        const f32x2 m2 = u ? pk2(m4.z, m4.w) : pk2(m4.x, m4.y);
        const f32x2 sv = pk2(__uint_as_float(v[k]), __uint_as_float(v[k + 1]));
        float y0, y1;
        up2(fma2(mul2(sv, ks2), q2, add2(m2, lvs2)), y0, y1);
        if (kMasked) {
          const int n = col0 + c0 + k;
          if (poison) y0 = y1 = NAN;
          if (!sees<F>(p, x, t, n, tok)) y0 = -INFINITY;
          if (!sees<F>(p, x, t, n + 1, tok)) y1 = -INFINITY;
        }
        big = fmaxf(big, fmaxf(y0, y1));
        const float p0 = ex2(y0), p1 = ex2(y1);
        const int li = (c0 + k) / 2;
        l[li] = fma2(pk2(p0, p1), ivs2, l[li]);
        h[k / 2] = pack_pair(p0, p1, __half());
      }
    }
    const int n = col0 + c0;
    const uint32_t at = swz<F::kPSpan>(row * F::kPSpan + (n % (F::kPSpan / 2)) * 2);
    *reinterpret_cast<uint4 *>(sp + (n / (F::kPSpan / 2)) * (kTile * F::kPSpan) + at) =
        make_uint4(h[0], h[1], h[2], h[3]);
  }
  return big > kTrigger;
}

// Before a tile is taken again: the largest y of each of this thread's columns over the warp's 32
// tokens, to wmax[column], and what the first attempt added to l taken off again. (That leaves at
// most 2^-24 of the weight taken off, which stays in the new sum anyway; where it was infinite, the
// old sum is less than 2^-100 of the new one. A NaN stays.)
template <class F>
__device__ __forceinline__ void retract(const AttnArgs &p, const Item &x, const Token &t, uint32_t ts,
                                        int col0, const float *qs, const float *nm, const int *tok,
                                        int lane, float *wmax, f32x2 (&l)[F::C / 2]) {
#pragma unroll
  for (int c0 = 0; c0 < F::C; c0 += F::CH) {
    uint32_t s[F::CH];
    tmem_ld(ts + c0, s);
    tmem_wait(s);
    float y[F::CH];
#pragma unroll
    for (int c = 0; c < F::CH; ++c) {
      const int n = col0 + c0 + c;
      y[c] = __fmaf_rn(__uint_as_float(s[c]) * t.ks2, qs[n], t.lvs);
      if (!sees<F>(p, x, t, n, tok)) y[c] = -INFINITY;
    }
#pragma unroll
    for (int c = 0; c < F::CH; c += 2) {
      const int n = col0 + c0 + c;
      float l0, l1;
      up2(l[(c0 + c) / 2], l0, l1);
      l0 = l0 == INFINITY ? 0.f : l0 - ex2(y[c] + nm[n]) * t.ivs;
      l1 = l1 == INFINITY ? 0.f : l1 - ex2(y[c + 1] + nm[n + 1]) * t.ivs;
      l[(c0 + c) / 2] = pk2(l0, l1);
      if (y[c] != y[c]) y[c] = -INFINITY;
      if (y[c + 1] != y[c + 1]) y[c + 1] = -INFINITY;
    }
    const float m = reduce_columns<F::CH, true>(y, lane);
    if (lane < F::CH) wmax[col0 + c0 + lane] = m;
  }
}

template <class F>
__global__ void __launch_bounds__(kAttnThreads, 1)
    kv_attention_kernel(const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v,
                        const __grid_constant__ AttnArgs p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Small &sm = *reinterpret_cast<Small *>(smem + F::kOffSmall);
  float *qs = reinterpret_cast<float *>(smem + F::kOffSmall + sizeof(Small));
  float *nm = qs + F::NT;   // -m of each group
  int *tok = reinterpret_cast<int *>(nm + 2 * F::NT);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < F::S; ++s) {
      tc::mbar_init(&sm.full[s], 33);               // 32 lanes' scales and the byte count
      tc::mbar_init(&sm.empty[s], 1 + kGroupWarps); // the score MMAs; each warp of a group
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm.sfull[i], 1);
      tc::mbar_init(&sm.pfull[i], 1);
      tc::mbar_init(&sm.pfree[i], 1);
    }
    tc::mbar_init(&sm.qfull, 1);
    tc::mbar_init(&sm.done, 1);
    tc::mbar_fence_init();
  }
  if (tid < 2 * kTile) sm.vnan[tid / kTile][tid % kTile] = 0;
  if (warp == kMma) tmem_alloc(&sm.tmem, F::kTmem);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int t0 = 0, t1 = 0, skip = 0;
  Item x{};
  tc::fence_before_sync();
  locate<F::NT>(p, sm, t0, t1, x, skip);
  tc::fence_after_sync();
  const uint32_t tmem = sm.tmem;
  if (tid == 0 && t0 < t1) {
    p.start[blockIdx.x] = make_int4(x.b, x.h, x.rt, skip);
    p.start[gridDim.x + blockIdx.x] = make_int4(x.tiles, t0, t1, 0);
  } else if (tid == 0) {
    p.start[gridDim.x + blockIdx.x] = make_int4(0, t0, t1, 0);
  }
  bool ok = true;   // false after a wait gave up: no further waits, and no further work is issued
  if (warp == kProducer) {
    int it = 0;
    const int per_tile = kTile >> p.a.page_shift;
    for (int t = t0; t < t1 && ok;) {
      const int cnt = min(x.tiles - skip, t1 - t);
      // the page number of this lane's page in tile k of the segment (0 past the end)
      const int32_t *table = p.a.page_table + static_cast<long long>(x.b) * p.a.pps;
      auto page_of = [&](int k) {
        const int slot = (skip + k) * kTile + (lane << p.a.page_shift);
        return lane < per_tile && slot < x.end ? __ldg(table + (slot >> p.a.page_shift)) : 0;
      };
      int next = page_of(0);
      for (int k = 0; k < cnt && ok; ++k, ++it) {
        const int s = it % F::S;
        const int slot = (skip + k) * kTile + (lane << p.a.page_shift);
        const bool want = lane < per_tile && slot < x.end;
        const int page = next;
        if (k + 1 < cnt) next = page_of(k + 1);   // on its way while this tile waits for room
        const bool good = want && page >= 0 && page < p.a.num_pages;
        if (want && !good) set_status(p.a.status, SPEC_ERR_PAGE);
        const uint32_t goods = __ballot_sync(0xffffffffu, good);
        ok = wait_for(&sm.empty[s], ((it / F::S) & 1) ^ 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0)
          tc::mbar_expect_tx(&sm.full[s], __popc(goods) * 2 * (F::D << p.a.page_shift));
        __syncwarp();
        if (good) {
          const int head = page * p.a.Hkv + x.h;
          const int row = head << p.a.page_shift;
          const uint32_t dst = tc::saddr(smem + s * 2 * F::kSideBytes) +
                               (lane << p.a.page_shift) * F::D;
          tma_load_2d(dst, &map_k, 0, row, &sm.full[s]);
          tma_load_2d(dst + F::kSideBytes, &map_v, 0, row, &sm.full[s]);
          copy4(&sm.ks[s][lane], p.a.k_scale + head);
          copy4(&sm.vs[s][lane], p.a.v_scale + head);
          mbar_arrive_copies(&sm.full[s]);
        } else {
          if (want) sm.ks[s][lane] = sm.vs[s][lane] = NAN;   // what reads the page is NaN
          mbar_arrive(&sm.full[s]);
        }
      }
      t += cnt;
      skip = 0;
      if (t < t1) item_next<F::NT>(p, x);
    }
    // the last copies of each stage land before the CTA may end
    for (int k = max(0, it - F::S); k < it; ++k)
      if (!tc::mbar_wait(&sm.full[k % F::S], (k / F::S) & 1)) ok = false;
  } else if (warp == kMma) {
    // The whole warp walks the tiles and one elected lane issues: inside a branch of one lane the
    // descriptors are not known to be uniform, and issuing a tile's 16 MMAs took 1400 clocks.
    constexpr uint32_t id_s = attn_idesc(kTile, F::NT, false), id_o = attn_idesc(128, F::NT, true);
    const uint32_t base = tc::saddr(smem);
    auto scores = [&](int it) {
      const uint64_t da = smem_desc<F::D>(base + (it % F::S) * 2 * F::kSideBytes, 16, 8 * F::D);
      const uint64_t db = smem_desc<F::D>(base + F::kOffQ, 16, 8 * F::D);
      const uint32_t d = tmem + (it & 1) * F::NT;   // the group's scores
      if (elect_one()) {
#pragma unroll
        for (int term = 0; term < F::kTerms; ++term)
#pragma unroll
          for (int kk = 0; kk < F::D / 32; ++kk)   // 32 dims of e4m3: 32 bytes on
            mma_f8(d, da + 2 * kk, db + term * (F::kQBytes / 16) + 2 * kk, id_s,
                   (term | kk) != 0);
        mma_commit(&sm.empty[it % F::S]);
        mma_commit(&sm.sfull[it & 1]);
      }
      __syncwarp();
    };
    auto values = [&](int it, bool first) {
      const int grp = it & 1;
      // one block of 64 dims (D = 64) stands for both halves of the MMA's rows
      const uint64_t da = smem_desc<128>(base + F::kOffV16 + grp * F::kVfBytes,
                                         F::D > 64 ? kTile * 128 : 0, 1024);
      const uint64_t db = smem_desc<F::kPSpan>(base + F::kOffP + grp * F::kPBytes,
                                               kTile * F::kPSpan, 8 * F::kPSpan);
      const uint32_t d = tmem + (2 + grp) * F::NT;
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)   // 16 tokens
          mma_f16(d, da + kk * (16 * 128 / 16), db + kk * F::kPSpan, id_o, !(first && kk == 0));
        mma_commit(&sm.pfree[grp]);
      }
      __syncwarp();
    };
    int it = 0, seg = 0;
    bool pending = false, pending_first = false;
    auto wait = [&](uint64_t *bar, int parity) {
      ok = ok && wait_for(bar, parity);
      ok = __all_sync(0xffffffffu, ok);
      tc::fence_after_sync();
    };
    auto drain = [&]() {   // the value MMAs of the tile before
      if (!pending) return;
      wait(&sm.pfull[(it - 1) & 1], ((it - 1) >> 1) & 1);
      if (!ok) return;
      values(it - 1, pending_first);
      pending = false;
    };
    for (int t = t0; t < t1 && ok; ++seg) {
      const int cnt = min(x.tiles - skip, t1 - t);
      drain();
      wait(&sm.qfull, seg & 1);
      for (int k = 0; k < cnt && ok; ++k) {
        wait(&sm.full[it % F::S], (it / F::S) & 1);
        if (!ok) break;
        scores(it);
        drain();
        if (!ok) break;
        pending = true;
        pending_first = k < 2;   // each group's first tile of the segment
        ++it;
      }
      t += cnt;
      skip = 0;
      if (t < t1) item_next<F::NT>(p, x);
    }
    if (ok) drain();
    if (elect_one()) mma_commit(&sm.done);   // every MMA issued has completed before the CTA may end
    if (!wait_for(&sm.done, 0)) ok = false;
    __syncwarp();
  } else {
    const int grp = warp / kGroupWarps, gtid = tid % kGroupThreads;
    const int quad = warp & 3;
    const int col0 = (warp >> 2 & 1) * F::C;
    const int row = quad * 32 + lane;   // token of the tile; in the epilogue the dim
    const uint32_t tlane = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t ts = tlane + grp * F::NT + col0;         // this thread's scores
    const uint32_t to = tlane + (2 + grp) * F::NT + col0;   // its group's accumulators
    uint8_t *sv16 = smem + F::kOffV16 + grp * F::kVfBytes;
    uint8_t *sp = smem + F::kOffP + grp * F::kPBytes;
    float *gnm = nm + grp * F::NT;
    uint8_t *vnan = sm.vnan[grp];
    int it = 0;   // tiles of the range so far; the groups take them in turn
    auto wait = [&](uint64_t *bar, int parity) {
      ok = ok && wait_for(bar, parity);
      __syncwarp();
    };
    for (int t = t0; t < t1;) {
      const int cnt = min(x.tiles - skip, t1 - t);
      load_queries<F>(p, x, smem + F::kOffQ, qs, nm, tok);
      fence_async();
      soft_sync();
      if (tid == 0) mbar_arrive(&sm.qfull);
      f32x2 l[F::C / 2];
#pragma unroll
      for (int c = 0; c < F::C / 2; ++c) l[c] = pk2(0.f, 0.f);
      for (int k = (it ^ grp) & 1; k < cnt; k += 2) {
        const int n = it + k, s = n % F::S, use = n >> 1;
        const int slot0 = (skip + k) * kTile;
        wait(&sm.full[s], (n / F::S) & 1);
        uint4 w[Widen<F>::kSteps];
        fetch_values<F>(smem + s * 2 * F::kSideBytes + F::kSideBytes, gtid, x.end - slot0, w);
        const float ks = sm.ks[s][row >> p.a.page_shift], vs = sm.vs[s][row >> p.a.page_shift];
        wait(&sm.pfree[grp], (use & 1) ^ 1);
        const bool nan = widen<F>(w, sv16, gtid, vnan);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.empty[s]);
        // a NaN scale (a bad page) makes the scores of its tokens NaN through lvs, and only those:
        // ivs multiplies the zero weights of rows that do not see them too, so it stays finite
        Token tk;
        const float vse = vs < kMinValueScale ? kMinValueScale : vs;
        tk.ks2 = ks * p.scale2;
        tk.lvs = __log2f(vse);
        tk.ivs = vs == vs ? __frcp_rn(vse) : 1.f;
        const int j = slot0 + row - x.len;
        tk.j = -1;
        tk.from = 0;
        if (slot0 + row >= x.end) {   // no scale was copied for a page past the end
          tk.from = F::NT;
          tk.ks2 = tk.lvs = tk.ivs = 0.f;
        } else if (j >= 0 && p.a.mask)
          tk.j = j;
        else if (j >= 0)
          tk.from = static_cast<int>(
              min(static_cast<long long>(F::NT),
                  static_cast<long long>(j) * p.G - static_cast<long long>(x.rt) * F::NT));
        const bool masked = slot0 + kTile > min(x.len, x.end);
        wait(&sm.sfull[grp], use & 1);
        tc::fence_after_sync();
        bool again = false;
#pragma unroll 1
        for (;;) {
          bool over;
          if (masked || again)
            over = weigh<F, true>(p, x, tk, again && vnan[row], ts, col0, sp, qs, gnm, tok, row, l);
          else
            over = weigh<F, false>(p, x, tk, false, ts, col0, sp, qs, gnm, tok, row, l);
          fence_async();
          tc::fence_before_sync();
          if (!group_any(grp, !again && (over || nan))) break;
          tc::fence_after_sync();
          // new references: maxima over the tile's tokens (P's buffer holds them meanwhile)
          float *wmax = reinterpret_cast<float *>(sp), *fac = wmax + 4 * F::NT;
          retract<F>(p, x, tk, ts, col0, qs, gnm, tok, lane, wmax + quad * F::NT, l);
          group_sync(grp);
          if (gtid < F::NT) {
            const float m = fmaxf(fmaxf(wmax[gtid], wmax[F::NT + gtid]),
                                  fmaxf(wmax[2 * F::NT + gtid], wmax[3 * F::NT + gtid]));
            const float old = gnm[gtid];
            const bool grow = m + old > kTrigger;
            const float now = grow ? kBias - m : old;
            fac[gtid] = grow ? ex2(now - old) : 1.f;   // 2^(m_old - m_new)
            gnm[gtid] = now;
          }
          group_sync(grp);
          // (the group's last value MMAs completed before its buffers were written)
#pragma unroll
          for (int c0 = 0; c0 < F::C; c0 += F::CH) {
            float f[F::CH];
#pragma unroll
            for (int c = 0; c < F::CH; ++c) f[c] = fac[col0 + c0 + c];
            if (k > 1) {
              uint32_t o[F::CH];
              tmem_ld(to + c0, o);
              tmem_wait(o);
#pragma unroll
              for (int c = 0; c < F::CH; ++c)
                o[c] = __float_as_uint(__uint_as_float(o[c]) * f[c]);
              tmem_st(to + c0, o);
            }
#pragma unroll
            for (int c = 0; c < F::CH; c += 2)
              l[(c0 + c) / 2] = mul2(l[(c0 + c) / 2], pk2(f[c], f[c + 1]));
          }
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          group_sync(grp);   // fac is read before P overwrites it
          again = true;
        }
        if (again) {
          group_sync(grp);
          if (gtid < kTile) vnan[gtid] = 0;
          group_sync(grp);   // the next tile's marks come after
        }
        if (gtid == 0) mbar_arrive(&sm.pfull[grp]);
      }
      it += cnt;
      // The item's (or its part's) result. All value MMAs have completed: each group's denominators
      // over the tile's 128 lanes, then the groups joined, each lane's dim of every column.
      for (int last = it - 1; last >= 0 && last >= it - 2; --last)
        wait(&sm.pfree[last & 1], (last >> 1) & 1);
      tc::fence_after_sync();
      float *lsum = reinterpret_cast<float *>(smem + F::kOffP), *fac = lsum + 8 * F::NT;
      soft_sync();
#pragma unroll
      for (int c0 = 0; c0 < F::C; c0 += F::CH) {
        float v[F::CH];
#pragma unroll
        for (int c = 0; c < F::CH; c += 2) up2(l[(c0 + c) / 2], v[c], v[c + 1]);
        const float sum = reduce_columns<F::CH, false>(v, lane);
        if (lane < F::CH) lsum[(grp * 4 + quad) * F::NT + col0 + c0 + lane] = sum;
      }
      soft_sync();
      const bool whole = skip == 0 && cnt == x.tiles;
      const long long part = 2LL * blockIdx.x + (skip == 0 ? 1 : 0);
      if (tid < F::NT) {
        float sum[2], wt[2];
        const float m = fminf(nm[tid], nm[F::NT + tid]);   // -m of the larger reference
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const float *v = lsum + 4 * g * F::NT + tid;
          sum[g] = (v[0] + v[F::NT]) + (v[2 * F::NT] + v[3 * F::NT]);
          wt[g] = ex2(m - nm[g * F::NT + tid]);   // 0 for a group that saw nothing, beside one that did
        }
        const float total = sum[0] * wt[0] + sum[1] * wt[1];
        const long long r = static_cast<long long>(x.rt) * F::NT + tid;
        const int i = static_cast<int>(r / p.G), g = static_cast<int>(r - static_cast<long long>(i) * p.G);
        float lse2 = total == 0.f ? -INFINITY : log2f(total) - m;
        float f = total == 0.f ? 0.f : 1.f / total;
        if (!x.ok) {
          lse2 = f = NAN;
        } else if (whole && i >= x.n) {   // padding
          f = 0.f;
          lse2 = -INFINITY;
        }
        fac[tid] = sum[0] == 0.f ? 0.f * f : wt[0] * f;   // (0 NaN is NaN)
        fac[F::NT + tid] = sum[1] == 0.f ? 0.f * f : wt[1] * f;
        if (!whole)
          p.part_lse[part * F::NT + tid] = lse2;
        else if (p.lse && i < p.a.N)
          p.lse[(static_cast<long long>(x.b) * p.a.N + i) * p.a.Hq + static_cast<long long>(x.h) * p.G + g] =
              lse2 * kLn2;
      }
      soft_sync();
      using T = typename F::T;
      const int e0 = (warp >> 2) * F::EC;
#pragma unroll 1
      for (int c0 = e0; c0 < e0 + F::EC; c0 += F::ECH) {
        uint32_t o[F::ECH], o1[F::ECH];
        tmem_ld(tlane + 2 * F::NT + c0, o);
        tmem_ld(tlane + 3 * F::NT + c0, o1);
        tmem_wait(o);
        tmem_wait(o1);
        if (row < F::D) {
#pragma unroll
          for (int c = 0; c < F::ECH; ++c) {
            const int n = c0 + c;
            // a group that saw nothing counts 0 whatever its accumulator holds
            const float f0 = fac[n], f1 = fac[F::NT + n];
            const float v = (f0 == 0.f ? 0.f : __uint_as_float(o[c]) * f0) +
                            (f1 == 0.f ? 0.f : __uint_as_float(o1[c]) * f1);
            if (!whole) {
              p.part_o[(part * F::NT + n) * F::D + row] = v;
            } else {
              const long long r = static_cast<long long>(x.rt) * F::NT + n;
              const int i = tok[n];
              const long long g = r - static_cast<long long>(i) * p.G;
              if (g < p.G)
                static_cast<T *>(p.out)[((static_cast<long long>(x.b) * p.a.N + i) * p.a.Hq +
                                         static_cast<long long>(x.h) * p.G + g) * F::D + row] =
                    static_cast<T>(v);
            }
          }
        }
      }
      if (!x.ok && tid == 0) set_status(p.a.status, SPEC_ERR_LENGTH);
      tc::fence_before_sync();
      soft_sync();   // lsum, fac and tok are read before the next item's writes
      t += cnt;
      skip = 0;
      if (t < t1) item_next<F::NT>(p, x);
    }
  }
  if (!ok) set_status(p.a.status, SPEC_ERR_TIMEOUT);
  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMma) {
    tc::fence_after_sync();
    tmem_free(tmem, F::kTmem);
  }
}

// Joins the parts of the items that cross ranges. Block (c, rows): the item that range c begins
// inside of, if c is the first range to do so; one warp per row.
template <class F>
__global__ void __launch_bounds__(256) kv_attention_join(const __grid_constant__ AttnArgs p,
                                                         int ctas) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kBlocks = F::NT / 8;
  const int c = 1 + blockIdx.x / kBlocks;
  const int n = (blockIdx.x % kBlocks) * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  // (written by other CTAs: read from L2)
  auto empty = [&](int at) {
    const int4 e = __ldcg(p.start + at);
    return e.y >= e.z;
  };
  const int4 d = __ldcg(p.start + ctas + c);           // tiles of its first item, t0, t1
  if (d.y >= d.z) return;
  const int4 s = __ldcg(p.start + c);
  const int begin = d.y - s.w, end = begin + d.x;   // the item's tiles on the line
  if (s.w == 0) return;
  // the range with the tile before: the item's first part, or another block's item
  int first = c - 1;   // (ranges may be empty when there are few tiles)
  while (empty(ctas + first)) --first;
  if (begin < __ldcg(p.start + ctas + first).y) return;
  const long long r = static_cast<long long>(s.z) * F::NT + n;
  const int i = static_cast<int>(r / p.G), g = static_cast<int>(r - static_cast<long long>(i) * p.G);
  if (i >= p.a.N) return;
  float m = -INFINITY;
  for (int k = first; k < ctas; ++k) {
    const int4 e = __ldcg(p.start + ctas + k);
    if (e.y >= end) break;
    if (e.y >= e.z) continue;
    m = fmax_nan(m, __ldcg(p.part_lse + (2LL * k + (k == first ? 1 : 0)) * F::NT + n));
  }
  constexpr int E = F::D / 32;
  float acc[E], sum = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  if (m != -INFINITY)
    for (int k = first; k < ctas; ++k) {
      const int4 e = __ldcg(p.start + ctas + k);
      if (e.y >= end) break;
      if (e.y >= e.z) continue;
      const long long part = (2LL * k + (k == first ? 1 : 0)) * F::NT + n;
      const float w = ex2(__ldcg(p.part_lse + part) - m);
      sum += w;
      const float *o = p.part_o + part * F::D + lane * E;
#pragma unroll
      for (int q = 0; q < E; ++q) acc[q] = __fmaf_rn(w, __ldcg(o + q), acc[q]);
    }
  int len, nn;
  const bool ok = kv_lengths(p.a, s.x, len, nn);
  const bool pad = ok && i >= nn;
  const float f = pad || m == -INFINITY ? 0.f : 1.f / sum;
  using T = typename F::T;
  const long long at = (static_cast<long long>(s.x) * p.a.N + i) * p.a.Hq +
                       static_cast<long long>(s.y) * p.G + g;
  T *o = static_cast<T *>(p.out) + at * F::D + lane * E;
#pragma unroll
  for (int q = 0; q < E; q += 2)
    *reinterpret_cast<uint32_t *>(o + q) =
        pad ? 0u : pack_pair(acc[q] * f, acc[q + 1] * f, T());
  if (p.lse && lane == 0)
    p.lse[at] = pad || m == -INFINITY ? -INFINITY : (m + log2f(sum)) * kLn2;
}

// ------------------------------------------------------------------ launch

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
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
bool make_map(CUtensorMap *m, const void *base, long long rows, int D, int page, bool swizzle) {
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

// Columns of a tile: the query rows of a key head when one tile holds them, else 128 (fp16 queries,
// whose third term takes the room, 64).
int tile_columns(int dtype, long long rows) {
  if (rows <= 16) return 16;
  if (rows <= 32) return 32;
  return rows <= 64 || dtype == SPEC_F16 ? 64 : 128;
}

template <class F>
cudaError_t launch_cfg(AttnArgs &p, const CUtensorMap &mk, const CUtensorMap &mv, int sms,
                       char *ws, cudaStream_t stream) {
  static std::atomic<bool> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  constexpr int smem = smem_bytes<F>();
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  if (dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kv_attention_kernel<F>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev].store(true, std::memory_order_release);
  }
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  p.start = reinterpret_cast<int4 *>(ws);
  p.part_lse = reinterpret_cast<float *>(ws + 2 * kMaxCtas * sizeof(int4));
  p.part_o = p.part_lse + 2 * kMaxCtas * F::NT;
  const long long rows = static_cast<long long>(p.a.N) * p.G;
  p.RT = static_cast<int>((rows + F::NT - 1) / F::NT);
  // a plain stream-ordered launch: nearly all of an SM's shared memory is one CTA's
  kv_attention_kernel<F><<<ctas, kAttnThreads, smem, stream>>>(mk, mv, p);
  e = cudaGetLastError();
  if (e != cudaSuccess || ctas == 1) return e;
  return launch_kv(kv_attention_join<F>, static_cast<long long>(ctas - 1) * (F::NT / 8), 256, 0,
                   stream, p, ctas);
}

template <typename T, int D>
cudaError_t launch_columns(int nt, AttnArgs &p, const CUtensorMap &mk, const CUtensorMap &mv,
                           int sms, char *ws, cudaStream_t stream) {
  if (nt == 16) return launch_cfg<Cfg<T, D, 16, 4>>(p, mk, mv, sms, ws, stream);
  if (nt == 32) return launch_cfg<Cfg<T, D, 32, 4>>(p, mk, mv, sms, ws, stream);
  if constexpr (!__is_same(T, __half))
    if (nt == 128) return launch_cfg<Cfg<T, D, 128, 2>>(p, mk, mv, sms, ws, stream);
  return launch_cfg<Cfg<T, D, 64, 3>>(p, mk, mv, sms, ws, stream);
}

}  // namespace

size_t kv_attention_workspace(int B, int N, int Hq, int Hkv, int D) {
  const long long rows = static_cast<long long>(N) * (Hq / Hkv);
  const size_t nt = tile_columns(SPEC_BF16, rows);   // the wider of the types
  return 2 * kMaxCtas * (sizeof(int4) + nt * sizeof(float) * (1 + D));
}

cudaError_t launch_kv_attention(const KvArgs &a, const void *q, long long q_stride, int dtype,
                                float scale, void *out, float *lse, void *ws,
                                cudaStream_t stream) {
  static std::atomic<int> sm_counts[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int sms = dev < 64 ? sm_counts[dev].load(std::memory_order_acquire) : 0;
  if (sms <= 0) {
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (dev < 64) sm_counts[dev].store(sms, std::memory_order_release);
  }
  CUtensorMap mk, mv;
  const long long rows = (static_cast<long long>(a.num_pages) * a.Hkv) << a.page_shift;
  if (!make_map(&mk, a.k, rows, a.D, a.page, true) || !make_map(&mv, a.v, rows, a.D, a.page, false))
    return cudaErrorInvalidValue;
  AttnArgs p{};
  p.a = a;
  p.q = q;
  p.q_stride = q_stride;
  p.scale2 = scale * kLog2e;
  p.out = out;
  p.lse = lse;
  p.G = a.Hq / a.Hkv;
  const int nt = tile_columns(dtype, static_cast<long long>(a.N) * p.G);
  char *w = static_cast<char *>(ws);
  if (dtype == SPEC_BF16)
    return a.D == 64 ? launch_columns<__nv_bfloat16, 64>(nt, p, mk, mv, sms, w, stream)
                     : launch_columns<__nv_bfloat16, 128>(nt, p, mk, mv, sms, w, stream);
  return a.D == 64 ? launch_columns<__half, 64>(nt, p, mk, mv, sms, w, stream)
                   : launch_columns<__half, 128>(nt, p, mk, mv, sms, w, stream);
}

}  // namespace specv
