// spec_kv_attention.cu -- attention of few query rows (up to 32 for a key head: single tokens, short
// chains) over the paged e4m3 cache, on the 5th-generation tensor cores; and the choice of kernel.
//
// The mathematics. For the rows r = (token i, query head g) that share a key head, over the slots t
// that the row may see, with page scales ks, vs and e4m3 bytes kb, vb:
//   x[r,t] = scale log2(e) ks[t] (q[r] . kb[t]),   out[r] = sum_t 2^x vs[t] vb[t] / sum_t 2^x
// The value scale goes into the exponent: with y = x + log2 vs[t] and a reference m[r] (a running
// upper estimate of y), p = 2^(y - m) is what multiplies the bytes vb, and p / vs[t] what the
// denominator adds, so bytes of pages with unlike scales meet in one accumulator.
//
// Orientation. Tokens, of which there are always many, lie along the MMA's 128 rows, and the query
// rows (1 to 32 of them, padded to 16) along its columns: S^T = K Q^T, O^T = V^T P^T. Both cost
// tensor time in proportion to the query rows that exist. K's e4m3 bytes are an MMA operand as TMA
// lands them: Q is the sum of 2 (bf16) or 3 (fp16) e4m3 terms, whose products accumulate in the
// same fp32 accumulator (two terms hold bf16's 8 significant bits exactly down to 2^-9 of the
// row's largest element, three fp16's 11 down to 2^-6; smaller elements are off by at most 2^-17
// of the largest). P is fp16 (11 bits; e4m3 terms would flush weights
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
//
// What bounds it: HBM, which it does not quite fill. 64 sequences of about 15000 tokens, one new token,
// 32 query and 8 key heads of 128: 322 us for 1.95 GB, 6.05 TB/s (90 % of the measured copy rate). A
// tile's chain (wait, widen, scores, weights, barrier) takes a group about 3600 clocks, which two groups
// in turn hide but for a tenth; issuing the 16 MMAs takes their own warp 950 of a tile's 1650. With one
// group 607 us; with the MMAs issued from a branch of one lane, where their descriptors are not known to
// be uniform, 503 us. Tried and not kept: the query terms as columns side by side (8 MMAs fewer, the terms
// added by the softmax: 362 against 333 us), the page constants worked out by the copying warp (407), scores
// two tiles ahead of the values with the weights before the widening (390: a stage is held longer than
// four of them last), waits without a vote, as the kernel for many rows has them (354: more spills). At 96
// registers, what 18 warps leave, all forms but that of 16 columns and 64 dims spill 40 to 44 bytes.
#include "spec_kv_attn.h"

namespace specv {

using namespace attn;

namespace {

constexpr int kGroupWarps = 8;      // softmax warps of a tile
constexpr int kGroupThreads = 32 * kGroupWarps;
constexpr int kSoftThreads = 2 * kGroupThreads;
constexpr int kProducer = 2 * kGroupWarps, kMma = kProducer + 1;   // warps
constexpr int kAttnThreads = 32 * (kMma + 1);
constexpr float kBias = 8.f;        // a new reference puts the largest weight at 2^8 ...
constexpr float kTrigger = 15.f;    // ... and is taken when one exceeds 2^15 (fp16 ends at 2^16)

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
  static constexpr int kPSpan = 2 * NT;                  // bytes of a row of P
  static constexpr int kPBytes = kTile * kPSpan;
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
  uint8_t vnan[2][kTile];      // by group: the token's values hold NaN (see scrub_values)
  uint32_t tmem;
  LocateScratch loc;
};
template <class F> constexpr int smem_bytes() {   // + qs, nm of each group, tok
  return F::kOffSmall + static_cast<int>(sizeof(Small)) + 4 * F::NT * 4;
}

// ------------------------------------------------------------------ softmax threads

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
    *reinterpret_cast<uint4 *>(sp + swz<F::kPSpan>(row * F::kPSpan + n * 2)) =
        make_uint4(h[0], h[1], h[2], h[3]);
  }
  return big > kTrigger;
}

// Before a tile is taken again: the largest y of each of this thread's columns over the warp's 32
// tokens, to wmax[column], and what the first attempt added to l, by the same expression, taken off
// again. (That leaves at most half a unit of the sum, which the new sum is not smaller than. Where the sum
// was infinite the old one is dropped: with value scales within 2^80 of each other each weight in it is
// below 2^-32 of the new one's, for y passed m by 128, or by 48 and more where 1 / vs is what passed the
// range. A NaN stays.)
template <class F>
__device__ __forceinline__ void retract(const AttnArgs &p, const Item &x, const Token &t, uint32_t ts,
                                        int col0, const float *qs, const float *nm, const int *tok,
                                        int lane, float *wmax, f32x2 (&l)[F::C / 2]) {
#pragma unroll
  for (int c0 = 0; c0 < F::C; c0 += F::CH) {
    uint32_t s[F::CH];
    tmem_ld(ts + c0, s);
    tmem_wait(s);
    float y[F::CH];   // without the reference
    float w[F::CH];   // as the first attempt weighed it
#pragma unroll
    for (int c = 0; c < F::CH; ++c) {
      const int n = col0 + c0 + c;
      const float z = __uint_as_float(s[c]) * t.ks2;
      y[c] = __fmaf_rn(z, qs[n], t.lvs);
      w[c] = ex2(__fmaf_rn(z, qs[n], __fadd_rn(nm[n], t.lvs)));
      if (!sees<F>(p, x, t, n, tok)) {
        y[c] = -INFINITY;
        w[c] = 0.f;
      }
    }
#pragma unroll
    for (int c = 0; c < F::CH; c += 2) {
      float l0, l1;
      up2(l[(c0 + c) / 2], l0, l1);
      l0 = l0 == INFINITY ? 0.f : __fmaf_rn(-w[c], t.ivs, l0);
      l1 = l1 == INFINITY ? 0.f : __fmaf_rn(-w[c + 1], t.ivs, l1);
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
  int t0 = 0, t1 = 0, total = 0, skip = 0;
  Item x{};
  tc::fence_before_sync();
  locate<F::NT, kAttnThreads>(p, sm.loc, t0, t1, total, x, skip);
  tc::fence_after_sync();
  const uint32_t tmem = sm.tmem;
  if (tid == 0) publish_range(p, x, skip, t0, t1, total);
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
      if (!wait_for(&sm.full[k % F::S], (k / F::S) & 1)) ok = false;
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
                                               16, 8 * F::kPSpan);
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
      load_queries<typename F::T, F::D, F::NT, F::NT, F::kTerms, kSoftThreads>(
          p, x, RowMap::of<F::NT>(p, x.rt), F::NT, tid, smem + F::kOffQ, qs);
      if (tid < F::NT) {
        nm[tid] = nm[F::NT + tid] = kNoRef;
        const long long i = (static_cast<long long>(x.rt) * F::NT + tid) / p.G;
        tok[tid] = static_cast<int>(min(i, static_cast<long long>(p.a.N - 1)));
      }
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
        uint4 w[Widen<F::D, kGroupThreads>::kSteps];
        fetch_values<F::D, kGroupThreads>(smem + s * 2 * F::kSideBytes + F::kSideBytes, gtid, x.end - slot0, w);
        const float ks = sm.ks[s][row >> p.a.page_shift], vs = sm.vs[s][row >> p.a.page_shift];
        wait(&sm.pfree[grp], (use & 1) ^ 1);
        const bool masked = slot0 + kTile > min(x.len, x.end);
        const bool nan = masked && scrub_values<F::D, kGroupThreads>(
                                       w, gtid, [&](int at) { vnan[at] = 1; });
        widen<F::D, kGroupThreads>(w, sv16, gtid);
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
            if (!SPEC_CHECK(p.a, n < F::NT && part < 2LL * gridDim.x && x.b < p.a.B)) continue;
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

// ------------------------------------------------------------------ launch

template <class F>
cudaError_t launch_cfg(AttnArgs &p, const CUtensorMap &mk, const CUtensorMap &mv, int ctas, char *ws,
                       cudaStream_t stream) {
  static std::atomic<bool> ready[64];
  constexpr int smem = smem_bytes<F>();
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  cudaError_t e = allow_smem(kv_attention_kernel<F>, smem, ready);
  if (e != cudaSuccess) return e;
  plan_parts(p, ws, F::NT);
  // In plain stream order, so the kernel waits for nothing itself; it lets its join be scheduled early.
  // (Not measured: a launch as a programmatic dependent, whose set-up would run under the kernel before.)
  kv_attention_kernel<F><<<ctas, kAttnThreads, smem, stream>>>(mk, mv, p);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_join<typename F::T, F::D, F::NT>(p, ctas, stream);
}

template <typename T, int D>
cudaError_t launch_columns(bool wide, AttnArgs &p, const CUtensorMap &mk, const CUtensorMap &mv,
                           int ctas, char *ws, cudaStream_t stream) {
  return wide ? launch_cfg<Cfg<T, D, 32, 4>>(p, mk, mv, ctas, ws, stream)
              : launch_cfg<Cfg<T, D, 16, 4>>(p, mk, mv, ctas, ws, stream);
}

}  // namespace

size_t kv_attention_workspace(int B, int N, int Hq, int Hkv, int D) {
  const size_t nt = kv_row_tile(static_cast<long long>(N) * (Hq / Hkv));
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
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  const long long query_rows = static_cast<long long>(a.N) * p.G;
  char *w = static_cast<char *>(ws);
  if (kv_row_tile(query_rows) > 32) return launch_attention_rows(p, dtype, mk, mv, ctas, w, stream);
  const bool wide = kv_row_tile(query_rows) == 32;
  if (dtype == SPEC_BF16)
    return a.D == 64 ? launch_columns<__nv_bfloat16, 64>(wide, p, mk, mv, ctas, w, stream)
                     : launch_columns<__nv_bfloat16, 128>(wide, p, mk, mv, ctas, w, stream);
  return a.D == 64 ? launch_columns<__half, 64>(wide, p, mk, mv, ctas, w, stream)
                   : launch_columns<__half, 128>(wide, p, mk, mv, ctas, w, stream);
}

}  // namespace specv
