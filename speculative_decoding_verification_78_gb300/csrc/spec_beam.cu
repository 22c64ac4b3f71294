// spec_beam.cu -- beam search's selection over beams and vocabulary, and the reordering of what belongs to
// the beams.
//
// The mathematics. Candidate (k, v) of a batch row has the score s_k + l[k,v] - L_k, L_k = log sum_v e^l[k,v];
// the n best are wanted, ordered by score, equal ones by beam and token. Two kernels, as for verification:
// a stream kernel reads every logit once and leaves (maximum, sum) for each 4 KB unit of a row; a CTA a batch
// row then picks units by their maxima and tokens from those units.
//
// Exactness. The order of two candidates of one beam is that of their logits, whatever L_k. Candidates of
// different beams are compared by L_k from fp32 sums, whose error is bounded (kCoarse); where two that matter
// lie nearer than that, the units that make up most of the L_k concerned are summed again to about 1e-10, as many
// as it takes to tell the two apart, and the selection is repeated. Scores are compared as integers of 192 bits, whole
// multiples of 2^-48, which hold any sum of fp32 numbers: beside a score of -1e9 fp32 pairs lose what tells beams
// apart. So tokens and parents are those of exact arithmetic (but for scores closer than 1e-9). The sums are taken in
// the order of the token numbers wherever a row lies in memory, so that beams with equal logits have equal L_k; those
// that are taken again are sums of integers, which are equal for rows that hold the same logits in another order too.
//
// What bounds it: for many beams HBM while the logits stream (64 x 8 beams x 152064 in bf16: 156 MB in 26 us, 5.9
// TB/s; 58 % of the issue slots, the rest waits for ex2 and for loads), then the finishing CTAs' chain of about ten
// short steps (17 000 clocks, of which a row's sums 3400, counting distances 2700, listing quarters of units 3200,
// reading those again 4200; each part runs once, and fetching its code is a good deal of it); together 34 us a call among
// others. For few beams that chain and the host (4 beams x 32000: 9 us a call in a graph of ten, 22 among others).
#include "spec_beam.h"
#include "spec_common.cuh"
#include "spec_kv.h"

namespace specv {

namespace {

constexpr int kFinishThreads = 512, kFinishWarps = kFinishThreads / 32;
constexpr float kLog2eHi = 0x1.715476p+0f, kLog2eLo = 0x1.4ae0cp-26f;   // their sum: log2(e) to 2^-50
constexpr float kLn2Hi = 0x1.62e43p-1f, kLn2Lo = -0x1.05c61p-29f;       // their sum: ln 2 to 2^-53
constexpr double kLog2ed = 1.44269504088896340736;
// A unit whose maximum is below this in magnitude is summed against the integer R above its maximum's
// logarithm: 2^(l log2 e - R), so that units are joined by powers of two. Beyond it (where R would not be an
// exact fp32 integer with room for a fraction) against its maximum itself.
constexpr float kPlainMax = 1048576.f;
// The bound of a unit sum's relative error, 1.8e-6: 2^-22 of ex2; the rounding of the exponent, 2^-24 |t| ln 2, and
// what log2(e)'s second word leaves of it, 10^-8 |t|, where |t| of 2048 terms below one of at least 2^-1 is at most 8
// on average; 18 roundings of sums and of the second word's factor. And that of a sum taken again (exp_pair), with
// what its logarithm adds.
constexpr float kCoarse = 2e-6f, kFine = 2e-10f;
constexpr float kUnitCut = 0x1p-40f;   // what a unit that is not summed again may lack, beside 2^R (see fixed)

__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// ------------------------------------------------------------------ reading a row by token numbers

// Elements e0 .. of the row as one vector, -inf past its end, where that is not a whole aligned vector: one of
// an unaligned row is put together from the two aligned ones it lies in, if both lie inside the row.
template <typename E>
__device__ __noinline__ uint4 load_uneven(const E *row, int V, int e0) {
  constexpr int kEPV = Elem<E>::kPerVec;
  const uint32_t ni = Elem<E>::kNegInfWord;
  uint32_t r[4] = {ni, ni, ni, ni};
  if (e0 >= V) return make_uint4(ni, ni, ni, ni);
  const E *at = row + e0;
  const unsigned mis = static_cast<unsigned>(reinterpret_cast<uintptr_t>(row) & 15u);
  if (mis != 0 && e0 > 0 && e0 + 2 * kEPV <= V) {
    const uint4 *p = reinterpret_cast<const uint4 *>(reinterpret_cast<uintptr_t>(at) - mis);
    const uint4 a = __ldg(p), b = __ldg(p + 1);
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    const unsigned q = mis >> 2, sh = (mis & 3u) * 8u;
    if (q & 1)
#pragma unroll
      for (int i = 0; i < 7; ++i) w[i] = w[i + 1];
    if (q & 2)
#pragma unroll
      for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    return make_uint4(__funnelshift_r(w[0], w[1], sh), __funnelshift_r(w[1], w[2], sh),
                      __funnelshift_r(w[2], w[3], sh), __funnelshift_r(w[3], w[4], sh));
  }
#pragma unroll
  for (int e = 0; e < kEPV; ++e)
    if (e0 + e < V) {
      const uint32_t bits = __float_as_uint(ld_elem<E>(at + e));
      if (sizeof(E) == 4)
        r[e] = bits;
      else
        r[e / 2] = (e & 1) ? (r[e / 2] & 0xffffu) | (bits & 0xffff0000u) : (r[e / 2] & 0xffff0000u) | (bits >> 16);
    }
  return make_uint4(r[0], r[1], r[2], r[3]);
}
// Vectors g, g + 32, ... of the row: the whole ones first, whose loads are on their way together.
template <typename E, int kN>
__device__ __forceinline__ void load_groups(const E *row, int V, int g, uint4 (&buf)[kN]) {
  constexpr int kEPV = Elem<E>::kPerVec;
  const bool even = (reinterpret_cast<uintptr_t>(row) & 15u) == 0;
#pragma unroll
  for (int j = 0; j < kN; ++j)
    if (even && (g + 32 * j + 1) * kEPV <= V) buf[j] = ld_stream(reinterpret_cast<const uint4 *>(row) + g + 32 * j);
  if (even && (g + 32 * (kN - 1) + 1) * kEPV <= V) return;
#pragma unroll
  for (int j = 0; j < kN; ++j)
    if (!even || (g + 32 * j + 1) * kEPV > V) buf[j] = load_uneven<E>(row, V, (g + 32 * j) * kEPV);
}

// What a beam contributes: nothing (score -inf), one candidate (at its end), or its row.
enum BeamKind : int { kUnused = 0, kEnded = 1, kLive = 2, kBad = 3 };
__device__ __forceinline__ int beam_kind(const BeamArgs &a, int row, float &s) {
  s = ld_given(a.scores + row);
  if (s == -INFINITY) return kUnused;
  if (s != s || s == INFINITY) return kBad;
  return a.done && ld_given(a.done + row) ? kEnded : kLive;
}

__device__ __forceinline__ float unit_ref(float m) { return ceilf(__fmul_rn(m, kLog2eHi)); }

template <typename E>
__global__ void __launch_bounds__(256, 4) beam_stream_kernel(const __grid_constant__ BeamArgs a) {
  constexpr int kEPV = Elem<E>::kPerVec;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  for (int unit = blockIdx.x * 8 + (threadIdx.x >> 5); unit < a.units; unit += 8 * gridDim.x) {
    const int row_i = static_cast<int>(static_cast<unsigned>(unit) / static_cast<unsigned>(a.C));
    const int chunk = unit - row_i * a.C;
    float score;
    if (beam_kind(a, row_i, score) != kLive) continue;
    if (!SPEC_CHECK(a, row_i < a.B * a.K && chunk < a.C)) continue;
    const E *row = static_cast<const E *>(a.logits) + static_cast<long long>(row_i) * a.V;
    uint4 buf[kVPL];
    load_groups<E>(row, a.V, chunk * kUnitVecs + lane, buf);
    float quarter[4];   // maxima (NaN ranks highest)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      quarter[q] = key_float(__reduce_max_sync(
          0xffffffffu, float_key(fmax_nan(vec_max<E>(buf[2 * q]), vec_max<E>(buf[2 * q + 1])))));
    float m = fmax_nan(fmax_nan(quarter[0], quarter[1]), fmax_nan(quarter[2], quarter[3]));
    float s = 0.f;
    if (m != -INFINITY) {
      f32x2 acc[4] = {pk2(0.f, 0.f), pk2(0.f, 0.f), pk2(0.f, 0.f), pk2(0.f, 0.f)};
      if (fabsf(m) < kPlainMax) {
        const float R = unit_ref(m);
        const f32x2 hi = pk2(kLog2eHi, kLog2eHi), nr = pk2(-R, -R);
#pragma unroll
        for (int j = 0; j < kVPL; ++j)
#pragma unroll
          for (int e = 0; e < kEPV; e += 2) {
            const f32x2 x = pk2(vec_elem<E>(buf[j], e), vec_elem<E>(buf[j], e + 1));
            float t0, t1;
            up2(fma2(x, hi, nr), t0, t1);
            f32x2 &c = acc[(j * (kEPV / 2) + e / 2) & 3];
            c = add2(c, pk2(ex2(t0), ex2(t1)));
          }
      } else {   // (NaN and +inf come here and leave NaN in the maximum's place)
#pragma unroll
        for (int j = 0; j < kVPL; ++j)
#pragma unroll
          for (int e = 0; e < kEPV; e += 2)
            acc[(e / 2) & 3] = add2(acc[(e / 2) & 3], pk2(ex2_shift(vec_elem<E>(buf[j], e), m, kLog2eHi),
                                                          ex2_shift(vec_elem<E>(buf[j], e + 1), m, kLog2eHi)));
      }
      float v0, v1;
      up2(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])), v0, v1);
      s = __fadd_rn(v0, v1);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, o));
      // 2^(m lo) for log2(e)'s second word, with the largest logit for each: those that count are near it
      if (fabsf(m) < kPlainMax) {
        const float y = m * (kLog2eLo * kLn2Hi);
        s = __fmaf_rn(s, __fmaf_rn(y * y, __fmaf_rn(y, 1.f / 6.f, 0.5f), y), s);
      }
      if (m == INFINITY) m = NAN;
    }
    if (lane == 0) {
      a.part[unit] = make_uint2(__float_as_uint(m), __float_as_uint(s));
      a.quarters[unit] = make_float4(quarter[0], quarter[1], quarter[2], quarter[3]);
    }
  }
}

// ------------------------------------------------------------------ an exponential to 1e-10

// e^(x - M), x <= M, as a sum of two fp32 numbers. With x - M = d + dl exactly, t = (x - M) log2 e = n + f,
// |f| <= 1/2: 2^n e^y with y = f ln 2 in two words; 1 + y + y^2/2 + y^3/6 in two words and the rest of
// Taylor's series, below 7e-4, in one.
__device__ __forceinline__ void exp_pair(float x, float M, float &hi, float &lo) {
  const float d = __fsub_rn(x, M);
  if (!(d > -87.f)) {
    hi = lo = 0.f;
    return;
  }
  const float bb = __fsub_rn(d, x);
  const float dl = __fadd_rn(__fsub_rn(x, __fsub_rn(d, bb)), __fsub_rn(-M, bb));
  const float t = __fmul_rn(d, kLog2eHi);
  const float te = __fmaf_rn(dl, kLog2eHi, __fmaf_rn(d, kLog2eLo, __fmaf_rn(d, kLog2eHi, -t)));
  const float n = rintf(t), f = __fsub_rn(t, n);
  const float yh = __fmul_rn(f, kLn2Hi);
  const float yl = __fmaf_rn(te, kLn2Hi, __fmaf_rn(f, kLn2Lo, __fmaf_rn(f, kLn2Hi, -yh)));
  const float y2h = __fmul_rn(yh, yh);
  const float y2l = __fmaf_rn(2.f * yh, yl, __fmaf_rn(yh, yh, -y2h));
  const float y3h = __fmul_rn(y2h, yh);
  const float y3l = __fmaf_rn(y2h, yl, __fmaf_rn(y2l, yh, __fmaf_rn(y2h, yh, -y3h)));
  constexpr float kSixthHi = 0x1.555556p-3f, kSixthLo = -0x1.555556p-28f;
  const float ch = __fmul_rn(y3h, kSixthHi);
  const float cl = __fmaf_rn(y3l, kSixthHi, __fmaf_rn(y3h, kSixthLo, __fmaf_rn(y3h, kSixthHi, -ch)));
  float q = 1.f / 3628800.f;
  q = __fmaf_rn(q, yh, 1.f / 362880.f);
  q = __fmaf_rn(q, yh, 1.f / 40320.f);
  q = __fmaf_rn(q, yh, 1.f / 5040.f);
  q = __fmaf_rn(q, yh, 1.f / 720.f);
  q = __fmaf_rn(q, yh, 1.f / 120.f);
  q = __fmaf_rn(q, yh, 1.f / 24.f);
  const float rest = __fmul_rn(__fmul_rn(y2h, y2h), q);
  // (each sum's second term is the smaller)
  const float s1 = __fadd_rn(1.f, yh), e1 = __fsub_rn(yh, __fsub_rn(s1, 1.f));
  const float h2 = 0.5f * y2h;
  const float s2 = __fadd_rn(s1, h2), e2 = __fsub_rn(h2, __fsub_rn(s2, s1));
  const float s3 = __fadd_rn(s2, ch), e3 = __fsub_rn(ch, __fsub_rn(s3, s2));
  const float low = ((e1 + e2) + (e3 + yl)) + ((0.5f * y2l + cl) + rest);
  const float scale = __uint_as_float(static_cast<uint32_t>(static_cast<int>(n) + 127) << 23);
  hi = s3 * scale;
  lo = low * scale;
}

// A sum of such pairs (each at most 1, at most 2^20 of them) that does not depend on their order: each is cut into
// multiples of 2^-20, 2^-41 and 2^-62, which leaves less than 2^-62 of it; up to eight are added in fp32, which holds
// those sums exactly, and then as integers. (4 equal beams x 32000, one of which is summed again: 2 us of 41 for it;
// with two conversions of each term to 64 bits 14 of 53.)
struct ExactSum {
  long long n[3] = {0, 0, 0};
  // x rounded to a multiple of 2^-23 kOne, |x| < kOne / 4
  static __device__ __forceinline__ float cut(float x, float kOne) {
    return __fsub_rn(__fadd_rn(x, 1.5f * kOne), 1.5f * kOne);
  }
  static __device__ __forceinline__ void split(float hi, float lo, float (&t)[3]) {
    const float x = __fadd_rn(hi, lo);   // (lo may be 2^-10 of it)
    lo = __fsub_rn(lo, __fsub_rn(x, hi));
    const float a = cut(x, 0x1p3f), r = __fsub_rn(x, a);
    const float b = cut(r, 0x1p-18f), c = cut(lo, 0x1p-18f);
    const float d = cut(__fadd_rn(__fsub_rn(r, b), __fsub_rn(lo, c)), 0x1p-39f);
    t[0] = __fadd_rn(t[0], a);
    t[1] = __fadd_rn(t[1], __fadd_rn(b, c));
    t[2] = __fadd_rn(t[2], d);
  }
  __device__ __forceinline__ void add(const float (&t)[3]) {
    n[0] += __float2int_rn(t[0] * 0x1p20f);
    n[1] += __float2int_rn(t[1] * 0x1p41f);
    n[2] += __float2int_rn(t[2] * 0x1p62f);
  }
  __device__ __forceinline__ double value() const {
    return static_cast<double>(n[0]) * 0x1p-20 +
           (static_cast<double>(n[1]) * 0x1p-41 + static_cast<double>(n[2]) * 0x1p-62);
  }
};

// log(n 2^-40) for n > 0, as a sum of two fp32 numbers, to about 1e-10: with n 2^-40 = x 2^e, x in [1, 2),
// fp32's logarithm y of x, put right by x e^-y - 1, and e ln 2.
__device__ __forceinline__ void log_pair(unsigned long long n, float &hi, float &lo) {
  const int top = 63 - __clzll(static_cast<long long>(n));
  const unsigned long long w = n << (63 - top);          // x 2^63
  const float xh = __uint_as_float((127u << 23) | static_cast<uint32_t>((w >> 40) & 0x7fffffu));
  const float xl = static_cast<float>(static_cast<uint32_t>(w >> 8)) * 0x1p-55f;   // its next 32 bits
  const float y = logf(xh);
  float eh, el;
  exp_pair(-y, 0.f, eh, el);
  const float p = __fmul_rn(xh, eh);   // near 1: p - 1 is exact
  const float r = __fadd_rn(__fsub_rn(p, 1.f), __fmaf_rn(xh, el, __fmaf_rn(xl, eh, __fmaf_rn(xh, eh, -p))));
  const float e = static_cast<float>(top - 40);
  const float th = __fmul_rn(e, kLn2Hi);
  hi = __fadd_rn(th, y);
  const float bb = __fsub_rn(hi, th);
  lo = __fadd_rn(__fadd_rn(__fsub_rn(th, __fsub_rn(hi, bb)), __fsub_rn(y, bb)),
                 __fadd_rn(r, __fmaf_rn(e, kLn2Lo, __fmaf_rn(e, kLn2Hi, -th))));
}

// ------------------------------------------------------------------ selection
//
// What bounds the selection is the chain of its steps, and 64-bit floating point, of which an SM does two
// operations a clock (a warp's instruction takes its scheduler 64): L_k is a pair of fp32 numbers, and scores,
// taken for the few hundred candidates only, are integers.

// A number as a whole multiple of 2^-48: 192 bits, two's complement (fp32's range is 2^128: sums of a few of its
// numbers fit). Rounding to it keeps the order of numbers, and nothing is rounded after.
struct Fixed {
  unsigned long long lo, mid;
  long long hi;
};
__device__ __forceinline__ Fixed operator+(const Fixed &x, const Fixed &y) {
  Fixed r;
  asm("add.cc.u64 %0, %3, %6;\n\taddc.cc.u64 %1, %4, %7;\n\taddc.u64 %2, %5, %8;"
      : "=l"(r.lo), "=l"(r.mid), "=l"(r.hi)
      : "l"(x.lo), "l"(x.mid), "l"(x.hi), "l"(y.lo), "l"(y.mid), "l"(y.hi));
  return r;
}
__device__ __forceinline__ Fixed operator-(const Fixed &x, const Fixed &y) {
  Fixed r;
  asm("sub.cc.u64 %0, %3, %6;\n\tsubc.cc.u64 %1, %4, %7;\n\tsubc.u64 %2, %5, %8;"
      : "=l"(r.lo), "=l"(r.mid), "=l"(r.hi)
      : "l"(x.lo), "l"(x.mid), "l"(x.hi), "l"(y.lo), "l"(y.mid), "l"(y.hi));
  return r;
}
__device__ __forceinline__ bool operator==(const Fixed &x, const Fixed &y) {
  return x.lo == y.lo && x.mid == y.mid && x.hi == y.hi;
}
__device__ __forceinline__ bool operator>(const Fixed &x, const Fixed &y) {
  return x.hi != y.hi ? x.hi > y.hi : x.mid != y.mid ? x.mid > y.mid : x.lo > y.lo;
}
__device__ __forceinline__ Fixed fixed_of(long long v) {   // v 2^-48
  return Fixed{static_cast<unsigned long long>(v), static_cast<unsigned long long>(v >> 63), v >> 63};
}
__device__ __forceinline__ long long near_fixed(float f) { return __float2ll_rn(f * 0x1p48f); }   // |f| < 2^14
// (What numbers of ordinary size do not need is called: a CTA runs this code once, so that fetching it costs as much.)
__device__ __noinline__ Fixed far_fixed(float f) {
  const uint32_t bits = __float_as_uint(f);
  const unsigned long long mant = (bits & 0x7fffffu) | 0x800000u;
  const int up = static_cast<int>(bits >> 23 & 255u) - 127 - 23 + 48, word = up >> 6, at = up & 63;   // 39 .. 152
  const unsigned long long low = mant << at, high = at > 40 ? mant >> (64 - at) : 0ull;
  const Fixed r{word == 0 ? low : 0ull, word == 0 ? high : word == 1 ? low : 0ull,
                static_cast<long long>(word == 0 ? 0ull : word == 1 ? high : low)};
  return bits >> 31 ? Fixed{0, 0, 0} - r : r;
}
__device__ __forceinline__ Fixed fixed_of(float f) {   // (no infinity, no NaN)
  return fabsf(f) < 16384.f ? fixed_of(near_fixed(f)) : far_fixed(f);
}
__device__ __noinline__ float far_float(const Fixed &x) {
  return static_cast<float>(x.lo) * 0x1p-48f + (static_cast<float>(x.mid) * 0x1p16f + static_cast<float>(x.hi) * 0x1p80f);
}
__device__ __forceinline__ float float_of(const Fixed &x) {   // x >= 0
  return x.mid | static_cast<unsigned long long>(x.hi) ? far_float(x) : static_cast<float>(x.lo) * 0x1p-48f;
}
// (h, l) += (x, y), y and l small beside the others
__device__ __forceinline__ void pair_add(float &h, float &l, float x, float y) {
  const float t = __fadd_rn(h, x), bb = __fsub_rn(t, h);
  l = __fadd_rn(__fadd_rn(__fsub_rn(h, __fsub_rn(t, bb)), __fsub_rn(x, bb)), __fadd_rn(l, y));
  h = t;
}

// A candidate: its beam, logit and place in the beam.
struct Cand {
  float l;
  int k, at;
};
// Equal scores go by beam; within one by logit (which may differ by less than scores tell), then by place.
__device__ __forceinline__ bool before(const Cand &x, const Cand &y) {
  if (x.k != y.k) return x.k < y.k;
  return x.l > y.l || (x.l == y.l && x.at < y.at);
}
// One with its score; none (k: kNoBeam) comes last.
constexpr int kNoBeam = 0x7fffffff;
struct Pick {
  Fixed score;
  Cand c;
  __device__ __forceinline__ bool some() const { return c.k != kNoBeam; }
};
__device__ __forceinline__ bool before(const Pick &x, const Pick &y) {
  if (!x.some() || !y.some()) return x.some();
  return x.score == y.score ? before(x.c, y.c) : x.score > y.score;
}
__device__ __forceinline__ Fixed shuffle_xor(const Fixed &x, int o) {
  return Fixed{__shfl_xor_sync(0xffffffffu, x.lo, o), __shfl_xor_sync(0xffffffffu, x.mid, o),
               __shfl_xor_sync(0xffffffffu, x.hi, o)};
}
__device__ __forceinline__ Pick warp_best(Pick p) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Pick q;
    q.score = shuffle_xor(p.score, o);
    q.c.l = __shfl_xor_sync(0xffffffffu, p.c.l, o);
    q.c.k = __shfl_xor_sync(0xffffffffu, p.c.k, o);
    q.c.at = __shfl_xor_sync(0xffffffffu, p.c.at, o);
    if (before(q, p)) p = q;
  }
  return p;
}
__device__ __forceinline__ Pick no_pick() { return Pick{{0, 0, 0}, {-INFINITY, kNoBeam, 0}}; }

constexpr int kBins = 1024, kMaxParts = 512, kMaxCands = 512;
constexpr int kStaged = 2048;   // units whose maxima are kept in shared memory

// Bin of a distance d >= 0 from the best score: 32 bins an octave from 2^-8 to 2^24, what is nearer in the first
// and what is farther in the last. A distance is known to 2^-22 of itself, a bin is 2^-5 wide, and no bin but
// the first narrower than 2^-13: a candidate is in its bin or, where that matters, in the next, kCoarse included.
__device__ __forceinline__ int bin_of(float d) {
  return min(max(static_cast<int>(__float_as_uint(d) >> 18) - ((127 - 8) << 5), 0), kBins - 1);
}

static_assert(SPEC_MAX_BEST <= kFinishThreads, "a thread for each result");

struct FinishShared {
  float base[SPEC_MAX_BEAMS];      // how far a beam's best candidate is from the best of all
  __align__(16) int hist[kBins];
  int edge, parts, cands;
  float staged[kStaged];
  int part_list[kMaxParts];        // quarters of units: 4 unit + quarter
  ulonglong2 key[kMaxCands];       // a candidate's distance from the best, and what equal ones go by
  Cand cand[kMaxCands];            // place: the token
  int order[kMaxCands];
  Fixed offset[SPEC_MAX_BEAMS];    // what a beam's logits lack to be scores: s - top - log_sum
  Fixed best_of[SPEC_MAX_BEAMS];   // a beam's best score
  Fixed best_score;                // of all
  float2 log_sum[SPEC_MAX_BEAMS];  // L_k - top: the sum of two words
  float s[SPEC_MAX_BEAMS], top[SPEC_MAX_BEAMS];
  int kind[SPEC_MAX_BEAMS];
  float slack[SPEC_MAX_BEAMS];     // how far L_k may be off
  int target[SPEC_MAX_BEAMS];      // what that has to come down to (as the bits of a positive float)
  Pick warp[kFinishWarps], best;
  int unit[SPEC_MAX_BEST];     // chosen units, in order
  Pick head[SPEC_MAX_BEST];    // the best of each that is left; place: the token
  ExactSum sum[kFinishWarps];
  int bad, again;
  float least;
  unsigned long long rest;
  int left;   // units
};

// The longer parts of it that are seldom taken are functions of their own, made of the same members (one that were a
// member itself would keep the others' fields in memory).
template <typename E>
__device__ __noinline__ float2 large_sum_apart(const BeamArgs &a, FinishShared &sh, int b, int k, float m);
template <typename E>
__device__ __noinline__ void refine_apart(const BeamArgs &a, FinishShared &sh, int b, int k);
template <typename E>
__device__ __noinline__ int rank_far_apart(const BeamArgs &a, FinishShared &sh, int b, int count);
template <typename E>
__device__ __noinline__ bool select_any_apart(const BeamArgs &a, FinishShared &sh, int b);

template <typename E>
struct Finish {
  const BeamArgs &a;
  FinishShared &sh;
  const int b, tid, lane, warp;

  __device__ __forceinline__ const E *row(int k) const {
    return static_cast<const E *>(a.logits) + (static_cast<long long>(b) * a.K + k) * a.V;
  }
  __device__ __forceinline__ uint2 part(int u) const {
    return __ldcg(a.part + static_cast<long long>(b) * a.K * a.C + u);
  }
  // unit u = k C + chunk of the batch row, by its largest candidate
  __device__ __forceinline__ Pick unit_pick(int u) const {
    const int k = u / a.C, chunk = u - k * a.C;
    if (sh.kind[k] == kEnded && chunk == 0) return Pick{sh.best_of[k], {0.f, k, chunk}};
    if (sh.kind[k] != kLive) return no_pick();
    const float m = __uint_as_float(part(u).x);
    return m > -INFINITY ? Pick{score(k, m), {m, k, chunk}} : no_pick();
  }
  // the score of a beam's candidate with logit l (an ended beam's: 0)
  __device__ __forceinline__ Fixed score(int k, float l) const { return sh.offset[k] + fixed_of(l); }
  // and as it is returned, of the words that it is made of
  __device__ __forceinline__ float score_out(const Cand &c) const {
    float x = sh.s[c.k], y = 0.f, d = c.l, dl = 0.f;
    pair_add(x, y, -sh.log_sum[c.k].x, -sh.log_sum[c.k].y);
    pair_add(d, dl, -sh.top[c.k], 0.f);
    const float far = __fadd_rn(x, d);
    if (!(far > -INFINITY)) return -INFINITY;   // beyond fp32
    pair_add(x, y, d, dl);
    return __fadd_rn(x, y);
  }
  // two candidates of beams k and j, `gap` apart, whose order the sums as they are do not tell: asks for better ones
  __device__ __forceinline__ void compare(float gap, int k, int j) const {
    if (k == j || !(gap <= sh.slack[k] + sh.slack[j])) return;
    // 0 as well: sums that fp32 rounds alike are not the same yet
    want(k, 0.4f * gap);
    want(j, 0.4f * gap);
  }
  // A beam whose sum has been improved and does not tell either is summed whole: the gap was the sums' errors.
  __device__ __forceinline__ void want(int k, float slack) const {
    if (sh.slack[k] <= kFine || sh.slack[k] <= slack) return;
    atomicMin(&sh.target[k], sh.slack[k] < kCoarse ? 0 : __float_as_int(slack));
    sh.again = 1;
  }

  // L_k from the unit sums, a warp a beam. Sums against powers of two are added as whole multiples of 2^-40
  // (a unit's is at most 2^12, and there are at most 2^10): exactly, but for what lies below that.
  __device__ __forceinline__ void sums() const {
    for (int k = warp; k < a.K; k += kFinishWarps) {
      float s;
      const int kind = beam_kind(a, b * a.K + k, s);
      float m = -INFINITY;          // of the units so far
      unsigned long long t = 0;     // their sum against the power of two of m
      for (int c0 = 0; c0 < a.C; c0 += 4 * 32) {
        uint2 w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int c = c0 + u * 32 + lane;
          w[u] = c < a.C ? part(k * a.C + c) : make_uint2(0xff800000u, 0u);
          if (c < a.C && k * a.C + c < kStaged) sh.staged[k * a.C + c] = __uint_as_float(w[u].x);
        }
        float top = m;
#pragma unroll
        for (int u = 0; u < 4; ++u) top = fmax_nan(top, __uint_as_float(w[u].x));
        top = key_float(__reduce_max_sync(0xffffffffu, float_key(top)));
        const float R = unit_ref(top);
        t = scaled(t, unit_ref(m) - R);
        m = top;
#pragma unroll
        for (int u = 0; u < 4; ++u) t += fixed(w[u], R);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      const bool live = kind == kLive;
      float h = 0.f, l = 0.f, top = 0.f;
      if (live && plain_row(m)) {
        top = m;
        log_pair(t, h, l);
        // + R ln 2 - m, of which R ln 2 and m may be large and near each other
        const float R = unit_ref(m), rh = __fmul_rn(R, kLn2Hi);
        const float rl = __fmaf_rn(R, kLn2Lo, __fmaf_rn(R, kLn2Hi, -rh));
        float d = rh, dl = rl;
        pair_add(d, dl, -m, 0.f);
        pair_add(h, l, d, dl);
      } else if (live) {
        top = m;
        const float2 x = large_sum_apart<E>(a, sh, b, k, m);
        h = x.x;
        l = x.y;
      }
      if (lane == 0) {
        sh.kind[k] = kind;
        sh.s[k] = s;
        sh.slack[k] = live ? kCoarse : 0.f;
        sh.target[k] = 0x7f800000;
        if (kind == kBad || (live && !(fabsf(m) < INFINITY)))
          sh.bad = 1;
        else
          set_sum(k, top, h, l);
      }
    }
  }
  // a row that is summed against powers of two (a unit below -kPlainMax adds nothing to it)
  static __device__ __forceinline__ bool plain_row(float m) { return m > 64.f - kPlainMax && m < kPlainMax; }
  // a unit's sum against 2^R, in units of 2^-40
  static __device__ __forceinline__ unsigned long long fixed(uint2 w, float R) {
    const uint32_t bits = w.y;   // a sum in [2^-1, 2^12), or 0
    if (!bits) return 0;
    const unsigned long long mant = (bits & 0x7fffffu) | 0x800000u;
    const int e = static_cast<int>(bits >> 23) - 127 - 23 + 40;   // of its last bit
    return scaled(e >= 0 ? mant << min(e, 40) : mant >> min(-e, 63), unit_ref(__uint_as_float(w.x)) - R);
  }
  static __device__ __forceinline__ unsigned long long scaled(unsigned long long t, float e) {   // t 2^e, e <= 0
    return e > -64.f ? t >> static_cast<int>(-e) : 0ull;
  }
  __device__ __forceinline__ void set_sum(int k, float top, float h, float l) const {
    sh.top[k] = top;
    sh.log_sum[k] = make_float2(h, l);
    if (sh.kind[k] != kLive && sh.kind[k] != kEnded) return;
    sh.best_of[k] = fixed_of(sh.s[k]) - fixed_of(near_fixed(h) + near_fixed(l));
    sh.offset[k] = sh.best_of[k] - fixed_of(top);
  }
  // log sum_v e^(l - m) of a row whose largest logit m is too large for powers of two, in 64 bits
  __device__ __forceinline__ float2 large_sum(int k, float m) const {
    double t = 0.;
    for (int c = lane; c < a.C; c += 32) {
      const uint2 w = part(k * a.C + c);
      const float um = __uint_as_float(w.x);
      if (um == -INFINITY) continue;
      // from the unit's reference to its maximum, and from there to the row's
      const double to_max = fabsf(um) < kPlainMax ? unit_ref(um) - um * kLog2ed : 0.;
      t += static_cast<double>(__uint_as_float(w.y)) * exp2(to_max + (static_cast<double>(um) - m) * kLog2ed);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    const double x = log(t);
    const float h = static_cast<float>(x);
    return make_float2(h, static_cast<float>(x - h));
  }

  // Whether beam k's row is beam j's, bit for bit (the whole CTA; 128 vectors of each at a time a warp).
  __device__ __forceinline__ bool same_row(int k, int j) const {
    bool same = true;
    for (int c = warp; c < a.C * (kUnitVecs / 128) && same; c += kFinishWarps) {
      uint4 v[4], w[4];
      load_groups<E>(row(k), a.V, c * 128 + lane, v);
      load_groups<E>(row(j), a.V, c * 128 + lane, w);
      bool here = true;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        here = here && v[q].x == w[q].x && v[q].y == w[q].y && v[q].z == w[q].z && v[q].w == w[q].w;
      same = __all_sync(0xffffffffu, here);
    }
    return __syncthreads_and(same);
  }

  // L_k again, to within sh.target[k], by the whole CTA: the units that hold most of the sum are summed again, the
  // others (all that may stay out by their shares) count as they are. Beams that start from one row with one score
  // are all nearer than their sums tell: the first is summed, the others only compared with it (bf16, in a
  // graph of ten: 4 x 32000 alike 38 us a call, the same in other orders, each summed, 90; 2 x 64 x 152064 alike 480).
  __device__ __forceinline__ void refine(int k) const {
    const float M = sh.top[k], target = __int_as_float(sh.target[k]);
    for (int j = 0; j < k; ++j)
      if (sh.kind[j] == kLive && sh.s[j] == sh.s[k] && sh.top[j] == M && sh.slack[j] <= fmaxf(target, kFine)) {
        if (!same_row(k, j)) break;   // (what else there is that looks the same is not searched for)
        if (tid == 0) {
          sh.log_sum[k] = sh.log_sum[j];
          sh.offset[k] = sh.offset[j];
          sh.best_of[k] = sh.best_of[j];
          sh.slack[k] = sh.slack[j];
          sh.target[k] = 0x7f800000;
        }
        __syncthreads();
        return;
      }
    const bool plain = plain_row(M);
    const float R = unit_ref(M);
    float *weight = reinterpret_cast<float *>(sh.key);   // of each unit, against 2^R (at most 2^10 units)
    static_assert(sizeof(sh.key) >= 4 * (SPEC_MAX_V / (4 * kUnitVecs)), "room for a row's units");
    for (int c = tid; c < a.C; c += kFinishThreads) {
      const uint2 w = part(k * a.C + c);
      weight[c] = plain ? static_cast<float>(fixed(w, R)) * 0x1p-40f : 1.f;
    }
    if (tid == 0) sh.least = 0.f;
    __syncthreads();
    if (warp == 0 && plain && target > kFine) {   // a threshold a lane: 2^(10 - lane); the largest that leaves out little enough
      const float at = ldexpf(1.f, 10 - lane);
      float all = 0.f, out = 0.f, cut_off = 0.f;
      for (int c = 0; c < a.C; ++c) {
        all += weight[c];
        if (weight[c] < at) {
          out += weight[c];
          cut_off += kUnitCut;
        }
      }
      const unsigned fits =
          __ballot_sync(0xffffffffu, out * (1.01f * kCoarse) + kFine * all + cut_off <= target * all);
      if (lane == 0 && fits) sh.least = ldexpf(1.f, 10 - (__ffs(fits) - 1));
    }
    __syncthreads();
    const float least = sh.least;
    if (warp == kFinishWarps - 1) {
      unsigned long long rest = 0;
      int left = 0;
      for (int c = lane; c < a.C; c += 32)
        if (weight[c] < least) {
          rest += fixed(part(k * a.C + c), R);
          ++left;
        }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, o);
      left = __reduce_add_sync(0xffffffffu, left);
      if (lane == 0) {
        sh.rest = rest;
        sh.left = left;
      }
    }
    ExactSum sum;
    int n = 0;
    for (int c = 0; c < a.C; ++c) {   // half of the CTA a unit
      if (weight[c] < least) continue;
      if ((n++ & 1) != tid / kUnitVecs) continue;
      uint4 v[1];
      load_groups<E>(row(k), a.V, c * kUnitVecs + tid % kUnitVecs, v);
      float t[3] = {0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < Elem<E>::kPerVec; ++e) {
        float xh, xl;
        exp_pair(vec_elem<E>(v[0], e), M, xh, xl);
        ExactSum::split(xh, xl, t);
      }
      sum.add(t);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < 3; ++i) sum.n[i] += __shfl_xor_sync(0xffffffffu, sum.n[i], o);
    if (lane == 0) sh.sum[warp] = sum;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kFinishWarps; ++w)
        for (int i = 0; i < 3; ++i) sum.n[i] += sh.sum[w].n[i];
      const double all = sum.value();
      const double out = sh.rest ? static_cast<double>(sh.rest) * 0x1p-40 * exp(R / kLog2ed - M) : 0.;
      const double x = log(all + out);
      const float hi = static_cast<float>(x);
      set_sum(k, M, hi, static_cast<float>(x - hi));
      // not above what was asked for, whatever was rounded: else the same would be asked for again
      // (a sum is at least half of 2^R)
      const float cut_off = static_cast<float>(sh.left) * (2.f * kUnitCut);
      sh.slack[k] =
          sh.left ? fminf(kFine + static_cast<float>(out / (all + out)) * kCoarse + cut_off, target) : kFine;
      sh.target[k] = 0x7f800000;
    }
    __syncthreads();
  }

  // The first bin up to which at least `n` of the counted things lie, to sh.edge (kBins - 1 if there are fewer).
  __device__ __forceinline__ void find_edge(int n) const {
    if (warp == 0) {
      constexpr int kChunks = kBins / 128;   // a lane has four bins of each
      int4 c[kChunks];
      int sum[kChunks];
#pragma unroll
      for (int i = 0; i < kChunks; ++i) c[i] = reinterpret_cast<const int4 *>(sh.hist)[i * 32 + lane];
#pragma unroll
      for (int i = 0; i < kChunks; ++i) sum[i] = __reduce_add_sync(0xffffffffu, c[i].x + c[i].y + c[i].z + c[i].w);
      int before = 0, at = -1;
      int4 mine = make_int4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < kChunks; ++i)
        if (at < 0) {
          if (before + sum[i] >= n) {
            at = i;
            mine = c[i];
          } else {
            before += sum[i];
          }
        }
      if (at < 0) {
        if (lane == 0) sh.edge = kBins - 1;
      } else {
        const int all = mine.x + mine.y + mine.z + mine.w;
        int incl = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        int x = before + incl - all;
        if (x < n && x + all >= n) {
          int e = at * 128 + lane * 4;
          if ((x += mine.x) < n) ++e;
          if (x < n && (x += mine.y) < n) ++e;
          if (x < n && (x += mine.z) < n) ++e;
          sh.edge = e;
        }
      }
    }
    __syncthreads();
  }
  __device__ __forceinline__ void clear_hist_only() const {
#pragma unroll
    for (int i = 0; i < kBins / kFinishThreads; ++i) sh.hist[i * kFinishThreads + tid] = 0;
  }
  __device__ __forceinline__ void clear_hist() const {
    clear_hist_only();
    if (tid == 0) sh.parts = sh.cands = 0;
  }
  // the distance of unit u's best candidate, negative if it has none
  __device__ __forceinline__ float unit_distance(int u) const {
    const int k = u / a.C, chunk = u - k * a.C, kind = sh.kind[k];
    if (kind == kEnded) return chunk == 0 ? sh.base[k] : -1.f;
    if (kind != kLive) return -1.f;
    const float m = u < kStaged ? sh.staged[u] : __uint_as_float(part(u).x);
    return m > -INFINITY ? sh.base[k] + (sh.top[k] - m) : -1.f;
  }
  __device__ __forceinline__ void push(int k, float l, int token) const {
    const int i = atomicAdd(&sh.cands, 1);
    if (i < kMaxCands) sh.cand[i] = Cand{l, k, token};
  }
  // Lists (or, with `count`, counts by their distances) the listed quarters' candidates with a distance of at
  // most `most`.
  __device__ __forceinline__ void each_token(float most, bool count) const {
    constexpr int kAhead = 2;   // quarters of a warp whose loads are on their way together
    for (int i0 = warp; i0 < sh.parts; i0 += kAhead * kFinishWarps) {
      uint4 buf[kAhead][2];
      int beam[kAhead], token[kAhead];
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const int i = i0 + q * kFinishWarps;
        beam[q] = -1;
        if (i >= sh.parts) continue;
        const int part = sh.part_list[i], k = (part >> 2) / a.C;
        const int g = ((part >> 2) - k * a.C) * kUnitVecs + (part & 3) * 64 + lane;
        beam[q] = k;
        token[q] = g * Elem<E>::kPerVec;
        if (sh.kind[k] == kEnded) continue;
        load_groups<E>(row(k), a.V, g, buf[q]);
      }
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const int k = beam[q];
        if (k < 0) continue;
        const float base = sh.base[k], top = sh.top[k];
        const bool ended = sh.kind[k] == kEnded;
        if (ended && lane == 0) {
          if (count)
            atomicAdd(&sh.hist[bin_of(base)], 1);
          else
            push(k, 0.f, a.pad);
        }
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          if (ended || !(base + (top - vec_max<E>(buf[q][v])) <= most)) continue;
          unsigned near = 0;
#pragma unroll
          for (int e = 0; e < Elem<E>::kPerVec; ++e) {
            const float l = vec_elem<E>(buf[q][v], e);
            if (l > -INFINITY && base + (top - l) <= most) near |= 1u << e;
          }
#pragma unroll 1
          for (; near; near &= near - 1) {
            const int e = __ffs(near) - 1;
            const float l = element(buf[q][v], e);
            if (count)
              atomicAdd(&sh.hist[bin_of(base + (top - l))], 1);
            else
              push(k, l, token[q] + v * 32 * Elem<E>::kPerVec + e);
          }
        }
      }
    }
  }
  static __device__ __forceinline__ float element(const uint4 &v, int e) {   // e not known when compiled
    const int i = sizeof(E) == 4 ? e : e >> 1;
    const uint32_t w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
    return sizeof(E) == 4 ? __uint_as_float(w) : (e & 1) ? bf_hi(w) : bf_lo(w);
  }
  static __device__ __forceinline__ float bin_end(int bin) {   // distances in it and below are less than this
    return bin >= kBins - 1 ? INFINITY : __uint_as_float(static_cast<unsigned>(bin + 1 + ((127 - 8) << 5)) << 18);
  }

  // The places of `count` listed candidates by their whole scores.
  __device__ __forceinline__ int rank_far(int count) const {
    if (tid >= count) return 0;
    const Cand me = sh.cand[tid];
    const Fixed mine = score(me.k, me.l);
    int rank = 0;
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
      const Cand c = sh.cand[i];
      const Fixed x = score(c.k, c.l);
      rank += x == mine ? before(c, me) : x > mine;
    }
    return rank;
  }

  // Where a few hundred candidates are all that can matter: finds them by their distances, and ranks them by
  // counting. Returns 0 where there are more, 1 when done, -1 if sums have to be improved first.
  __device__ int select_few() const {
    if (tid < 32) {   // the best score of all; distances are then sums of small numbers
      Fixed top{0, 0, static_cast<long long>(1ull << 63)};   // (less than any)
      for (int k = lane; k < a.K; k += 32)
        if ((sh.kind[k] == kLive || sh.kind[k] == kEnded) && sh.best_of[k] > top) top = sh.best_of[k];
#pragma unroll 1
      for (int o = 16; o > 0; o >>= 1) {
        if (o >= a.K) continue;   // (lanes without a beam have none to give)
        const Fixed x = shuffle_xor(top, o);
        if (x > top) top = x;
      }
      top = Fixed{__shfl_sync(0xffffffffu, top.lo, 0), __shfl_sync(0xffffffffu, top.mid, 0),
                  __shfl_sync(0xffffffffu, top.hi, 0)};
      if (lane == 0) sh.best_score = top;
      for (int k = lane; k < a.K; k += 32)
        if (sh.kind[k] == kLive || sh.kind[k] == kEnded) sh.base[k] = float_of(top - sh.best_of[k]);
    }
    clear_hist();
    __syncthreads();
    const int all = a.K * a.C;
    for (int u = tid; u < all; u += kFinishThreads) {
      const float d = unit_distance(u);
      if (d >= 0.f) atomicAdd(&sh.hist[bin_of(d)], 1);
    }
    __syncthreads();
    find_edge(a.n);
    int edge = sh.edge;
    const float most = bin_end(edge + 1);
    for (int u = tid; u < all; u += kFinishThreads) {
      const float d = unit_distance(u);
      if (!(d >= 0.f && d <= most)) continue;
      const int k = u / a.C;
      if (sh.kind[k] == kEnded) {
        const int i = atomicAdd(&sh.parts, 1);
        if (i < kMaxParts) sh.part_list[i] = 4 * u;
        continue;
      }
      const float4 m = __ldcg(a.quarters + static_cast<long long>(b) * all + u);
      const float base = sh.base[k], top = sh.top[k];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float x = q == 0 ? m.x : q == 1 ? m.y : q == 2 ? m.z : m.w;
        if (x == -INFINITY || !(base + (top - x) <= most)) continue;
        const int i = atomicAdd(&sh.parts, 1);
        if (i < kMaxParts) sh.part_list[i] = 4 * u + q;
      }
    }
    __syncthreads();
    if (sh.parts > kMaxParts) return 0;
    // Lists the tokens. With fewer units than candidates wanted, or with too many tokens in that range, their own
    // distances are counted first and give a nearer edge.
    float limit = most;
    bool counting = edge == kBins - 1, counted = false;
    if (counting) {   // (the units' counts give way to the tokens')
      __syncthreads();
      clear_hist_only();
      __syncthreads();
    }
    for (;;) {
      each_token(limit, counting);
      __syncthreads();
      if (!counting && sh.cands <= kMaxCands) break;
      if (!counting && counted) return 0;
      if (counting) {
        find_edge(a.n);
        limit = bin_end(sh.edge + 1);
        counting = false;
        counted = true;
      } else {
        counting = true;
        __syncthreads();   // all have seen how many there were
        clear_hist_only();
        if (tid == 0) sh.cands = 0;
        __syncthreads();
      }
    }
    const int count = sh.cands;
    // Distances from the best score, which as a rule fit 64 bits; among equal ones: beam, logit (the largest first), token
    ulonglong2 mine = make_ulonglong2(0, 0);
    Cand c{0.f, 0, 0};
    float out = 0.f;
    bool far = false;
    if (tid < count) {
      c = sh.cand[tid];
      out = score_out(c);
      const Fixed d = sh.best_score - score(c.k, c.l);
      far = (d.mid | static_cast<unsigned long long>(d.hi)) != 0;
      mine = make_ulonglong2(d.lo, static_cast<unsigned long long>(c.k) << 52 |
                                       static_cast<unsigned long long>(~float_key(__fadd_rn(c.l, 0.f))) << 20 | c.at);
      sh.key[tid] = mine;
    }
    far = __syncthreads_or(far);
    int rank = 0;
    if (far) {
      rank = rank_far_apart<E>(a, sh, b, count);
    } else if (tid < count) {
#pragma unroll 4
      for (int i = 0; i < count; ++i) {
        const ulonglong2 x = sh.key[i];
        rank += x.x < mine.x || (x.x == mine.x && x.y < mine.y);
      }
    }
    if (tid < count) sh.order[rank] = tid;
    __syncthreads();
    if (tid > 0 && tid < count) {   // with the one before it; those not chosen with the last chosen one
      const int i = sh.order[min(tid, a.n) - 1], j = sh.order[tid];
      const Cand &p = sh.cand[i], &q = sh.cand[j];
      if (p.k != q.k)
        compare(far ? float_of(score(p.k, p.l) - score(q.k, q.l)) : static_cast<float>(sh.key[j].x - sh.key[i].x) * 0x1p-48f,
                p.k, q.k);
    }
    __syncthreads();
    if (sh.again) return -1;
    const long long row = static_cast<long long>(b) * a.n;
    if (tid < count && rank < a.n) {
      a.tokens[row + rank] = c.at;
      a.parents[row + rank] = b * a.K + c.k;
      a.out_scores[row + rank] = out;
    }
    if (tid >= count && tid < a.n) {
      a.tokens[row + tid] = a.parents[row + tid] = -1;
      a.out_scores[row + tid] = -INFINITY;
    }
    return 1;
  }

  // the best of this thread's units that ranks after `last` (none: of all)
  __device__ __forceinline__ Pick next_unit(const Pick &last) const {
    Pick best = no_pick();
    for (int u = tid; u < a.K * a.C; u += kFinishThreads) {
      const Pick p = unit_pick(u);
      if (p.some() && (!last.some() || before(last, p)) && before(p, best)) best = p;
    }
    return best;
  }

  // the best token of a chosen unit that ranks after (l, token); by one warp
  __device__ __forceinline__ void next_token(int j, float last_l, int last_t) const {
    const int u = sh.unit[j], k = u / a.C, chunk = u - k * a.C;
    float l = -INFINITY;
    int t = 0x7fffffff;
    if (sh.kind[k] == kEnded) {
      if (last_t < 0) {
        l = 0.f;
        t = a.pad;
      }
    } else {
      uint4 w[kVPL];
      load_groups<E>(row(k), a.V, chunk * kUnitVecs + lane, w);
#pragma unroll
      for (int v = 0; v < kVPL; ++v) {
        const int g = chunk * kUnitVecs + v * 32 + lane;
#pragma unroll
        for (int e = 0; e < Elem<E>::kPerVec; ++e) {
          const float x = vec_elem<E>(w[v], e);
          const int at = g * Elem<E>::kPerVec + e;
          const bool after = x < last_l || (x == last_l && at > last_t);
          if (x > -INFINITY && after && (x > l || (x == l && at < t))) {
            l = x;
            t = at;
          }
        }
      }
      const unsigned key = float_key(__fadd_rn(l, 0.f));
      const unsigned top = __reduce_max_sync(0xffffffffu, key);
      t = __reduce_min_sync(0xffffffffu, key == top ? t : 0x7fffffff);
      l = key_float(top);
    }
    if (lane == 0) {
      sh.head[j] = t != 0x7fffffff ? Pick{score(k, l), {l, k, t}} : no_pick();
    }
  }

  // The same for any numbers of equal candidates: units and then tokens one by one, each the best of what is
  // left. (4 x 8 beams x 32000 of one value each, 16 best: 179 us for 14.) False if
  // sums have to be improved first.
  __device__ bool select_any() const {
    // the n first units by their largest candidates: the n best candidates lie in them
    Pick last = no_pick();
    Pick mine = next_unit(last);
    int units = 0;
    for (; units < a.n; ++units) {
      const Pick w = warp_best(mine);
      if (lane == 0) sh.warp[warp] = w;
      __syncthreads();
      if (warp == 0) {
        const Pick all = warp_best(lane < kFinishWarps ? sh.warp[lane] : no_pick());
        if (lane == 0) {
          sh.best = all;
          if (units > 0 && all.some()) compare(float_of(last.score - all.score), last.c.k, all.c.k);
        }
      }
      __syncthreads();
      const Pick p = sh.best;
      if (!p.some()) break;
      if (tid == 0) sh.unit[units] = p.c.k * a.C + p.c.at;
      if (mine.c.k == p.c.k && mine.c.at == p.c.at) mine = next_unit(p);
      last = p;
    }
    if (units == a.n) {
      for (int u = tid; u < a.K * a.C; u += kFinishThreads) {
        const Pick p = unit_pick(u);
        if (p.some() && before(last, p)) compare(float_of(last.score - p.score), last.c.k, p.c.k);
      }
    }
    __syncthreads();
    if (sh.again) return false;
    for (int j = warp; j < units; j += kFinishWarps) next_token(j, INFINITY, -1);
    __syncthreads();
    int32_t *tokens = a.tokens + static_cast<long long>(b) * a.n;
    int32_t *parents = a.parents + static_cast<long long>(b) * a.n;
    float *scores = a.out_scores + static_cast<long long>(b) * a.n;
    Pick one_before = no_pick();
    int found = 0;
    for (; found < a.n; ++found) {
      Pick p = no_pick();   // every warp finds the best head by itself
      int j = 0;
      for (int i = lane; i < units; i += 32)
        if (before(sh.head[i], p)) p = sh.head[i];
      p = warp_best(p);
      if (!p.some()) break;
      const int k = p.c.k, token = p.c.at;
      const float l = p.c.l;
      while (sh.unit[j] != k * a.C + (sh.kind[k] == kEnded ? 0 : token / (kUnitVecs * Elem<E>::kPerVec))) ++j;
      if (tid == 0) {
        if (found > 0) compare(float_of(one_before.score - p.score), one_before.c.k, k);
        tokens[found] = token;
        parents[found] = b * a.K + k;
        scores[found] = score_out(p.c);
      }
      one_before = p;
      __syncthreads();
      if (warp == j % kFinishWarps) next_token(j, sh.kind[k] == kEnded ? -INFINITY : l, token);
      __syncthreads();
    }
    if (found == a.n)
      for (int j = tid; j < units; j += kFinishThreads)
        if (sh.head[j].some())
          compare(float_of(one_before.score - sh.head[j].score), one_before.c.k, sh.head[j].c.k);
    __syncthreads();
    if (sh.again) return false;
    for (int j = found + tid; j < a.n; j += kFinishThreads) {
      tokens[j] = parents[j] = -1;
      scores[j] = -INFINITY;
    }
    return true;
  }
};

template <typename E>
__device__ __forceinline__ Finish<E> finish_of(const BeamArgs &a, FinishShared &sh, int b) {
  const int tid = threadIdx.x;
  return Finish<E>{a, sh, b, tid, tid & 31, tid >> 5};
}
template <typename E>
__device__ __noinline__ float2 large_sum_apart(const BeamArgs &a, FinishShared &sh, int b, int k, float m) {
  return finish_of<E>(a, sh, b).large_sum(k, m);
}
template <typename E>
__device__ __noinline__ void refine_apart(const BeamArgs &a, FinishShared &sh, int b, int k) {
  finish_of<E>(a, sh, b).refine(k);
}
template <typename E>
__device__ __noinline__ int rank_far_apart(const BeamArgs &a, FinishShared &sh, int b, int count) {
  return finish_of<E>(a, sh, b).rank_far(count);
}
template <typename E>
__device__ __noinline__ bool select_any_apart(const BeamArgs &a, FinishShared &sh, int b) {
  return finish_of<E>(a, sh, b).select_any();
}

// One CTA a batch row.
template <typename E>
__global__ void __launch_bounds__(kFinishThreads, 1) beam_finish_kernel(const __grid_constant__ BeamArgs a) {
  __shared__ FinishShared sh;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, b = blockIdx.x;
  const Finish<E> f = finish_of<E>(a, sh, b);
  if (tid == 0) sh.bad = sh.again = 0;
  __syncthreads();
  f.sums();
  __syncthreads();
  if (sh.bad) {
    if (tid == 0) set_status(a.status, SPEC_ERR_NONFINITE);
    for (int j = tid; j < a.n; j += kFinishThreads) {
      const long long at = static_cast<long long>(b) * a.n + j;
      a.tokens[at] = a.parents[at] = -1;
      a.out_scores[at] = NAN;
    }
    return;
  }
  // Each time around, a beam that asks is improved, at most twice: to its target, below what it had, and then to kFine,
  // below which nothing is asked for. So it ends after 2 K at the latest.
  for (int round = 0; round <= 2 * SPEC_MAX_BEAMS; ++round) {
    const int done = f.select_few();
    if (done == 1) return;
    __syncthreads();
    if (done == 0 && select_any_apart<E>(a, sh, b)) return;
    __syncthreads();
    if (tid == 0) sh.again = 0;
    for (int k = 0; k < a.K; ++k)
      if (sh.target[k] != 0x7f800000) refine_apart<E>(a, sh, b, k);
    __syncthreads();
  }
}

// ------------------------------------------------------------------ reordering

// A CTA a (row, state), which is a launch's time for the beams of a batch (128 rows of 8 KB and of 2 KB: 3.5 us; few long
// rows leave most of the GPU idle: 4 of 2.5 MB 55 us): row c
// of each state from row parents[c] of the one before; zeros without a parent.
template <typename W>
__device__ __forceinline__ void copy_row(const char *from, char *to, long long bytes) {
  const long long n = bytes / static_cast<long long>(sizeof(W));
  for (long long i0 = threadIdx.x; i0 < n; i0 += 4 * 256) {
    W w[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i0 + u * 256 < n) w[u] = from ? reinterpret_cast<const W *>(from)[i0 + u * 256] : W{};
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i0 + u * 256 < n) reinterpret_cast<W *>(to)[i0 + u * 256] = w[u];
  }
}

__global__ void __launch_bounds__(256) beam_reorder_kernel(const __grid_constant__ ReorderArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x / a.states, s = blockIdx.x - c * a.states;
  const int p = ld_given(a.parents + c);
  const bool ok = p >= 0 && p < a.rows_in;
  if (!ok && p != -1 && threadIdx.x == 0) set_status(a.status, SPEC_ERR_PARENT);
  const long long bytes = a.bytes[s];
  const char *from = ok ? a.in[s] + p * bytes : nullptr;
  char *to = a.out[s] + c * bytes;
  switch (a.grain[s]) {
    case 16: copy_row<uint4>(from, to, bytes); break;
    case 8: copy_row<uint2>(from, to, bytes); break;
    case 4: copy_row<uint32_t>(from, to, bytes); break;
    case 2: copy_row<uint16_t>(from, to, bytes); break;
    default: copy_row<uint8_t>(from, to, bytes);
  }
}

template <typename E>
cudaError_t launch_select(const BeamArgs &a, int sms, cudaStream_t stream) {
  const int groups = (a.units + 7) / 8;
  const cudaError_t e = launch_kv(beam_stream_kernel<E>, groups < 4 * sms ? groups : 4 * sms, 256, 0, stream, a);
  return e != cudaSuccess ? e : launch_kv(beam_finish_kernel<E>, a.B, kFinishThreads, 0, stream, a);
}

}  // namespace

cudaError_t launch_beam_select(int dtype, const BeamArgs &a, int sms, cudaStream_t stream) {
  return dtype == SPEC_BF16 ? launch_select<uint16_t>(a, sms, stream) : launch_select<float>(a, sms, stream);
}

cudaError_t launch_beam_reorder(const ReorderArgs &a, cudaStream_t stream) {
  return launch_kv(beam_reorder_kernel, static_cast<long long>(a.rows_out) * a.states, 256, 0, stream, a);
}

}  // namespace specv
