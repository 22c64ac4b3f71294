// spec_kv_append.cu -- new tokens into the paged e4m3 cache (keys rotated by their positions, one
// power-of-two scale for each page and head, queries rotated beside them), and the accepted path of a
// verified tree moved to the front of the new tokens' slots.
//
// Appending reads 2 bytes an element and writes 1 (keys, values) or 2 (queries): HBM bounds long calls,
// latency short ones. The scale costs no second pass: a CTA holds a page's new rows of one head in
// registers, reduces their largest magnitude and writes them. It takes several heads of the page in
// turn (the next head's rows on their way meanwhile), so that the cosines and sines of its tokens,
// twice a head's bytes, are loaded once for all of them; calls with few pages give each head a CTA. The
// queries' warps take up to eight head groups of a token on the same cosines and sines. A page that held
// tokens has them stored again only when its scale grows.
#include "spec_kv.h"

namespace specv {

namespace {

constexpr int kQIters = 8;   // head groups of a query task

// The position of new token i of sequence b; a position outside the table is reported and read as 0.
__device__ __forceinline__ int kv_position(const KvArgs &a, const RopeArgs &r, int b, int i,
                                           int len) {
  long long pos;
  if (r.positions) {
    pos = ld_given(r.positions + static_cast<long long>(b) * a.N + i);
  } else if (a.mask) {   // ancestors and itself: depth + 1 bits
    int bits = 0;
    const uint32_t *row = a.mask + (static_cast<long long>(b) * a.N + i) * a.W;
    for (int w = 0; w < a.W; ++w) bits += __popc(ld_given(row + w));
    pos = static_cast<long long>(len) + (bits > 0 ? bits - 1 : 0);
  } else {
    pos = static_cast<long long>(len) + i;
  }
  if (pos < 0 || pos >= r.rows) {
    set_status(a.status, SPEC_ERR_POSITION);
    return 0;
  }
  return static_cast<int>(pos);
}

// A head's row is D / 16 units of two vectors of 8 elements. Unit u < R / 16 rotates by the cosines and
// sines 8 u .. 8 u + 7: its vectors are 8 u and R / 2 + 8 u (halves: partners), or 16 u and 16 u + 8
// (interleaved pairs: partners side by side). The others are what is left, two vectors side by side.
struct Unit {
  int a, b;    // first elements of its vectors
  bool turn;
};
__device__ __forceinline__ Unit unit_of(const RopeArgs &r, int u, bool rotate) {
  Unit x;
  x.turn = rotate && u < r.R / 16;
  if (x.turn && !r.pairs) {
    x.a = 8 * u;
    x.b = r.R / 2 + 8 * u;
  } else {
    x.a = 16 * u;
    x.b = 16 * u + 8;
  }
  return x;
}
struct Angles {
  float c[8], s[8];
};
__device__ __forceinline__ void load_angles(const RopeArgs &r, int pos, int u, Angles &t) {
  const float *row = r.rope + static_cast<long long>(pos) * r.R + 8 * u;
  if (r.vec4) {   // (R is a multiple of 16, so rows and halves are aligned when the table is)
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 c = __ldg(reinterpret_cast<const float4 *>(row + i));
      const float4 s = __ldg(reinterpret_cast<const float4 *>(row + r.R / 2 + i));
      t.c[i] = c.x, t.c[i + 1] = c.y, t.c[i + 2] = c.z, t.c[i + 3] = c.w;
      t.s[i] = s.x, t.s[i + 1] = s.y, t.s[i + 2] = s.z, t.s[i + 3] = s.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      t.c[i] = __ldg(row + i);
      t.s[i] = __ldg(row + r.R / 2 + i);
    }
  }
}
// x c + y s with one product rounded; within 1.5 units in the last place of the sum, whatever cancels
// (Kahan's, with the product's error); or as a 32-bit number that rounds to fewer bits as the exact sum does.
enum Turn { kRounded, kClose, kExact };
template <Turn kTurn>
__device__ __forceinline__ float turned(float x, float c, float y, float s) {
  const float w = y * s;
  if (kTurn == kRounded) return __fmaf_rn(x, c, w);
  const float ew = __fmaf_rn(y, s, -w);
  if (kTurn == kClose) return __fadd_rn(__fmaf_rn(x, c, w), ew);
  // both products with their errors (Dekker's, by FMA), the sum of the products with its (Knuth's)
  const float p = x * c, ep = __fmaf_rn(x, c, -p);
  const float sum = __fadd_rn(p, w), part = __fsub_rn(sum, p);
  const float es = __fadd_rn(__fsub_rn(p, __fsub_rn(sum, part)), __fsub_rn(w, part));
  const float err = __fadd_rn(es, __fadd_rn(ep, ew)), r = __fadd_rn(sum, err);
  if (!(fabsf(r) < INFINITY)) return sum;   // (the errors of an infinite sum are NaN)
  // a border is never met by rounding to it: what was rounded off moves such a number by a unit
  const float rest = __fsub_rn(err, __fsub_rn(r, sum));
  const int bits = __float_as_int(r);
  return (bits & 0x7ffff) || rest == 0.f ? r
                                         : __int_as_float(bits + ((rest > 0.f) == (r > 0.f) ? 1 : -1));
}
template <Turn kTurn>
__device__ __forceinline__ void rotate(const RopeArgs &r, const Angles &t, float (&f)[8],
                                       float (&g)[8]) {
  if (r.pairs) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = f[2 * i], y = f[2 * i + 1], z = g[2 * i], w = g[2 * i + 1];
      f[2 * i] = turned<kTurn>(x, t.c[i], -y, t.s[i]);
      f[2 * i + 1] = turned<kTurn>(y, t.c[i], x, t.s[i]);
      g[2 * i] = turned<kTurn>(z, t.c[4 + i], -w, t.s[4 + i]);
      g[2 * i + 1] = turned<kTurn>(w, t.c[4 + i], z, t.s[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = f[i], y = g[i];
      f[i] = turned<kTurn>(x, t.c[i], -y, t.s[i]);
      g[i] = turned<kTurn>(y, t.c[i], x, t.s[i]);
    }
  }
}

// Keys are rounded to 4 significant bits next, where a sum that is off by a unit or two in the last place
// puts about one element in a million on the other side of a border. Borders are multiples of 2^19 units,
// so a thread that holds a number within 4 units of one (one thread in 4000) turns its 16 again exactly.
// In a graph, 8 x 4096 tokens of 8 key and 32 query heads: 142 us, 136 without, 164 with every sum exact.
__device__ __forceinline__ bool near_border(const float (&f)[2][8]) {
  uint32_t least = 8;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    least = min(least, (__float_as_uint(f[i >> 3][i & 7]) + 4u) & 0x7ffffu);
  return least < 8;
}

// One warp's queries: token `task / blocks`, up to kQIters groups of 32 / (D / 16) heads.
template <typename T>
__device__ __forceinline__ void append_queries(const KvArgs &a, const RopeArgs &r, long long task,
                                               int lane) {
  const int upr = a.D / 16, per = 32 / upr;   // units of a row; heads of a group
  const int blocks = (a.Hq + per * kQIters - 1) / (per * kQIters);
  const long long token = task / blocks;
  if (token >= static_cast<long long>(a.B) * a.N) return;
  const int h0 = static_cast<int>(task - token * blocks) * per * kQIters + lane / upr;
  const int b = static_cast<int>(token / a.N);
  const int i = static_cast<int>(token - static_cast<long long>(b) * a.N);
  int len, n;
  if (!kv_lengths(a, b, len, n) || i >= n) return;
  const int u = lane % upr;
  const Unit x = unit_of(r, u, true);
  const T *src = static_cast<const T *>(r.q) + token * r.q_stride;
  T *dst = static_cast<T *>(r.q_out) + token * a.Hq * a.D;
  uint4 raw[kQIters][2];
#pragma unroll
  for (int k = 0; k < kQIters; ++k) {
    const int h = h0 + k * per;
    if (h < a.Hq) {
      // (plain loads: where q_out is q, the read-only path is not open to them)
      raw[k][0] = *reinterpret_cast<const uint4 *>(src + h * a.D + x.a);
      raw[k][1] = *reinterpret_cast<const uint4 *>(src + h * a.D + x.b);
    }
  }
  Angles t;
  if (x.turn) load_angles(r, kv_position(a, r, b, i, len), u, t);
  __syncwarp();   // q_out may be q: nothing of a row is stored before all of it is read
#pragma unroll
  for (int k = 0; k < kQIters; ++k) {
    const int h = h0 + k * per;
    if (h < a.Hq) {
      if (x.turn) {
        float f[8], g[8];
        vec_to_floats<T>(raw[k][0], f);
        vec_to_floats<T>(raw[k][1], g);
        rotate<kRounded>(r, t, f, g);
        raw[k][0] = floats_to_vec<T>(f);
        raw[k][1] = floats_to_vec<T>(g);
      }
      *reinterpret_cast<uint4 *>(dst + h * a.D + x.a) = raw[k][0];
      *reinterpret_cast<uint4 *>(dst + h * a.D + x.b) = raw[k][1];
    }
  }
}

// kU: units of a thread; kThreads * kU units cover a page of one head. Heads h0 .. h0 + hpc - 1 of a
// page, keys or values; the CTAs from `kv_ctas` on rotate queries.
template <typename T, int kU, int kThreads>
__global__ void __launch_bounds__(kThreads, 512 / kThreads)
    kv_append_kernel(const __grid_constant__ KvArgs a, const __grid_constant__ RopeArgs r, int hpc,
                     int kv_ctas) {
  __shared__ float warp_max[2][kThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x;
  if (static_cast<int>(blockIdx.x) >= kv_ctas) {
    const long long task = static_cast<long long>(blockIdx.x - kv_ctas) * (kThreads / 32) + (tid >> 5);
    append_queries<T>(a, r, task, tid & 31);
    return;
  }
  unsigned x = blockIdx.x;
  const int side = static_cast<int>(x & 1);
  x >>= 1;
  const unsigned groups = (a.Hkv + hpc - 1) / hpc;
  const int h0 = static_cast<int>(x % groups) * hpc;
  x /= groups;
  const int pi = static_cast<int>(x % r.touched);
  const int b = static_cast<int>(x / r.touched);
  int len, n;
  if (!kv_lengths(a, b, len, n)) {
    if (tid == 0) set_status(a.status, SPEC_ERR_LENGTH);
    return;
  }
  const int local = (len >> a.page_shift) + pi;
  const int p0 = local << a.page_shift;
  const int from = max(len, p0), to = min(len + n, p0 + a.page);   // the page's new tokens
  if (from >= to) return;
  int page;
  if (!kv_page(a, b, local, page)) {
    if (tid == 0) set_status(a.status, SPEC_ERR_PAGE);
    return;
  }
  const int upr = a.D / 16;
  const bool turning = side == 0 && r.R > 0;
  const T *src = static_cast<const T *>(side ? r.v : r.k);
  const long long stride = side ? r.v_stride : r.k_stride;
  Unit un[kU];
  int row[kU];        // of the page, or -1: nothing of this thread's
  const T *at[kU];
  Angles t[kU];
#pragma unroll
  for (int k = 0; k < kU; ++k) {
    const int id = k * kThreads + tid;
    row[k] = id / upr;
    un[k] = unit_of(r, id - row[k] * upr, turning);
    const int slot = p0 + row[k];
    at[k] = src + (static_cast<long long>(b) * a.N + (slot - len)) * stride;
    if (row[k] >= a.page) row[k] = -1;
    if (row[k] >= 0 && un[k].turn && slot >= from && slot < to)
      load_angles(r, kv_position(a, r, b, slot - len, len), id % upr, t[k]);
  }
  const int h1 = min(a.Hkv, h0 + hpc);
  uint4 raw[kU][2];
  auto fetch = [&](int h) {
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int slot = p0 + row[k];
      if (row[k] >= 0 && slot >= from && slot < to) {
        raw[k][0] = ld_given(reinterpret_cast<const uint4 *>(at[k] + h * a.D + un[k].a));
        raw[k][1] = ld_given(reinterpret_cast<const uint4 *>(at[k] + h * a.D + un[k].b));
      }
    }
  };
  fetch(h0);
  const bool held = from > p0;
  bool finite = true;
  for (int h = h0; h < h1; ++h) {
    const long long head = static_cast<long long>(page) * a.Hkv + h;
    float *scale = (side ? a.v_scale : a.k_scale) + head;
    uint8_t *dst = (side ? a.v : a.k) + (head << a.page_shift) * a.D;
    const float old = held ? *scale : 0.f;
    float f[kU][2][8];
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int slot = p0 + row[k];
      if (row[k] >= 0 && slot >= from && slot < to) {
        vec_to_floats<T>(raw[k][0], f[k][0]);
        vec_to_floats<T>(raw[k][1], f[k][1]);
        if (un[k].turn) {
          rotate<kClose>(r, t[k], f[k][0], f[k][1]);
          if (near_border(f[k])) {
            vec_to_floats<T>(raw[k][0], f[k][0]);
            vec_to_floats<T>(raw[k][1], f[k][1]);
            rotate<kExact>(r, t[k], f[k][0], f[k][1]);
          }
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float m = fabsf(f[k][e >> 3][e & 7]);
          const bool ok = m < INFINITY;   // false for NaN too
          finite = finite && ok;
          amax = fmaxf(amax, ok ? m : 0.f);
        }
      }
    }
    if (h + 1 < h1) fetch(h + 1);
    // magnitudes order like their bit patterns
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
    float *wm = warp_max[h & 1];   // the other half may still be read for the head before
    if ((tid & 31) == 0) wm[tid >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) amax = fmaxf(amax, wm[w]);
    const float s = fmaxf(kv_scale_for(amax), old);
    const float inv = 1.f / s;   // exact for a power of two
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      if (row[k] < 0 || !SPEC_CHECK(a, row[k] < a.page && head < static_cast<long long>(a.num_pages) * a.Hkv))
        continue;
      const int slot = p0 + row[k];
      uint2 *oa = reinterpret_cast<uint2 *>(dst + row[k] * a.D + un[k].a);
      uint2 *ob = reinterpret_cast<uint2 *>(dst + row[k] * a.D + un[k].b);
      if (slot >= from && slot < to) {
        const uint2 wa = floats_to_e4m3(f[k][0], inv), wb = floats_to_e4m3(f[k][1], inv);
        if (un[k].b == un[k].a + 8) {   // side by side: 16 bytes
          *reinterpret_cast<uint4 *>(oa) = make_uint4(wa.x, wa.y, wb.x, wb.y);
        } else {
          *oa = wa;
          *ob = wb;
        }
      } else if (held && s != old && slot < from) {   // the rows the page held, at the new scale
        float g[8];
        e4m3_to_floats(*oa, g);
        *oa = floats_to_e4m3(g, old / s);
        e4m3_to_floats(*ob, g);
        *ob = floats_to_e4m3(g, old / s);
      }
    }
    if (tid == 0 && s != old) *scale = s;
  }
  if (!finite) set_status(a.status, SPEC_ERR_NONFINITE);
}

template <typename T, int kU, int kThreads>
cudaError_t launch_append(const KvArgs &a, const RopeArgs &r, int hpc, cudaStream_t stream) {
  const int groups = (a.Hkv + hpc - 1) / hpc;
  const long long kv = 2LL * groups * r.touched * a.B;
  const int per = 32 / (a.D / 16) * kQIters;   // heads of a query task
  const long long tasks = static_cast<long long>(a.B) * a.N * ((a.Hq + per - 1) / per);
  const long long grid = kv + (tasks + kThreads / 32 - 1) / (kThreads / 32);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_kv(kv_append_kernel<T, kU, kThreads>, grid, kThreads, 0, stream, a, r, hpc,
                   static_cast<int>(kv));
}

template <typename T>
cudaError_t launch_append_for(const KvArgs &a, const RopeArgs &r, cudaStream_t stream) {
  // heads of a CTA: as many as leave about two CTAs for each SM
  int hpc = 1;
  while (hpc < a.Hkv && 2LL * a.B * r.touched * ((a.Hkv + 2 * hpc - 1) / (2 * hpc)) >= 304) hpc *= 2;
  const int units = a.page * a.D / 16;
  if (units <= 256) return launch_append<T, 1, 256>(a, r, hpc, stream);
  if (units <= 512) return launch_append<T, 2, 256>(a, r, hpc, stream);
  return launch_append<T, 2, 512>(a, r, hpc, stream);
}

// ------------------------------------------------------------------ the accepted path
//
// One warp per layer, sequence, head and side; a few rows of 64 or 128 bytes move, so the call is all
// latency, and many small tasks at once hide it (one CTA each, a page in registers, took 127 us for
// 32 trees in 32 layers of 8 heads). The path's nodes increase and node k of it is at least k, so moving
// rows forward in the order of k never overwrites a row still to be moved. Page by page of the
// destination: the largest magnitude of the rows that move there raises the page's scale if it must,
// the page is stored again when it did, and the rows are moved.
constexpr int kCommitWarps = 4;

__global__ void __launch_bounds__(32 * kCommitWarps)
    kv_commit_kernel(const __grid_constant__ KvArgs a, const int32_t *path_nodes,
                     const int32_t *accept_len, int32_t *out_lens, long long tasks) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  long long x = static_cast<long long>(blockIdx.x) * kCommitWarps + (threadIdx.x >> 5);
  if (x >= tasks) return;
  const int side = static_cast<int>(x & 1);
  x >>= 1;
  const int h = static_cast<int>(x % a.Hkv);
  x /= a.Hkv;
  const int b = static_cast<int>(x % a.B);
  const long long layer = x / a.B;
  const int len = ld_given(a.seq_lens + b), acc = ld_given(accept_len + b);
  const int32_t *path = path_nodes + static_cast<long long>(b) * a.N;
  bool bad = acc < -1 || acc >= a.N;
  bool moves = false;
  int top = 0;   // the path's last node
  if (!bad) {
    for (int k = lane; k <= acc; k += 32) {
      const int p = ld_given(path + k);
      bad = bad || (k == 0 ? p != 0 : p <= ld_given(path + k - 1)) || p >= a.N;
      moves = moves || p != k;
      top = max(top, p);
    }
  }
  bad = __any_sync(0xffffffffu, bad);
  moves = __any_sync(0xffffffffu, moves);
  top = __reduce_max_sync(0xffffffffu, top);
  const bool len_ok = len >= 0 && (bad || acc < 0 ||
                                   static_cast<long long>(len) + top <
                                       (static_cast<long long>(a.pps) << a.page_shift));
  if (side == 0 && h == 0 && layer == 0 && lane == 0) {
    if (!len_ok) set_status(a.status, SPEC_ERR_LENGTH);
    if (bad) set_status(a.status, SPEC_ERR_PATH);
    out_lens[b] = len_ok && !bad ? len + acc + 1 : len;
  }
  if (!len_ok || bad || !moves) return;
  const int dv = a.D / 8, per = 32 / dv;   // lanes of a row; rows at a time
  const int sub = lane / dv, d0 = lane % dv * 8;
  const long long layer_heads = layer * a.num_pages * a.Hkv;
  float *scales = (side ? a.v_scale : a.k_scale) + layer_heads;
  uint8_t *pool = (side ? a.v : a.k) + (layer_heads << a.page_shift) * a.D;
  for (int local = len >> a.page_shift; (local << a.page_shift) <= len + acc; ++local) {
    const int p0 = local << a.page_shift;
    const int k0 = max(0, p0 - len), k1 = min(acc + 1, p0 + a.page - len);   // path nodes that end here
    int page;
    if (!kv_page(a, b, local, page)) {
      if (lane == 0) set_status(a.status, SPEC_ERR_PAGE);
      continue;
    }
    const long long head = static_cast<long long>(page) * a.Hkv + h;
    uint8_t *dst = pool + (head << a.page_shift) * a.D;
    const float old = scales[head];
    float s = old;   // the page's scale
    // node k's row, dequantised; false if it stays where it is or its page is bad
    auto source = [&](int k, float (&f)[8]) {
      if (k >= k1) return false;
      const int node = ld_given(path + k);
      if (node == k) return false;
      const int slot = len + node;
      int spage;
      if (!kv_page(a, b, slot >> a.page_shift, spage)) {
        set_status(a.status, SPEC_ERR_PAGE);
        return false;
      }
      const long long shead = static_cast<long long>(spage) * a.Hkv + h;
      e4m3_to_floats(*reinterpret_cast<const uint2 *>(
                         pool + ((shead << a.page_shift) + (slot & (a.page - 1))) * a.D + d0),
                     f);
      const float m = spage == page ? s : scales[shead];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= m;
      return true;
    };
    float f[8];
    float amax = 0.f;
    bool any = false, mine = false;
    for (int k = k0; k < k1; k += per) {
      mine = source(k + sub, f);
      any = any || mine;
      if (mine)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float m = fabsf(f[e]);
          amax = fmaxf(amax, m < INFINITY ? m : 0.f);
        }
    }
    if (!__any_sync(0xffffffffu, any)) continue;
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
    s = fmaxf(kv_scale_for(amax), old);
    if (s != old) {   // the page at its new scale, rows still to be moved from it too
      __syncwarp();
      for (int r = sub; r < a.page; r += per) {
        uint2 *at = reinterpret_cast<uint2 *>(dst + r * a.D + d0);
        float g[8];
        e4m3_to_floats(*at, g);
        *at = floats_to_e4m3(g, old / s);
      }
      if (lane == 0) scales[head] = s;
      __syncwarp();
    }
    const float inv = 1.f / s;
    const bool kept = k1 - k0 <= per && s == old;   // the rows are still in the registers
    for (int k = k0; k < k1; k += per) {
      if (!kept) mine = source(k + sub, f);
      __syncwarp();   // every row of the step is read before any is written
      if (mine && SPEC_CHECK(a, len + k + sub >= p0 && len + k + sub < p0 + a.page))
        *reinterpret_cast<uint2 *>(dst + (len + k + sub - p0) * a.D + d0) = floats_to_e4m3(f, inv);
      __syncwarp();
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvArgs &a, const RopeArgs &r, int dtype, cudaStream_t stream) {
  return dtype == SPEC_BF16 ? launch_append_for<__nv_bfloat16>(a, r, stream)
                            : launch_append_for<__half>(a, r, stream);
}

cudaError_t launch_kv_commit(const KvArgs &a, int layers, const int32_t *path,
                             const int32_t *accept, int32_t *out_lens, cudaStream_t stream) {
  const long long tasks = 2LL * a.Hkv * a.B * layers;
  const long long grid = (tasks + kCommitWarps - 1) / kCommitWarps;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_kv(kv_commit_kernel, grid, 32 * kCommitWarps, 0, stream, a, path, accept, out_lens,
                   tasks);
}

}  // namespace specv
