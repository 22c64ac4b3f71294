// spec_kv_append.cu -- new tokens into the paged e4m3 cache: keys rotated by their positions, one
// power-of-two scale for each page and head, queries rotated beside them.
//
// One CTA per page that a sequence's new tokens touch, head, and side (keys or values): the CTA
// holds the page's new rows in registers (one read of 2 bytes an element), reduces their largest
// magnitude, and writes them as e4m3 at the page's scale (one byte an element), so the scale costs
// no second pass. A page that held tokens has them stored again only when its scale grows. Further
// CTAs rotate the queries. Nothing here is a contraction: HBM bounds long calls, latency short ones.
#include "spec_kv.cuh"

namespace specv {

namespace {

constexpr int kAppendThreads = 256;
constexpr int kQVecs = 4;   // query vectors (8 elements) per thread

// The position of new token i of sequence b; a position outside the table is reported and read as 0.
__device__ __forceinline__ int kv_position(const KvArgs &a, const RopeArgs &r, int b, int i,
                                           int len) {
  long long pos;
  if (r.positions) {
    pos = __ldg(r.positions + static_cast<long long>(b) * a.N + i);
  } else if (a.mask) {   // ancestors and itself: depth + 1 bits
    int bits = 0;
    const uint32_t *row = a.mask + (static_cast<long long>(b) * a.N + i) * a.W;
    for (int w = 0; w < a.W; ++w) bits += __popc(__ldg(row + w));
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

// Elements d0 .. d0 + 7 of one head's row of a token (at `row`), rotated by table row `pos`.
// Halves: the partner of element j < R/2 is j + R/2, eight of which are a vector of their own
// (R is a multiple of 16). Pairs: both partners lie in the vector.
template <typename T>
__device__ __forceinline__ void load_rotated(const RopeArgs &r, const T *row, int d0, int pos,
                                             float (&f)[8]) {
  vec_to_floats<T>(__ldg(reinterpret_cast<const uint4 *>(row + d0)), f);
  if (d0 >= r.R) return;
  const float *cs = r.rope + static_cast<long long>(pos) * r.R;
  const int half = r.R / 2;
  if (r.pairs) {
    // R / 2 is a multiple of 8 and d0 / 2 of 4: 16-byte aligned when the table is; the table is
    // only known to be 4-byte aligned, so scalar loads
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float c = __ldg(cs + d0 / 2 + i), s = __ldg(cs + half + d0 / 2 + i);
      const float x = f[2 * i], y = f[2 * i + 1];
      f[2 * i] = __fmaf_rn(x, c, -(y * s));
      f[2 * i + 1] = __fmaf_rn(y, c, x * s);
    }
  } else {
    const bool up = d0 >= half;
    const int j0 = up ? d0 - half : d0;
    float g[8];
    vec_to_floats<T>(__ldg(reinterpret_cast<const uint4 *>(row + (up ? j0 : j0 + half))), g);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = __ldg(cs + j0 + i), s = __ldg(cs + half + j0 + i);
      f[i] = up ? __fmaf_rn(f[i], c, g[i] * s) : __fmaf_rn(f[i], c, -(g[i] * s));
    }
  }
}

// kV: vectors of 8 elements per thread that cover a page of one head
template <typename T, int kV>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(KvArgs a, RopeArgs r) {
  __shared__ float warp_max[kAppendThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x;
  const int dv = a.D / 8;   // vectors per row
  const long long kv_ctas = 2LL * a.Hkv * r.touched * a.B;
  if (blockIdx.x >= kv_ctas) {   // queries
    const long long first = (blockIdx.x - kv_ctas) * kAppendThreads * kQVecs;
    const T *q = static_cast<const T *>(r.q);
    T *qo = static_cast<T *>(r.q_out);
    float f[kQVecs][8];
    long long at[kQVecs];
#pragma unroll
    for (int u = 0; u < kQVecs; ++u) {   // all loads before the stores: q_out may be q
      const long long vec = first + u * kAppendThreads + tid;
      at[u] = -1;
      if (vec >= r.q_vecs) continue;
      const long long rowh = vec / dv;   // (token, head)
      const int d0 = static_cast<int>(vec - rowh * dv) * 8;
      const long long token = rowh / a.Hq;
      const int h = static_cast<int>(rowh - token * a.Hq);
      const int b = static_cast<int>(token / a.N), i = static_cast<int>(token - static_cast<long long>(b) * a.N);
      int len, n;
      if (!kv_lengths(a, b, len, n) || i >= n) continue;
      const int pos = r.R ? kv_position(a, r, b, i, len) : 0;
      load_rotated<T>(r, q + token * r.q_stride + static_cast<long long>(h) * a.D, d0, pos, f[u]);
      at[u] = vec * 8;
    }
    __syncwarp();   // a head's row is within one warp: nothing of it is stored before all is read
#pragma unroll
    for (int u = 0; u < kQVecs; ++u)
      if (at[u] >= 0) *reinterpret_cast<uint4 *>(qo + at[u]) = floats_to_vec<T>(f[u]);
    return;
  }
  // one page of one head: keys (side 0) or values
  long long x = blockIdx.x;
  const int side = static_cast<int>(x & 1);
  x >>= 1;
  const int h = static_cast<int>(x % a.Hkv);
  x /= a.Hkv;
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
  const T *src = static_cast<const T *>(side ? r.v : r.k);
  const long long stride = side ? r.v_stride : r.k_stride;
  const bool turn = side == 0 && r.R > 0;
  const long long head = static_cast<long long>(page) * a.Hkv + h;
  float *scale = (side ? a.v_scale : a.k_scale) + head;
  uint8_t *dst = (side ? a.v : a.k) + (head << a.page_shift) * a.D;
  const bool held = from > p0;
  const float old = held ? *scale : 0.f;
  float f[kV][8];
  float amax = 0.f;
  bool finite = true;
#pragma unroll
  for (int u = 0; u < kV; ++u) {
    const int vec = u * kAppendThreads + tid;
    const int row = vec / dv, d0 = (vec - row * dv) * 8, t = p0 + row;
    if (row < a.page && t >= from && t < to) {
      const int i = t - len;
      const long long token = static_cast<long long>(b) * a.N + i;
      const T *at = src + token * stride + static_cast<long long>(h) * a.D;
      if (turn)
        load_rotated<T>(r, at, d0, kv_position(a, r, b, i, len), f[u]);
      else
        vec_to_floats<T>(__ldg(reinterpret_cast<const uint4 *>(at + d0)), f[u]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float m = fabsf(f[u][e]);
        const bool ok = m < INFINITY;   // false for NaN too
        finite = finite && ok;
        amax = fmaxf(amax, ok ? m : 0.f);
      }
    }
  }
  if (!finite) set_status(a.status, SPEC_ERR_NONFINITE);
  // magnitudes order like their bit patterns
  amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
  if ((tid & 31) == 0) warp_max[tid >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kAppendThreads / 32; ++w) amax = fmaxf(amax, warp_max[w]);
  const float s = fmaxf(kv_scale_for(amax), old);
  const float inv = 1.f / s;   // exact for a power of two
#pragma unroll
  for (int u = 0; u < kV; ++u) {
    const int vec = u * kAppendThreads + tid;
    const int row = vec / dv, d0 = (vec - row * dv) * 8, t = p0 + row;
    uint2 *out = reinterpret_cast<uint2 *>(dst + row * a.D + d0);
    if (row < a.page && t >= from && t < to) {
      *out = floats_to_e4m3(f[u], inv);
    } else if (held && s != old && t < from) {   // the rows the page held, at the new scale
      float g[8];
      e4m3_to_floats(*out, g);
      *out = floats_to_e4m3(g, old / s);
    }
  }
  if (tid == 0 && s != old) *scale = s;
}

template <typename T>
cudaError_t launch_append(const KvArgs &a, const RopeArgs &r, cudaStream_t stream) {
  const long long grid = 2LL * a.Hkv * r.touched * a.B +
                         (r.q_vecs + kAppendThreads * kQVecs - 1) / (kAppendThreads * kQVecs);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const int vecs = a.page * a.D / 8;
  if (vecs <= kAppendThreads)
    return launch_kv(kv_append_kernel<T, 1>, grid, kAppendThreads, 0, stream, a, r);
  if (vecs <= 2 * kAppendThreads)
    return launch_kv(kv_append_kernel<T, 2>, grid, kAppendThreads, 0, stream, a, r);
  if (vecs <= 4 * kAppendThreads)
    return launch_kv(kv_append_kernel<T, 4>, grid, kAppendThreads, 0, stream, a, r);
  return launch_kv(kv_append_kernel<T, 8>, grid, kAppendThreads, 0, stream, a, r);
}

// ------------------------------------------------------------------ the accepted path
//
// One CTA per layer, sequence, head and side. The path's nodes increase and node k of it is at
// least k, so moving rows forward in the order of k never overwrites a row still to be moved. Page
// by page of the destination: the rows that move there are read into registers (dequantised),
// their largest magnitude raises the page's scale if it must, the rest of the page is stored again
// when it did, and the rows are written.
__global__ void __launch_bounds__(kAppendThreads)
    kv_commit_kernel(KvArgs a, const int32_t *path_nodes, const int32_t *accept_len,
                     int32_t *out_lens) {
  __shared__ float warp_max[kAppendThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x;
  long long x = blockIdx.x;
  const int side = static_cast<int>(x & 1);
  x >>= 1;
  const int h = static_cast<int>(x % a.Hkv);
  x /= a.Hkv;
  const int b = static_cast<int>(x % a.B);
  const long long layer = x / a.B;
  const bool first = side == 0 && h == 0 && layer == 0;
  const int len = __ldg(a.seq_lens + b), acc = __ldg(accept_len + b);
  const int32_t *path = path_nodes + static_cast<long long>(b) * a.N;
  bool bad = acc < -1 || acc >= a.N;
  if (!bad)
    for (int k = tid; k <= acc; k += kAppendThreads) {
      const int p = __ldg(path + k);
      bad = bad || (k == 0 ? p != 0 : p <= __ldg(path + k - 1)) || p >= a.N;
    }
  bad = __syncthreads_or(bad) != 0;
  const long long last = bad || acc < 0 ? 0 : static_cast<long long>(len) + __ldg(path + acc);
  const bool len_ok = len >= 0 && last < (static_cast<long long>(a.pps) << a.page_shift);
  if (first && tid == 0) {
    if (!len_ok) set_status(a.status, SPEC_ERR_LENGTH);
    if (bad) set_status(a.status, SPEC_ERR_PATH);
    out_lens[b] = len_ok && !bad ? len + acc + 1 : len;
  }
  if (!len_ok || bad || acc < 1) return;
  const int dv = a.D / 8;
  const long long layer_heads = layer * a.num_pages * a.Hkv;
  float *scales = (side ? a.v_scale : a.k_scale) + layer_heads;
  uint8_t *pool = (side ? a.v : a.k) + (layer_heads << a.page_shift) * a.D;
  for (int local = len >> a.page_shift; (local << a.page_shift) <= len + acc; ++local) {
    const int p0 = local << a.page_shift;
    int page;
    if (!kv_page(a, b, local, page)) {
      if (tid == 0) set_status(a.status, SPEC_ERR_PAGE);
      continue;
    }
    const long long head = static_cast<long long>(page) * a.Hkv + h;
    uint8_t *dst = pool + (head << a.page_shift) * a.D;
    const float old = scales[head];
    float f[8][8];   // up to 128 rows of 128 elements: 8 vectors a thread
    uint32_t moves = 0;
    float amax = 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int vec = u * kAppendThreads + tid;
      const int row = vec / dv, d0 = (vec - row * dv) * 8, k = p0 + row - len;
      if (row >= a.page || k < 0 || k > acc) continue;
      const int from = len + __ldg(path + k);
      if (from == p0 + row) continue;
      int spage;
      if (!kv_page(a, b, from >> a.page_shift, spage)) {
        set_status(a.status, SPEC_ERR_PAGE);
        continue;
      }
      const long long shead = static_cast<long long>(spage) * a.Hkv + h;
      const float ss = scales[shead];
      e4m3_to_floats(*reinterpret_cast<const uint2 *>(
                         pool + ((shead << a.page_shift) + (from & (a.page - 1))) * a.D + d0),
                     f[u]);
      moves |= 1u << u;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        f[u][e] *= ss;
        const float m = fabsf(f[u][e]);
        amax = fmaxf(amax, m < INFINITY ? m : 0.f);
      }
    }
    if (!__syncthreads_or(moves != 0)) continue;
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
    if ((tid & 31) == 0) warp_max[tid >> 5] = amax;
    __syncthreads();   // every source row is in registers
#pragma unroll
    for (int w = 0; w < kAppendThreads / 32; ++w) amax = fmaxf(amax, warp_max[w]);
    const float s = fmaxf(kv_scale_for(amax), old);
    const float inv = 1.f / s;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int vec = u * kAppendThreads + tid;
      const int row = vec / dv, d0 = (vec - row * dv) * 8;
      if (row >= a.page) continue;
      uint2 *out = reinterpret_cast<uint2 *>(dst + row * a.D + d0);
      if (moves >> u & 1u) {
        *out = floats_to_e4m3(f[u], inv);
      } else if (s != old) {
        float g[8];
        e4m3_to_floats(*out, g);
        *out = floats_to_e4m3(g, old / s);
      }
    }
    if (tid == 0 && s != old) scales[head] = s;
    __syncthreads();   // the next page may read rows of this one
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvArgs &a, const RopeArgs &r, int dtype, cudaStream_t stream) {
  return dtype == SPEC_BF16 ? launch_append<__nv_bfloat16>(a, r, stream)
                            : launch_append<__half>(a, r, stream);
}

cudaError_t launch_kv_commit(const KvArgs &a, int layers, const int32_t *path,
                             const int32_t *accept, int32_t *out_lens, cudaStream_t stream) {
  const long long grid = 2LL * a.Hkv * a.B * layers;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_kv(kv_commit_kernel, grid, kAppendThreads, 0, stream, a, path, accept, out_lens);
}

}  // namespace specv
