// spec_kv_pages.cu -- the pages of the KV cache: which are free, which sequences hold them, and moving
// their contents. refs[p] counts the places of page tables that hold page p; a page with 0 is free, and
// that is all the state there is: whoever needs a page takes the lowest free one, in the order of
// (sequence, place), so the results do not depend on timing and the pool stays dense.
//
// Reference counts change by integer atomics, whose order does not show. Lists (free pages, pages to copy)
// are made by prefix sums in the order of page numbers, by one CTA: its steps wait for one another, not for
// bandwidth (a reservation for 16 sequences takes 5.6 us, for 256 x 64 tokens 9; where the free
// pages are the last of 250 000, 61 steps of 4096, about 50).
//
// Contents move at HBM's rate: 48 copies of up to 63 rows in 32 layers, 220 MB read and written, 32 us (6.9 TB/s); 391
// pages of 64 tokens in 16 layers, 1.64 GB, 255 to 262 us (6.3 TB/s; 16 KB a step instead of 32 267).
#include "spec_kv.h"

namespace specv {

namespace {

constexpr int kScanThreads = 1024;
constexpr int kScanWarps = kScanThreads / 32;

__device__ __forceinline__ void pdl_wait() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Exclusive prefix of v over the block's threads, and the block's total; `sums` holds a word a warp.
__device__ __forceinline__ int block_prefix(int v, int *sums, int &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();   // the sums of the time before have been read
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  const int mine = lane < kScanWarps ? sums[lane] : 0;
  int all = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, all, o);
    if (lane >= o) all += y;
  }
  total = __shfl_sync(0xffffffffu, all, 31);
  const int before = __shfl_sync(0xffffffffu, all - mine, warp);
  return before + incl - v;
}

// refs[page] -= 1; a page that nothing held stays at 0 and is reported
__device__ __forceinline__ void drop_ref(const PageArgs &a, int page) {
  if (page >= a.num_pages) {
    set_status(a.status, SPEC_ERR_PAGE);
    return;
  }
  if (atomicSub(a.refs + page, 1) <= 0) {
    atomicAdd(a.refs + page, 1);
    set_status(a.status, SPEC_ERR_REFS);
  }
}

__device__ __forceinline__ bool length_ok(const PageArgs &a, int len) {
  return len >= 0 && len <= (static_cast<long long>(a.pps) << a.page_shift);
}

// ------------------------------------------------------------------ giving pages back

// One CTA a sequence. window 0: every page of a sequence that has ended. Else the pages that lie wholly
// behind the window of the next token (their last slot is at most len - window) and not among the sinks',
// and those past the last token.
__global__ void __launch_bounds__(128) kv_release_kernel(const __grid_constant__ PageArgs a,
                                                         const int32_t *ended, int32_t *lens_io,
                                                         int window, int sinks) {
  pdl_wait();
  const int b = blockIdx.x;
  int32_t *row = a.table + static_cast<long long>(b) * a.pps;
  int lo = 0, hi = a.pps, tail = a.pps;   // places [lo, hi) and [tail, pps) go
  if (window == 0) {
    if (ended && !ld_given(ended + b)) return;
    if (threadIdx.x == 0) lens_io[b] = 0;
  } else {
    const int len = ld_given(a.seq_lens + b);
    if (!length_ok(a, len)) {
      if (threadIdx.x == 0) set_status(a.status, SPEC_ERR_LENGTH);
      return;
    }
    lo = static_cast<int>((static_cast<unsigned>(sinks) + a.page - 1) >> a.page_shift);
    hi = len - window + 1 > 0 ? (len - window + 1) >> a.page_shift : 0;
    tail = static_cast<int>((static_cast<unsigned>(len) + a.page - 1) >> a.page_shift);
  }
  for (int j = threadIdx.x; j < a.pps; j += blockDim.x) {
    if (!((j >= lo && j < hi) || j >= tail)) continue;
    const int page = row[j];
    if (page < 0) continue;
    row[j] = -1;
    drop_ref(a, page);
  }
}

// ------------------------------------------------------------------ taking pages

// The first `want` free pages (refs 0) in increasing order, to list[]; returns how many there are, at most
// `want`. Called by all threads of one CTA; the list is visible to them on return.
__device__ int lowest_free(const PageArgs &a, int want, int32_t *list, int *sums) {
  int found = 0;
  for (int p0 = 0; p0 < a.num_pages && found < want; p0 += 4 * kScanThreads) {
    const int p = p0 + 4 * threadIdx.x;
    bool free[4];
    int n = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      free[e] = p + e < a.num_pages && __ldcg(a.refs + p + e) == 0;
      n += free[e];
    }
    int total;
    int at = found + block_prefix(n, sums, total);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (free[e]) {
        if (at < want) list[at] = p + e;
        ++at;
      }
    found += total;
  }
  __syncthreads();
  return min(found, want);
}

// One CTA. Item i of the call is place i % touched of those that sequence i / touched's new tokens can touch;
// items without a page (or with an entry past the pool, which is reported) are numbered in order, and number r gets the
// r-th free page. A sequence whose last number is past the free pages gets none.
__global__ void __launch_bounds__(kScanThreads) kv_reserve_kernel(const __grid_constant__ PageArgs a,
                                                                  const int32_t *new_lens, int N,
                                                                  int touched, int32_t *granted,
                                                                  int32_t *list) {
  extern __shared__ int seq_end[];   // [B] numbers given out up to and with sequence b
  __shared__ int sums[kScanWarps];
  pdl_wait();
  const int tid = threadIdx.x;
  const int items = a.B * touched;
  // the item's place in the table if it lacks a page, else -1
  auto lacks = [&](int i) -> long long {
    const int b = i / touched, j = i - b * touched;
    const int len = ld_given(a.seq_lens + b), n = new_lens ? ld_given(new_lens + b) : N;
    if (n <= 0 || n > N || len < 0 || !length_ok(a, len) || !length_ok(a, len + n)) return -1;
    const int place = (len >> a.page_shift) + j;
    if (place > (len + n - 1) >> a.page_shift) return -1;
    const long long at = static_cast<long long>(b) * a.pps + place;
    const int page = a.table[at];
    if (page >= a.num_pages) set_status(a.status, SPEC_ERR_PAGE);
    return page < 0 || page >= a.num_pages ? at : -1;
  };
  int total = 0;
  for (int i0 = 0; i0 < items; i0 += kScanThreads) {
    const int i = i0 + tid;
    const bool want = i < items && lacks(i) >= 0;
    int sum;
    const int at = total + block_prefix(want, sums, sum);
    if (i < items && i % touched == touched - 1) seq_end[i / touched] = at + want;
    total += sum;
  }
  const int have = lowest_free(a, total, list, sums);
  int base = 0;
  for (int i0 = 0; i0 < items; i0 += kScanThreads) {
    const int i = i0 + tid;
    const long long place = i < items ? lacks(i) : -1;
    int sum;
    const int at = base + block_prefix(place >= 0, sums, sum);
    if (place >= 0 && seq_end[i / touched] <= have && SPEC_CHECK(a, at < a.num_pages)) {
      const int page = list[at];
      a.table[place] = page;
      a.refs[page] = 1;
    }
    base += sum;
  }
  for (int b = tid; b < a.B; b += kScanThreads) {
    const int len = ld_given(a.seq_lens + b), n = new_lens ? ld_given(new_lens + b) : N;
    int g = n;
    if (n < 0 || n > N || len < 0 || !length_ok(a, len) || !length_ok(a, len + n)) {
      set_status(a.status, SPEC_ERR_LENGTH);
      g = 0;
    } else if (seq_end[b] > have && seq_end[b] > (b > 0 ? seq_end[b - 1] : 0)) {
      set_status(a.status, SPEC_ERR_NO_PAGE);
      g = 0;
    }
    granted[b] = g;
  }
}

// ------------------------------------------------------------------ forking

// What becomes of a parent's pages: `full` of them are shared, the one after holds `rest` tokens.
struct Parent {
  int len, full, rest;
  bool ok;
};
__device__ __forceinline__ Parent parent_of(const PageArgs &a, int p) {
  Parent x;
  x.len = ld_given(a.seq_lens + p);
  x.ok = length_ok(a, x.len);
  x.full = x.ok ? x.len >> a.page_shift : 0;
  x.rest = x.ok ? x.len & (a.page - 1) : 0;
  return x;
}

// A child's row of full pages, by threads `me`, `me` + `step`, ... (the place after them is left to fork_pages).
__device__ __forceinline__ void fork_child(const PageArgs &a, const ForkArgs &f, int c, int me, int step) {
  const int p = ld_given(f.parents + c);
  Parent x{};
  x.ok = p >= 0 && p < a.B;
  if (x.ok) x = parent_of(a, p);
  if (me == 0) {
    if (p < -1 || p >= a.B) set_status(a.status, SPEC_ERR_PARENT);
    if (p >= 0 && p < a.B && !x.ok) set_status(a.status, SPEC_ERR_LENGTH);
    f.lens_out[c] = x.ok ? x.len : p == -1 ? 0 : -1;
  }
  const int32_t *row = a.table + static_cast<long long>(x.ok ? p : 0) * a.pps;
  int32_t *out = f.table_out + static_cast<long long>(c) * a.pps;
  for (int j = me; j < a.pps; j += step) {
    if (x.rest && j == x.full) continue;
    int page = j < x.full ? row[j] : -1;
    if (page >= a.num_pages) {
      set_status(a.status, SPEC_ERR_PAGE);
      page = -1;
    }
    out[j] = max(page, -1);
  }
}
// A parent's pages, whose counts grow by the n children that share them and shrink by one where the parent ends.
__device__ __forceinline__ void fork_parent(const PageArgs &a, const ForkArgs &f, int p, int n, int me,
                                            int step) {
  const Parent x = parent_of(a, p);
  if (!x.ok && f.release && me == 0) set_status(a.status, SPEC_ERR_LENGTH);   // (else its children say so)
  const int32_t *row = a.table + static_cast<long long>(p) * a.pps;
  for (int j = me; j < a.pps; j += step) {
    const int page = row[j];
    if (page < 0) continue;
    if (page >= a.num_pages) {
      if (f.release) set_status(a.status, SPEC_ERR_PAGE);
      continue;
    }
    // a page that is not full goes over to the first child of a parent that ends
    int by = x.ok && j < x.full ? n - f.release : f.release && !(x.rest && j == x.full && n) ? -1 : 0;
    if (by == 0) continue;
    const int old = atomicAdd(a.refs + page, by);
    if (old + by < 0) {
      atomicAdd(a.refs + page, -by);
      set_status(a.status, SPEC_ERR_REFS);
    }
  }
}

// CTAs 0 .. C - 1: a child each; the others a parent.
__global__ void __launch_bounds__(128) kv_fork_rows_kernel(const __grid_constant__ PageArgs a,
                                                           const __grid_constant__ ForkArgs f) {
  pdl_wait();
  __shared__ int children;
  if (blockIdx.x < static_cast<unsigned>(f.C)) {
    fork_child(a, f, blockIdx.x, threadIdx.x, blockDim.x);
    return;
  }
  const int p = blockIdx.x - f.C;
  if (threadIdx.x == 0) children = 0;
  __syncthreads();
  int n = 0;
  for (int c = threadIdx.x; c < f.C; c += blockDim.x) n += ld_given(f.parents + c) == p;
  if (n) atomicAdd(&children, n);
  __syncthreads();
  fork_parent(a, f, p, children, threadIdx.x, blockDim.x);
}

// One CTA: pages for the children that need a copy of the last page, in the order of the children, and the
// list of copies. A child that finds no page has none (its length is -1). kAll: it does the rows too, a warp a
// sequence: a launch less, which is worth it for up to kForkOne sequences, two a warp (4 beams: 10 us less of the
// host's time; 256 sequences of 9 pages take 7 us longer that way).
constexpr int kForkOne = 64, kForkPlaces = 1024;
template <bool kAll>
__global__ void __launch_bounds__(kScanThreads) kv_fork_pages_kernel(const __grid_constant__ PageArgs a,
                                                                     const __grid_constant__ ForkArgs f) {
  extern __shared__ int first[];   // [B] the first child of each parent; then, with kAll, their numbers
  __shared__ int sums[kScanWarps];
  pdl_wait();
  const int tid = threadIdx.x;
  int *children = first + a.B;
  for (int p = tid; p < a.B; p += kScanThreads) {
    first[p] = f.C;
    if (kAll) children[p] = 0;
  }
  __syncthreads();
  if (f.release || kAll)
    for (int c = tid; c < f.C; c += kScanThreads) {
      const int p = ld_given(f.parents + c);
      if (p < 0 || p >= a.B) continue;
      if (f.release) atomicMin(&first[p], c);
      if (kAll) atomicAdd(&children[p], 1);
    }
  if (kAll) {
    __syncthreads();
    const int lane = tid & 31, warp = tid >> 5;
    for (int i = warp; i < f.C + a.B; i += kScanWarps)
      if (i < f.C)
        fork_child(a, f, i, lane, 32);
      else
        fork_parent(a, f, i - f.C, children[i - f.C], lane, 32);
  }
  __syncthreads();
  struct Child {
    int p, src;   // src: the parent's last page if it is not full, else -1
    Parent x;
    bool copies;
  };
  auto child = [&](int c) {
    Child k{-1, -1, {}, false};
    if (c >= f.C) return k;
    k.p = ld_given(f.parents + c);
    if (k.p < 0 || k.p >= a.B) {
      k.p = -1;
      return k;
    }
    k.x = parent_of(a, k.p);
    if (!k.x.ok || !k.x.rest) return k;
    k.src = a.table[static_cast<long long>(k.p) * a.pps + k.x.full];
    k.copies = k.src >= 0 && k.src < a.num_pages && first[k.p] != c;
    return k;
  };
  int total = 0;
  for (int c0 = 0; c0 < f.C; c0 += kScanThreads) {
    int sum;
    block_prefix(child(c0 + tid).copies, sums, sum);
    total += sum;
  }
  const int have = lowest_free(a, total, f.list, sums);
  int base = 0;
  for (int c0 = 0; c0 < f.C; c0 += kScanThreads) {
    const int c = c0 + tid;
    const Child k = child(c);
    int sum;
    const int at = base + block_prefix(k.copies, sums, sum);
    base += sum;
    if (k.p < 0 || !k.x.rest) continue;
    int32_t *out = f.table_out + static_cast<long long>(c) * a.pps;
    if (k.copies && at < have && SPEC_CHECK(a, at < f.C)) {
      const int page = f.list[at];
      a.refs[page] = 1;
      out[k.x.full] = page;
      f.copies[at] = make_int4(k.src, page, k.x.rest, 0);
    } else if (k.copies) {   // no page left: the child gives back what it shares
      set_status(a.status, SPEC_ERR_NO_PAGE);
      for (int j = 0; j < k.x.full; ++j) {
        if (out[j] >= 0) drop_ref(a, out[j]);
        out[j] = -1;
      }
      out[k.x.full] = -1;
      f.lens_out[c] = -1;
    } else {
      if (k.src >= a.num_pages) set_status(a.status, SPEC_ERR_PAGE);
      out[k.x.full] = k.src >= 0 && k.src < a.num_pages ? k.src : -1;
    }
  }
  if (tid == 0) *f.count = have;
}

// ------------------------------------------------------------------ moving contents

// Copies the first rows of pages, in every layer: a warp a (copy, layer, head, K or V).
__global__ void __launch_bounds__(256) kv_copy_rows_kernel(const __grid_constant__ PoolArgs m,
                                                           const int4 *copies, const int32_t *count) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int n = __ldcg(count);
  const long long tasks = static_cast<long long>(n) * m.layers * m.Hkv * 2;
  const int head_bytes = m.page * m.D;
  for (long long t = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); t < tasks;
       t += 8LL * gridDim.x) {
    const int side = static_cast<int>(t & 1);
    long long r = t >> 1;
    const int h = static_cast<int>(r % m.Hkv);
    r /= m.Hkv;
    const int layer = static_cast<int>(r % m.layers);
    const int4 c = __ldcg(copies + r / m.layers);
    const long long src = (static_cast<long long>(layer) * m.num_pages + c.x) * m.Hkv + h;
    const long long dst = (static_cast<long long>(layer) * m.num_pages + c.y) * m.Hkv + h;
    uint8_t *pool = side ? m.v : m.k;
    float *scale = side ? m.v_scale : m.k_scale;
    const uint4 *from = reinterpret_cast<const uint4 *>(pool + src * head_bytes);
    uint4 *to = reinterpret_cast<uint4 *>(pool + dst * head_bytes);
    const int vecs = c.z * m.D / 16;
    if (lane == 0) scale[dst] = scale[src];
    for (int i0 = 0; i0 < vecs; i0 += 8 * 32) {
      uint4 w[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (i0 + u * 32 + lane < vecs) w[u] = from[i0 + u * 32 + lane];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (i0 + u * 32 + lane < vecs) to[i0 + u * 32 + lane] = w[u];
    }
  }
}

// ------------------------------------------------------------------ compaction

// One CTA: how many pages are live, where each goes, and the list of those that move: the i-th hole below
// that number takes the i-th live page from there on.
__global__ void __launch_bounds__(kScanThreads) kv_compact_map_kernel(const __grid_constant__ PageArgs a,
                                                                      int32_t *map, int32_t *live_out,
                                                                      int32_t *holes, int32_t *movers,
                                                                      int32_t *count) {
  __shared__ int sums[kScanWarps];
  pdl_wait();
  const int tid = threadIdx.x;
  int n = 0, live;
  for (int p = tid; p < a.num_pages; p += kScanThreads) n += __ldcg(a.refs + p) > 0;
  block_prefix(n, sums, live);
  int nh = 0, nm = 0;
  for (int p0 = 0; p0 < a.num_pages; p0 += kScanThreads) {
    const int p = p0 + tid;
    const bool held = p < a.num_pages && __ldcg(a.refs + p) > 0;
    const bool hole = p < a.num_pages && p < live && !held, mover = held && p >= live;
    // (a chunk's counts of both, in one sum)
    int sum;
    const int at = block_prefix((hole ? 1 : 0) | (mover ? 1 << 16 : 0), sums, sum);
    if (hole) holes[nh + (at & 0xffff)] = p;
    if (mover) movers[nm + (at >> 16)] = p;
    if (p < a.num_pages && !mover) map[p] = held ? p : -1;
    nh += sum & 0xffff;
    nm += sum >> 16;
  }
  __syncthreads();   // the lists
  for (int i = tid; i < nm; i += kScanThreads)
    if (SPEC_CHECK(a, i < nh)) map[movers[i]] = holes[i];
  if (tid == 0) {
    *live_out = live;
    *count = nm;
  }
}

constexpr int kMoveBytes = 32768, kMoveVecs = kMoveBytes / (16 * 256);   // of a CTA's step; of a thread in it

// Moves the listed pages, whole, in every layer, with their counts; and puts the new numbers into the table.
__global__ void __launch_bounds__(256) kv_compact_move_kernel(const __grid_constant__ PageArgs a,
                                                              const __grid_constant__ PoolArgs m,
                                                              const int32_t *map, const int32_t *holes,
                                                              const int32_t *movers,
                                                              const int32_t *count) {
  pdl_wait();
  const int tid = threadIdx.x;
  const int n = __ldcg(count);
  const long long bytes = static_cast<long long>(m.Hkv) * m.page * m.D;   // of a page in one layer
  const int steps = static_cast<int>((bytes + kMoveBytes - 1) / kMoveBytes);
  const long long tasks = static_cast<long long>(n) * m.layers * 2 * steps;
  for (long long t = blockIdx.x; t < tasks; t += gridDim.x) {
    const int step = static_cast<int>(t % steps);
    long long r = t / steps;
    const int side = static_cast<int>(r & 1);
    r >>= 1;
    const int layer = static_cast<int>(r % m.layers), i = static_cast<int>(r / m.layers);
    const int from = __ldcg(movers + i), to = __ldcg(holes + i);
    const long long src = static_cast<long long>(layer) * m.num_pages + from;
    const long long dst = static_cast<long long>(layer) * m.num_pages + to;
    uint8_t *pool = side ? m.v : m.k;
    const uint4 *s = reinterpret_cast<const uint4 *>(pool + src * bytes + static_cast<long long>(step) * kMoveBytes);
    uint4 *d = reinterpret_cast<uint4 *>(pool + dst * bytes + static_cast<long long>(step) * kMoveBytes);
    const int vecs = static_cast<int>(min(static_cast<long long>(kMoveBytes), bytes - static_cast<long long>(step) * kMoveBytes) / 16);
    uint4 w[kMoveVecs];
#pragma unroll
    for (int u = 0; u < kMoveVecs; ++u)
      if (u * 256 + tid < vecs) w[u] = __ldcs(s + u * 256 + tid);
#pragma unroll
    for (int u = 0; u < kMoveVecs; ++u)
      if (u * 256 + tid < vecs) __stcs(d + u * 256 + tid, w[u]);
    if (step == 0) {
      float *scale = side ? m.v_scale : m.k_scale;
      for (int h = tid; h < m.Hkv; h += 256) scale[dst * m.Hkv + h] = scale[src * m.Hkv + h];
      if (side == 0 && layer == 0 && tid == 0) {
        a.refs[to] = a.refs[from];
        a.refs[from] = 0;
      }
    }
  }
  const long long places = static_cast<long long>(a.B) * a.pps;
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + tid; i < places; i += 256LL * gridDim.x) {
    const int page = a.table[i];
    if (page < 0) continue;
    if (page >= a.num_pages) {
      set_status(a.status, SPEC_ERR_PAGE);
      continue;
    }
    const int now = __ldcg(map + page);
    if (now != page) a.table[i] = now;
  }
}

int grid_for(long long work, int most) {
  return static_cast<int>(work < 1 ? 1 : work < most ? work : most);
}

}  // namespace

cudaError_t launch_kv_release(const PageArgs &a, const int32_t *ended, int32_t *lens, int window,
                              int sinks, cudaStream_t stream) {
  return launch_kv(kv_release_kernel, a.B, 128, 0, stream, a, ended, lens, window, sinks);
}

cudaError_t launch_kv_reserve(const PageArgs &a, const int32_t *new_lens, int N, int32_t *granted,
                              void *ws, cudaStream_t stream) {
  int touched = (N + a.page - 2) / a.page + 1;
  if (touched > a.pps) touched = a.pps;
  return launch_kv(kv_reserve_kernel, 1, kScanThreads, a.B * sizeof(int), stream, a, new_lens, N,
                   touched, granted, static_cast<int32_t *>(ws) + 4);
}

cudaError_t launch_kv_fork(const PageArgs &a, const PoolArgs &m, ForkArgs f, void *ws,
                           cudaStream_t stream) {
  f.count = static_cast<int32_t *>(ws);
  f.copies = reinterpret_cast<int4 *>(f.count + 4);
  f.list = reinterpret_cast<int32_t *>(f.copies + f.C);
  cudaError_t e;
  if (f.C + a.B <= kForkOne && a.pps <= kForkPlaces) {
    e = launch_kv(kv_fork_pages_kernel<true>, 1, kScanThreads, 2 * a.B * sizeof(int), stream, a, f);
  } else {
    e = launch_kv(kv_fork_rows_kernel, static_cast<long long>(f.C) + a.B, 128, 0, stream, a, f);
    if (e != cudaSuccess) return e;
    e = launch_kv(kv_fork_pages_kernel<false>, 1, kScanThreads, a.B * sizeof(int), stream, a, f);
  }
  if (e != cudaSuccess) return e;
  const long long warps = static_cast<long long>(f.C) * m.layers * m.Hkv * 2;
  return launch_kv(kv_copy_rows_kernel, grid_for((warps + 7) / 8, 152 * 8), 256, 0, stream, m,
                   const_cast<const int4 *>(f.copies), const_cast<const int32_t *>(f.count));
}

cudaError_t launch_kv_compact(const PageArgs &a, const PoolArgs &m, int32_t *map, int32_t *live,
                              void *ws, cudaStream_t stream) {
  int32_t *count = static_cast<int32_t *>(ws), *holes = count + 4, *movers = holes + a.num_pages;
  cudaError_t e = launch_kv(kv_compact_map_kernel, 1, kScanThreads, 0, stream, a, map, live, holes,
                            movers, count);
  if (e != cudaSuccess) return e;
  const long long steps = (static_cast<long long>(m.Hkv) * m.page * m.D + kMoveBytes - 1) / kMoveBytes;
  const long long tasks = static_cast<long long>(m.num_pages) / 2 * m.layers * 2 * steps;
  const long long places = (static_cast<long long>(a.B) * a.pps + 255) / 256;
  return launch_kv(kv_compact_move_kernel, grid_for(tasks > places ? tasks : places, 152 * 8), 256, 0,
                   stream, a, m, const_cast<const int32_t *>(map), const_cast<const int32_t *>(holes),
                   const_cast<const int32_t *>(movers), const_cast<const int32_t *>(count));
}

// the lists of a compaction (holes, movers) or of a fork (copies, free pages) or of a reservation (free pages)
size_t kv_pages_workspace(int num_pages, int B) {
  const size_t p = 4 * static_cast<size_t>(num_pages), b = static_cast<size_t>(B);
  const size_t lists = 2 * p > 20 * b ? 2 * p : 20 * b;
  return (16 + lists + 255) / 256 * 256;
}

}  // namespace specv
