// spec_kv.h -- what the KV-cache kernels share: arguments, e4m3 and 16-bit element access, page
// scales, and launches.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "spec_common.cuh"

namespace specv {

constexpr float kE4m3Max = 448.f;
constexpr float kMinPageScale = 5.421010862427522e-20f;   // 2^-64

// A load of what a kernel before on the stream may have written (lengths, tables, queries, page scales). Not __ldg: the
// memory that reads has to stay as it is for the whole kernel, and one that is launched as a programmatic dependent
// begins while the kernel before still writes.
template <typename T> __device__ __forceinline__ T ld_given(const T *p) { return *p; }

struct KvArgs {
  uint8_t *k, *v;            // [num_pages, Hkv, page, D] e4m3
  float *k_scale, *v_scale;  // [num_pages, Hkv]
  const int32_t *page_table; // [B, pps]
  const int32_t *seq_lens;   // [B]
  const int32_t *new_lens;   // [B] or null
  const uint32_t *mask;      // [B, N, W] or null
  int32_t *status;
  int num_pages, page, page_shift, Hkv, D, pps;
  int B, N, W, Hq;
};

// Tokens of sequence b before the new ones and how many new ones it has; false (and a status)
// when they do not fit its page table.
__device__ __forceinline__ bool kv_lengths(const KvArgs &a, int b, int &len, int &n) {
  len = ld_given(a.seq_lens + b);
  n = a.new_lens ? ld_given(a.new_lens + b) : a.N;
  const long long cap = static_cast<long long>(a.pps) << a.page_shift;
  return len >= 0 && n >= 0 && n <= a.N && static_cast<long long>(len) + n <= cap;
}

__device__ __forceinline__ bool kv_page(const KvArgs &a, int b, int local, int &page) {
  page = ld_given(a.page_table + static_cast<long long>(b) * a.pps + local);
  return page >= 0 && page < a.num_pages;
}

// The smallest power of two s with amax <= 448 s, at least 2^-64, from the bits of amax: with
// amax = m 2^E, 448 = 1.75 2^8, so s = 2^(E - 8), or 2^(E - 7) when m > 1.75. (Exact: a
// logarithm could land on the wrong side of a boundary.)
__device__ __forceinline__ float kv_scale_for(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < 127 - 64 ? kMinPageScale : __uint_as_float(static_cast<uint32_t>(e) << 23);
}

// two fp32 -> two e4m3 (round to nearest even, saturating; `lo` in the low byte)
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// two e4m3 -> two fp16, exactly
__device__ __forceinline__ uint32_t e4m3_to_half2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}
__device__ __forceinline__ void e4m3_to_floats(uint2 w, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t two = ((i < 2 ? w.x : w.y) >> (16 * (i & 1))) & 0xffffu;
    const uint32_t h = e4m3_to_half2(two);
    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}
// eight fp32, times m, as e4m3
__device__ __forceinline__ uint2 floats_to_e4m3(const float (&f)[8], float m) {
  uint2 w;
  w.x = e4m3_pair(f[0] * m, f[1] * m) | (e4m3_pair(f[2] * m, f[3] * m) << 16);
  w.y = e4m3_pair(f[4] * m, f[5] * m) | (e4m3_pair(f[6] * m, f[7] * m) << 16);
  return w;
}

// 16-bit element types: eight of them (a 16-byte vector) to and from fp32
template <typename T> __device__ __forceinline__ void vec_to_floats(uint4 v, float (&f)[8]);
template <>
__device__ __forceinline__ void vec_to_floats<__nv_bfloat16>(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf_lo(w[i]);
    f[2 * i + 1] = bf_hi(w[i]);
  }
}
template <> __device__ __forceinline__ void vec_to_floats<__half>(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}
__device__ __forceinline__ uint32_t pack_pair(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_pair(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
template <typename T> __device__ __forceinline__ uint4 floats_to_vec(const float (&f)[8]) {
  return make_uint4(pack_pair(f[0], f[1], T()), pack_pair(f[2], f[3], T()),
                    pack_pair(f[4], f[5], T()), pack_pair(f[6], f[7], T()));
}

// Launches `kernel` on `stream` as a programmatic dependent of what precedes it there: it may be
// scheduled while that drains, so a kernel launched by it waits (griddepcontrol.wait) before it
// touches memory.
template <typename... P, typename... A>
inline cudaError_t launch_kv(void (*kernel)(P...), long long grid, int threads, size_t smem,
                             cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

struct RopeArgs {
  const void *q, *k, *v;
  long long q_stride, k_stride, v_stride;   // elements between consecutive tokens
  void *q_out;
  const float *rope;            // [rows, R] cosines | sines, or null
  const int32_t *positions;     // [B, N] or null
  int rows, R, pairs;
  int touched;                  // pages one sequence's new tokens can touch
  int vec4;                     // rope is 16-byte aligned
};

// Pages: counts of the places that hold them, and the table of the sequences concerned
struct PageArgs {
  int32_t *refs;             // [num_pages]
  int32_t *table;            // [B, pps]; a negative entry: no page
  const int32_t *seq_lens;   // [B]
  int32_t *status;
  int num_pages, page, page_shift, pps, B;
};
// All layers of a cache, for moving contents
struct PoolArgs {
  uint8_t *k, *v;
  float *k_scale, *v_scale;
  int num_pages, page, Hkv, D, layers;
};
struct ForkArgs {
  const int32_t *parents;    // [C]
  int32_t *table_out;        // [C, pps]
  int32_t *lens_out;         // [C]
  int32_t *count;            // copies to make: (page, its copy, rows)
  int4 *copies;
  int32_t *list;             // free pages
  int C, release;
};
cudaError_t launch_kv_release(const PageArgs &a, const int32_t *ended, int32_t *lens, int window,
                              int sinks, cudaStream_t stream);
cudaError_t launch_kv_reserve(const PageArgs &a, const int32_t *new_lens, int N, int32_t *granted,
                              void *ws, cudaStream_t stream);
cudaError_t launch_kv_fork(const PageArgs &a, const PoolArgs &m, ForkArgs f, void *ws,
                           cudaStream_t stream);
cudaError_t launch_kv_compact(const PageArgs &a, const PoolArgs &m, int32_t *map, int32_t *live,
                              void *ws, cudaStream_t stream);
size_t kv_pages_workspace(int num_pages, int B);

cudaError_t launch_kv_append(const KvArgs &a, const RopeArgs &r, int dtype, cudaStream_t stream);
cudaError_t launch_kv_commit(const KvArgs &a, int layers, const int32_t *path,
                             const int32_t *accept, int32_t *out_lens, cudaStream_t stream);
cudaError_t launch_kv_attention(const KvArgs &a, const void *q, long long q_stride, int dtype,
                                float scale, int window, int sinks, void *out, float *lse, void *ws,
                                cudaStream_t stream);   // window 0: none
size_t kv_attention_workspace(int B, int N, int Hq, int Hkv, int D);
// Query rows of a tile, for calls with `rows` of them a key head: up to 32 along the columns of an MMA, more
// along its lanes. (What each costs is measured at the two kernels.)
inline int kv_row_tile(long long rows) {
  return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 128 ? 128 : 256;
}

}  // namespace specv
