// spec_kv_attention.cu -- attention of the new tokens over the paged e4m3 cache.
//
// The simplest form: one CTA per new token and query head walks the cache 128 tokens at a time,
// one token per thread for the scores, one dim per thread for the values, with a running maximum
// and sum.
#include "spec_kv.cuh"

namespace specv {

namespace {

constexpr int kSimpleThreads = 128;

__device__ __forceinline__ float e4m3_to_float(uint8_t x) {
  const uint32_t h = e4m3_to_half2(x);
  return __half22float2(*reinterpret_cast<const __half2 *>(&h)).x;
}
__device__ __forceinline__ float block_reduce(float v, bool max, float *sh) {
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = max ? fmax_nan(v, w) : v + w;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  return max ? fmax_nan(fmax_nan(sh[0], sh[1]), fmax_nan(sh[2], sh[3]))
             : (sh[0] + sh[1]) + (sh[2] + sh[3]);
}

template <typename T>
__global__ void __launch_bounds__(kSimpleThreads)
    kv_attention_simple(KvArgs a, const T *q, long long q_stride, float scale, T *out,
                        float *lse) {
  __shared__ float qs[128], ps[128], sh[4];
  __shared__ float vs[128];
  __shared__ const uint8_t *vrow[128];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x;
  const int hq = blockIdx.x % a.Hq;
  const long long token = blockIdx.x / a.Hq;
  const int b = static_cast<int>(token / a.N), i = static_cast<int>(token - static_cast<long long>(b) * a.N);
  const int h = hq / (a.Hq / a.Hkv);
  T *o = out + (token * a.Hq + hq) * a.D;
  int len, n;
  const bool ok = kv_lengths(a, b, len, n);
  if (!ok && tid == 0) set_status(a.status, SPEC_ERR_LENGTH);
  if (tid < a.D)
    qs[tid] = static_cast<float>(q[token * q_stride + static_cast<long long>(hq) * a.D + tid]) * scale;
  __syncthreads();
  float m = -INFINITY, l = 0.f, acc = 0.f;
  const int end = !ok || i >= n ? 0 : a.mask ? len + n : len + i + 1;
  for (int t0 = 0; t0 < end; t0 += 128) {
    const int t = t0 + tid;
    bool see = t < end;
    if (see && a.mask && t >= len) {
      const int j = t - len;
      see = (__ldg(a.mask + (token * a.W) + (j >> 5)) >> (j & 31)) & 1u;
    }
    float x = -INFINITY;
    vs[tid] = 0.f;
    vrow[tid] = nullptr;
    if (see) {
      int page;
      if (!kv_page(a, b, t >> a.page_shift, page)) {
        set_status(a.status, SPEC_ERR_PAGE);
        x = NAN;
      } else {
        const long long head = static_cast<long long>(page) * a.Hkv + h;
        const long long row = ((head << a.page_shift) + (t & (a.page - 1))) * a.D;
        float dot = 0.f;
        for (int d = 0; d < a.D; ++d) dot += e4m3_to_float(a.k[row + d]) * qs[d];
        x = dot * a.k_scale[head];
        vs[tid] = a.v_scale[head];
        vrow[tid] = a.v + row;
      }
    }
    const float mn = block_reduce(fmax_nan(m, x), true, sh);
    const float mu = mn == -INFINITY ? 0.f : mn;
    const float p = __expf(x - mu), f = __expf(m - mu);
    ps[tid] = p;
    m = mn;
    l = l * f + block_reduce(p, false, sh);   // (its barriers also publish ps, vs, vrow)
    acc *= f;
    if (tid < a.D)
      for (int k = 0; k < 128; ++k)
        if (vrow[k]) acc += ps[k] * vs[k] * e4m3_to_float(vrow[k][tid]);
    __syncthreads();
  }
  if (tid < a.D) {
    const float r = !ok ? NAN : l == 0.f ? 0.f : acc / l;
    o[tid] = static_cast<T>(r);
  }
  if (lse && tid == 0) lse[token * a.Hq + hq] = !ok ? NAN : l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

size_t kv_attention_workspace(int B, int N, int Hq, int Hkv, int D) { return 256; }

cudaError_t launch_kv_attention(const KvArgs &a, const void *q, long long q_stride, int dtype,
                                float scale, void *out, float *lse, void *ws,
                                cudaStream_t stream) {
  const long long grid = static_cast<long long>(a.B) * a.N * a.Hq;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (dtype == SPEC_BF16)
    return launch_kv(kv_attention_simple<__nv_bfloat16>, grid, kSimpleThreads, 0, stream, a,
                     static_cast<const __nv_bfloat16 *>(q), q_stride, scale,
                     static_cast<__nv_bfloat16 *>(out), lse);
  return launch_kv(kv_attention_simple<__half>, grid, kSimpleThreads, 0, stream, a,
                   static_cast<const __half *>(q), q_stride, scale, static_cast<__half *>(out),
                   lse);
}

}  // namespace specv
