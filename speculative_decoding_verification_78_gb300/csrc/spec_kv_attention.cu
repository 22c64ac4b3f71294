// spec_kv_attention.cu -- attention over the paged cache: the choice of kernel, and the instances of the kernel
// for few query rows without a window.
#include "spec_kv_attention_cols.cuh"

namespace specv {

using namespace attn;

cudaError_t launch_attention_cols(AttnArgs &p, int dtype, const CUtensorMap &mk, const CUtensorMap &mv,
                                  int ctas, char *ws, cudaStream_t stream) {
  return launch_cols<false>(p, dtype, mk, mv, ctas, ws, stream);
}

size_t kv_attention_workspace(int B, int N, int Hq, int Hkv, int D) {
  const size_t nt = kv_row_tile(static_cast<long long>(N) * (Hq / Hkv));
  return 2 * kMaxCtas * (sizeof(int4) + nt * sizeof(float) * (1 + D));
}

cudaError_t launch_kv_attention(const KvArgs &a, const void *q, long long q_stride, int dtype,
                                float scale, int window, int sinks, void *out, float *lse, void *ws,
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
  p.window = window;
  p.sinks = sinks;
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  const bool cols = kv_row_tile(static_cast<long long>(a.N) * p.G) <= 32;
  const auto launch = window > 0 ? (cols ? launch_window_cols : launch_window_rows)
                                 : (cols ? launch_attention_cols : launch_attention_rows);
  return launch(p, dtype, mk, mv, ctas, static_cast<char *>(ws), stream);
}

}  // namespace specv
