// spec_kv_window_rows.cu -- instances of the attention kernel for many query rows, with a window and sinks.
#include "spec_kv_attention_rows.cuh"

namespace specv {

cudaError_t launch_window_rows(attn::AttnArgs &p, int dtype, const CUtensorMap &mk,
                               const CUtensorMap &mv, int ctas, char *ws, cudaStream_t stream) {
  return launch_rows<true>(p, dtype, mk, mv, ctas, ws, stream);
}

}  // namespace specv
