// spec_kv_window.cu -- instances of the attention kernel for few query rows, with a window and sinks.
#include "spec_kv_attention_cols.cuh"

namespace specv {

cudaError_t launch_window_cols(attn::AttnArgs &p, int dtype, const CUtensorMap &mk,
                               const CUtensorMap &mv, int ctas, char *ws, cudaStream_t stream) {
  return launch_cols<true>(p, dtype, mk, mv, ctas, ws, stream);
}

}  // namespace specv
