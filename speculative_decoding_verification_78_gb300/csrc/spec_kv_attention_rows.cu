// spec_kv_attention_rows.cu -- instances of the attention kernel for many query rows, without a window.
#include "spec_kv_attention_rows.cuh"

namespace specv {

cudaError_t launch_attention_rows(attn::AttnArgs &p, int dtype, const CUtensorMap &mk,
                                  const CUtensorMap &mv, int ctas, char *ws, cudaStream_t stream) {
  return launch_rows<false>(p, dtype, mk, mv, ctas, ws, stream);
}

}  // namespace specv
