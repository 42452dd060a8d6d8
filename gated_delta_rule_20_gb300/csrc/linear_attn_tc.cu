#include "linear_attn.h"
namespace gdn {
bool linear_attn_tc_supported(const LinearAttn&) { return false; }
gdn_status launch_linear_attn_tc(const LinearAttn&, const LinearAttnSplit&, int, int, int32_t*, cudaStream_t) { return GDN_ERR_UNSUPPORTED; }
}
