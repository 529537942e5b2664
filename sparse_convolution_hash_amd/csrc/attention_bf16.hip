// The attention kernels for bf16.
#include "attention.h"

namespace spc {
namespace attn {

spc_status launch_fwd_bf16(const Args& p, const Cut& c, hipStream_t stream) { return launch_fwd<BF16>(p, c, stream); }
spc_status launch_bwd_bf16(const Args& p, const Cut& q, const Cut& k, hipStream_t stream) { return launch_bwd<BF16>(p, q, k, stream); }

}  // namespace attn
}  // namespace spc
