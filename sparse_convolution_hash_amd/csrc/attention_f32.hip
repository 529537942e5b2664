// The attention kernels for f32.
#include "attention.h"

namespace spc {
namespace attn {

spc_status launch_fwd_f32(const Args& p, const Cut& c, hipStream_t stream) { return launch_fwd<F32>(p, c, stream); }
spc_status launch_bwd_f32(const Args& p, const Cut& q, const Cut& k, hipStream_t stream) { return launch_bwd<F32>(p, q, k, stream); }

}  // namespace attn
}  // namespace spc
