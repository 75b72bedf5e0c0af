// kv_attention_fp16.hip -- the attention kernels for fp16 rows.
#include "kv_attention_kernel.h"

namespace nf4 {
namespace kvattn {

template hipError_t launch_shape<kFP16>(const AttnArgs &, const Plan &, int, int, hipStream_t);

}  // namespace kvattn
}  // namespace nf4
