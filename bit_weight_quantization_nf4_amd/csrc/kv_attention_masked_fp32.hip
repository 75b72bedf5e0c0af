// kv_attention_masked_fp32.hip -- the masked attention kernels for fp32 rows.
#include "kv_attention_kernel.h"

namespace nf4 {
namespace kvattn {

NF4_KV_SHAPES(kFP32, true)

}  // namespace kvattn
}  // namespace nf4
