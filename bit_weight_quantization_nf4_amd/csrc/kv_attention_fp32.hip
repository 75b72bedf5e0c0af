// kv_attention_fp32.hip -- the attention kernels for fp32 rows.
#include "kv_attention_kernel.h"

namespace nf4 {
namespace kvattn {

NF4_KV_SHAPES(kFP32, false)

}  // namespace kvattn
}  // namespace nf4
