// kv_attention_masked_fp16.hip -- the masked attention kernels for fp16 rows.
#include "kv_attention_kernel.h"

namespace nf4 {
namespace kvattn {

NF4_KV_SHAPES(kFP16, true)

}  // namespace kvattn
}  // namespace nf4
