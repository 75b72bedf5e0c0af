// kv_attention_masked_bf16.hip -- the masked attention kernels for bf16 rows.
#include "kv_attention_kernel.h"

namespace nf4 {
namespace kvattn {

NF4_KV_SHAPES(kBF16, true)

}  // namespace kvattn
}  // namespace nf4
