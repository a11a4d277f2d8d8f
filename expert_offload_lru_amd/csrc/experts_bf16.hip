// Products over the rows of experts in bf16.
#include "expert_products.hpp"

namespace moe {
MOE_EXPERTS_OF(bf16, bf16)
}  // namespace moe
