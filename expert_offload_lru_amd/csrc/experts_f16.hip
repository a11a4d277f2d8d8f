// Products over the rows of experts in f16.
#include "expert_products.hpp"

namespace moe {
MOE_EXPERTS_OF(f16, f16)
}  // namespace moe
