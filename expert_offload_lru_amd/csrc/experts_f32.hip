// Products over the rows of experts in f32.
#include "expert_products.hpp"

namespace moe {
MOE_EXPERTS_OF(float, f32)
}  // namespace moe
