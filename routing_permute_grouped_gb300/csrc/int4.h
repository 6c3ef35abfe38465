// int4.h -- what the 4-bit weights' quantiser and their product share on the host.
#pragma once
#include <cstdint>

namespace moe {

// The rules on a row of codes; a moe_status_t.
int check_int4_row(int32_t group, int32_t K);

}  // namespace moe
