// Argument checks of the rotary positions that the block-scaled cache's host side
// shares.  Not part of the ABI.
#pragma once

#include "../../include/kvc.h"
#include "kvc_rotary.h"

namespace kvc {

kvc_status rotary_table(const kvc_rotary* r, const int32_t* d_pos, int32_t first, RotaryTable* t);
// `out`: the rows have a packed output too
kvc_status rows_in(const kvc_rows* r, int32_t batch, int32_t n, bool out, RowsIn* in);

}  // namespace kvc
