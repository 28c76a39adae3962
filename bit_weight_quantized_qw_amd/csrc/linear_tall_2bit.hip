// qgemm_linear by tall tiles, 2bit weights.
#include "linear_tall.h"

namespace qw {

template qw_status launch_linear_tall<QW_FMT_2BIT_G32>(const LinearArgs &, int, hipStream_t);

}  // namespace qw
