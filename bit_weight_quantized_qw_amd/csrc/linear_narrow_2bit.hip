// qgemm_linear by narrow tiles, 2bit weights.
#include "linear_narrow.h"

namespace qw {

template qw_status launch_linear_narrow<QW_FMT_2BIT_G32>(const LinearArgs &, int, hipStream_t);

}  // namespace qw
