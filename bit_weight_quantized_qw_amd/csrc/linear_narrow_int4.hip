// qgemm_linear by narrow tiles, INT4 weights.
#include "linear_narrow.h"

namespace qw {

template qw_status launch_linear_narrow<QW_FMT_INT4_G32>(const LinearArgs &, int, hipStream_t);

}  // namespace qw
