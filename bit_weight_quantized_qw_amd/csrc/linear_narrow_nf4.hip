// qgemm_linear by narrow tiles, NF4 weights.
#include "linear_narrow.h"

namespace qw {

template qw_status launch_linear_narrow<QW_FMT_NF4_B64>(const LinearArgs &, int, hipStream_t);

}  // namespace qw
