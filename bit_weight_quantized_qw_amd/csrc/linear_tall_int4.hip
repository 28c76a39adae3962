// qgemm_linear by tall tiles, INT4 weights.
#include "linear_tall.h"

namespace qw {

template qw_status launch_linear_tall<QW_FMT_INT4_G32>(const LinearArgs &, int, hipStream_t);

}  // namespace qw
