// qgemm_linear by tall tiles, NF4 weights.
#include "linear_tall.h"

namespace qw {

template qw_status launch_linear_tall<QW_FMT_NF4_B64>(const LinearArgs &, int, hipStream_t);

}  // namespace qw
