// kvx_attend8_tc_shared.cu -- the kernels of kvx_attend8_tc.cu for the passes of
// kvx_attend8_shared: queries that see all slots, results in fp32, or joined with what the
// first pass left.
#define KVX_ATTEND_SHARED 1
#include "kvx_attend8_tc.cu"
