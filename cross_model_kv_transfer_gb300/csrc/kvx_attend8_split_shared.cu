// kvx_attend8_split_shared.cu -- the kernels of kvx_attend8_split.cu for the passes of
// kvx_attend8_shared.
#define KVX_ATTEND_SHARED 1
#include "kvx_attend8_split.cu"
