// Paged-cache attention kernels for head dim 128.
#include "fa_paged_fwd.cuh"

FA_DEFINE_PAGED_HEAD_DIM(128)
