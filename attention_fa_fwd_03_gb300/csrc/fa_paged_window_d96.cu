// Paged-cache attention kernels for head dim 96 of windows.
#include "fa_paged_fwd.cuh"

FA_DEFINE_PAGED_WINDOW_HEAD_DIM(96)
