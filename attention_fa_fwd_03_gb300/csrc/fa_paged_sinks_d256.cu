// Paged-cache attention kernels for head dim 256 of windows with visible first keys.
#include "fa_paged_fwd.cuh"

FA_DEFINE_PAGED_SINKS_HEAD_DIM(256)
