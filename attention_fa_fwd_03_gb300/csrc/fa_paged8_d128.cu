// Attention over a paged cache held in 8 bits for head dim 128.
#include "fa_paged_fwd.cuh"

FA_DEFINE_PAGED8_HEAD_DIM(128)
