// Kernels for head dim 128 of windows with visible first keys.
#include "fa_inst.cuh"

FA_DEFINE_SINKS_HEAD_DIM(128, 2, 128, 2)
