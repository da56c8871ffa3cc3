// Kernels for head dim 64 of windows with visible first keys.
#include "fa_inst.cuh"

FA_DEFINE_SINKS_HEAD_DIM(64, 2, 128, 3)
