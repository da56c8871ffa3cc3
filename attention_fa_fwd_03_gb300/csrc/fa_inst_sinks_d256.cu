// Kernels for head dim 256 of windows with visible first keys.
#include "fa_inst.cuh"

FA_DEFINE_SINKS_HEAD_DIM(256, 1, 64, 2)
