// The norm with an output in e4m3 and scales.
#define SS_NORM_QUANT
#include "ss_rms_norm.cuh"
