// The norm with an output in the input's type.
#include "ss_rms_norm.cuh"
