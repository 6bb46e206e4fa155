// decode_kernel instantiations for block-scaled FP8 pools, 4 kv head(s) per sequence.
#define PA_HKV 4
#define PA_F8 true
#define PA_BS true
#include "pa_decode_inst.cuh"
