// decode_kernel instantiations for block-scaled FP8 pools, 2 kv head(s) per sequence.
#define PA_HKV 2
#define PA_F8 true
#define PA_BS true
#include "pa_decode_inst.cuh"
