// kda_lib.cu -- the library's one translation unit: the gated delta rule
// (kda_prefill.cu) and the softmax-attention operators beside it, which share
// its device error word, device facts and tensor-map encoder.
#include "kda_prefill.cu"

#include "kda_attn_api.cuh"
