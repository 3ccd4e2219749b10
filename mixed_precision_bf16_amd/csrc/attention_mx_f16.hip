// Instantiates the attention kernels for MXFP4 caches and FP16 activations.
#define FP4_ATTN_FMT 1
#define FP4_ATTN_ACT 1
#define FP4_ATTN_LAUNCH launch_attention_mx_f16
#include "attention_inst.inc"
