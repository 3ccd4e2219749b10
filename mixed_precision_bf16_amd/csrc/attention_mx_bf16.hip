// Instantiates the attention kernels for MXFP4 caches and BF16 activations.
#define FP4_ATTN_FMT 1
#define FP4_ATTN_ACT 0
#define FP4_ATTN_LAUNCH launch_attention_mx_bf16
#include "attention_inst.inc"
