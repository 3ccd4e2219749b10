// Instantiates the attention kernels for NVFP4 caches and BF16 activations.
#define FP4_ATTN_FMT 0
#define FP4_ATTN_ACT 0
#define FP4_ATTN_LAUNCH launch_attention_nv_bf16
#include "attention_inst.inc"
