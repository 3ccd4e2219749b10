// Instantiates the attention kernels for NVFP4 caches and FP16 activations.
#define FP4_ATTN_FMT 0
#define FP4_ATTN_ACT 1
#define FP4_ATTN_LAUNCH launch_attention_nv_f16
#include "attention_inst.inc"
