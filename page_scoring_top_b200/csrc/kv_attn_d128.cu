// kv_attn_d128.cu -- the attention kernels of head dims up to 128 (kv_attn.cuh).
#define IDX_KV_ATTN_DP 128
#include "kv_attn.cuh"
