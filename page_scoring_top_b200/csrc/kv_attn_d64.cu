// kv_attn_d64.cu -- the attention kernels of head dims up to 64 (kv_attn.cuh).
#define IDX_KV_ATTN_DP 64
#include "kv_attn.cuh"
