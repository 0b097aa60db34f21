// kv_attn_d256.cu -- the attention kernels of head dims up to 256 (kv_attn.cuh).
#define IDX_KV_ATTN_DP 256
#include "kv_attn.cuh"
