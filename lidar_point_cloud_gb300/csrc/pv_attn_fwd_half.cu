// The forward attention kernels for float16 (pv_attn_fwd.cu is for bfloat16).
#define PV_ATTN_HALF
#include "pv_attn_fwd.cu"
