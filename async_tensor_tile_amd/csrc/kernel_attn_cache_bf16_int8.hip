// kernel_attn_cache_bf16_int8.hip -- attention over the cache: queries of bf16, pools of int8 codes.
#include "attn_cache_launch.hpp"

namespace att {
template void launch_attn_cache<__bf16, KV_INT8>(const CacheArgs& a, hipStream_t stream);
}
