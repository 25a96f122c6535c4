// kernel_attn_cache_bf16_same.hip -- attention over the cache: queries of bf16, pools of the same type.
#include "attn_cache_launch.hpp"

namespace att {
template void launch_attn_cache<__bf16, KV_SAME>(const CacheArgs& a, hipStream_t stream);
}
