// kernel_attn_cache_bf16_e4m3.hip -- attention over the cache: queries of bf16, pools of e4m3 codes.
#include "attn_cache_launch.hpp"

namespace att {
template void launch_attn_cache<__bf16, KV_E4M3>(const CacheArgs& a, hipStream_t stream);
}
