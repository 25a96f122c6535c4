// kernel_attn_cache_f16_int8.hip -- attention over the cache: queries of f16, pools of int8 codes.
#include "attn_cache_launch.hpp"

namespace att {
template void launch_attn_cache<_Float16, KV_INT8>(const CacheArgs& a, hipStream_t stream);
}
