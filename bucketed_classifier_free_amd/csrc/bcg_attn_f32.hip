// Paged attention with fp32 queries and pages (bcg_attn_impl.h).
#include "bcg_attn_impl.h"

namespace bcg {
template hipError_t launch_decode<float, float>(const AttnParams&, hipStream_t);
template hipError_t launch_prompt<float, float>(const AttnParams&, hipStream_t);
template int prompt_columns<float, float>(int);
template int prompt_block<float, float>(int);
}  // namespace bcg
