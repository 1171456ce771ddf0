// Paged attention with bf16 queries and pages (bcg_attn_impl.h).
#include "bcg_attn_impl.h"

namespace bcg {
template hipError_t launch_decode<bf16_t, bf16_t>(const AttnParams&, hipStream_t);
template hipError_t launch_prompt<bf16_t, bf16_t>(const AttnParams&, hipStream_t);
template int prompt_columns<bf16_t, bf16_t>(int);
template int prompt_block<bf16_t, bf16_t>(int);
}  // namespace bcg
