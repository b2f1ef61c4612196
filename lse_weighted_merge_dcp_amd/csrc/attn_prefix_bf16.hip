// attn_prefix_bf16.hip -- attn_prefix_rows.hpp for bfloat16.
#include "attn_prefix_rows.hpp"

namespace dcpa {

hipError_t launch_prefix_bf16(const GroupArgs& a, bool kv8, bool wide, hipStream_t stream) { return run_rows<BF16T>(a, kv8, wide, stream); }

}  // namespace dcpa
