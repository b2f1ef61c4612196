// attn_prefix_f16.hip -- attn_prefix_rows.hpp for float16.
#include "attn_prefix_rows.hpp"

namespace dcpa {

hipError_t launch_prefix_f16(const GroupArgs& a, bool kv8, bool wide, hipStream_t stream) { return run_rows<F16T>(a, kv8, wide, stream); }

}  // namespace dcpa
