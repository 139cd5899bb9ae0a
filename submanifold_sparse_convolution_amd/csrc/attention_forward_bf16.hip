// Window attention on bf16 rows (a file a type: they compile in parallel).
#include "attention_forward.h"

namespace smc {

hipError_t launch_attention_bf16(const AttentionArgs& a, int lengths, hipStream_t s) { return attention_of_type<kBF16>(a, lengths, s); }

}  // namespace smc
