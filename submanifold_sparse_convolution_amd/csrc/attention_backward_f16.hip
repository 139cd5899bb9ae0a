// Gradients of window attention on f16 rows (a file a type: they compile in parallel).
#include "attention_backward.h"

namespace smc {

hipError_t launch_attention_backward_f16(const AttentionArgs& a, int lengths, hipStream_t s) {
    return attention_backward_of_type<kF16>(a, lengths, s);
}

}  // namespace smc
