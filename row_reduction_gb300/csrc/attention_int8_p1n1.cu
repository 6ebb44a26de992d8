// Attention over the cache: int8 codes, BF16 queries, 8 columns.
#include "attention_mma.cuh"
namespace mt {
MT_DEFINE_ATTENTION(launch_attention_int8_p1n1, true, 1, 1)
}  // namespace mt
