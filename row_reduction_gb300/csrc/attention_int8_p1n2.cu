// Attention over the cache: int8 codes, BF16 queries, 16 columns.
#include "attention_mma.cuh"
namespace mt {
MT_DEFINE_ATTENTION(launch_attention_int8_p1n2, true, 1, 2)
}  // namespace mt
