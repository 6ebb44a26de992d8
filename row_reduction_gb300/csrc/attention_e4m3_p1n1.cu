// Attention over the cache: e4m3 codes, BF16 queries, 8 columns.
#include "attention_mma.cuh"
namespace mt {
MT_DEFINE_ATTENTION(launch_attention_e4m3_p1n1, false, 1, 1)
}  // namespace mt
