// Attention over the cache: e4m3 codes, BF16 queries, 16 columns.
#include "attention_mma.cuh"
namespace mt {
MT_DEFINE_ATTENTION(launch_attention_e4m3_p1n2, false, 1, 2)
}  // namespace mt
