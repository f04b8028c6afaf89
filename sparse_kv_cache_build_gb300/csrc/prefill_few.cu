// Attention of few rows for bf16 caches: the kernel of prefill_few.cuh with each mask.
#include "prefill_few.cuh"

namespace skv {

template cudaError_t launch_prefill_few<Mask::kWindow>(const kv_cache_desc&, const PackedRows&,
                                                       const PrefillArgs&, DevCtx, cudaStream_t);
template cudaError_t launch_prefill_few<Mask::kTree>(const kv_cache_desc&, const PackedRows&,
                                                     const PrefillArgs&, DevCtx, cudaStream_t);

}  // namespace skv
