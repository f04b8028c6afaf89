// Sliding-window attention for bf16 caches: the kernel of prefill_mma.cuh with its mask.
#include "prefill_mma.cuh"

namespace skv {

template cudaError_t launch_prefill_mma<Mask::kWindow>(const kv_cache_desc&, const PackedRows&,
                                                       const PrefillArgs&, DevCtx, cudaStream_t);

}  // namespace skv
