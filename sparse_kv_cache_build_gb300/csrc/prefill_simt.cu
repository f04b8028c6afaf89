// Attention of packed rows for fp32 caches: the kernel of prefill_simt.cuh with each mask.
#include "prefill_simt.cuh"

namespace skv {

template cudaError_t launch_prefill_simt<Mask::kCausal>(const kv_cache_desc&, const PackedRows&,
                                                        const PrefillArgs&, DevCtx, cudaStream_t);
template cudaError_t launch_prefill_simt<Mask::kWindow>(const kv_cache_desc&, const PackedRows&,
                                                        const PrefillArgs&, DevCtx, cudaStream_t);
template cudaError_t launch_prefill_simt<Mask::kTree>(const kv_cache_desc&, const PackedRows&,
                                                      const PrefillArgs&, DevCtx, cudaStream_t);

}  // namespace skv
