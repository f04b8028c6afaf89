// Attention of few rows for fp32 caches: the kernel of prefill_simt_few.cuh with each mask.
#include "prefill_simt_few.cuh"

namespace skv {

template cudaError_t launch_prefill_simt_few<Mask::kWindow>(const kv_cache_desc&,
                                                            const PackedRows&, const PrefillArgs&,
                                                            DevCtx, cudaStream_t);
template cudaError_t launch_prefill_simt_few<Mask::kTree>(const kv_cache_desc&, const PackedRows&,
                                                          const PrefillArgs&, DevCtx,
                                                          cudaStream_t);

}  // namespace skv
