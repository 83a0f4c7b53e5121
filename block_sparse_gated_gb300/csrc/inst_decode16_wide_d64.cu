// Attention of many query rows over the 16-bit cache: head dimension 64.
#include "bsfa_decode16_wide.cuh"

namespace bsfa::decode16 {

template bsfa_status run_wide<64, false>(const CUtensorMap&, const CUtensorMap&, const DecArgs&,
                                         const Plan&, int, int, cudaStream_t);
template bsfa_status run_wide<64, true>(const CUtensorMap&, const CUtensorMap&, const DecArgs&,
                                        const Plan&, int, int, cudaStream_t);

}  // namespace bsfa::decode16
