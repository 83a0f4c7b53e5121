// Attention over the 16-bit cache: head dimension 128, fp16.
#include "bsfa_decode16.cuh"

namespace bsfa::decode16 {

template bsfa_status run<128, true>(const DecArgs&, const Plan&, int, int, cudaStream_t);

}  // namespace bsfa::decode16
