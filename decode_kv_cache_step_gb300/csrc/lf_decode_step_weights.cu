// Instantiations of the decode-step kernel that evict by the accumulated
// attention weight: the last-CTA merge and both rings of the cluster merge.
#include "lf_step_kernel.cuh"

namespace lf {
namespace {

template <int D, int G>
cudaError_t launch_dg(const CUtensorMap& tmK, const CUtensorMap& tmV, const StepParams& p,
                      int units, cudaStream_t stream, int stages, bool cluster, bool pdl) {
    if (!cluster) return launch_t<D, G, 2, kWeights, false>(tmK, tmV, p, units, stream, pdl);
    return stages == kDeepStages
               ? launch_t<D, G, kDeepStages, kWeights, true>(tmK, tmV, p, units, stream, pdl)
               : launch_t<D, G, 2, kWeights, true>(tmK, tmV, p, units, stream, pdl);
}

}  // namespace

int max_active_clusters_weights(int D, int G, int stages, int csize) {
#define LF_STEP_CASE(DD, GG)                                                            \
    if (D == DD && G == GG)                                                             \
        return stages == kDeepStages                                                    \
                   ? max_active_clusters_t<DD, GG, kDeepStages, kWeights>(csize)        \
                   : max_active_clusters_t<DD, GG, 2, kWeights>(csize);
    LF_STEP_CASE(64, 1) LF_STEP_CASE(64, 2) LF_STEP_CASE(64, 4) LF_STEP_CASE(64, 8)
    LF_STEP_CASE(128, 1) LF_STEP_CASE(128, 2) LF_STEP_CASE(128, 4) LF_STEP_CASE(128, 8)
#undef LF_STEP_CASE
    return 0;
}

cudaError_t launch_decode_step_weights(int D, int G, int stages, bool cluster,
                                       const CUtensorMap& tmK, const CUtensorMap& tmV,
                                       const StepParams& p, int units, cudaStream_t stream,
                                       bool pdl) {
#define LF_STEP_CASE(DD, GG) \
    if (D == DD && G == GG) return launch_dg<DD, GG>(tmK, tmV, p, units, stream, stages, cluster, pdl);
    LF_STEP_CASE(64, 1) LF_STEP_CASE(64, 2) LF_STEP_CASE(64, 4) LF_STEP_CASE(64, 8)
    LF_STEP_CASE(128, 1) LF_STEP_CASE(128, 2) LF_STEP_CASE(128, 4) LF_STEP_CASE(128, 8)
#undef LF_STEP_CASE
    return cudaErrorInvalidValue;
}

}  // namespace lf
