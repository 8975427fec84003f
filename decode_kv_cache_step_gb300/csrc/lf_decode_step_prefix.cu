// Instantiations of the decode-step kernel whose merge joins a shared-prefix
// attention: the unit's slots and the prefix share one softmax, so the output
// and LongFlowScore's weights are normalised over both.
//
// The pieces of the prefix's attention enter the merge of the unit's last CTA
// like chunks of its own. Only that merge waits for the attention kernel, so
// the slots stream while the prefix's last CTAs run (us per call, with the
// wait at the step's start -> in the merge: nine prefixes of up to 5003
// tokens over 67 ragged sequences 63 -> 50, a 16384-token prefix over 128
// full caches of 2400 slots 219 -> 213, of which the slots alone take 186 at
// the measured copy rate). Without a memset of the counters and pieces before
// the attention these take 48 and 212, one sequence of 2400 slots with a prefix
// of 1000 tokens 12.7 instead of 16.5.
#include "lf_step_kernel.cuh"

namespace lf {
namespace {

template <int D, int G>
cudaError_t launch_dg(const CUtensorMap& tmK, const CUtensorMap& tmV, const StepParams& p,
                      int units, cudaStream_t stream, int score, bool pdl) {
    return score ? launch_t<D, G, 2, true, false, true>(tmK, tmV, p, units, stream, pdl)
                 : launch_t<D, G, 2, false, false, true>(tmK, tmV, p, units, stream, pdl);
}

}  // namespace

cudaError_t launch_decode_step_prefix(int D, int G, int score, const CUtensorMap& tmK,
                                      const CUtensorMap& tmV, const StepParams& p, int units,
                                      cudaStream_t stream) {
    const char* env = std::getenv("LF_PDL");
    const bool pdl = !(env && std::atoi(env) == 0);
#define LF_STEP_CASE(DD, GG) \
    if (D == DD && G == GG) return launch_dg<DD, GG>(tmK, tmV, p, units, stream, score, pdl);
    LF_STEP_CASE(64, 1) LF_STEP_CASE(64, 2) LF_STEP_CASE(64, 4) LF_STEP_CASE(64, 8)
    LF_STEP_CASE(128, 1) LF_STEP_CASE(128, 2) LF_STEP_CASE(128, 4) LF_STEP_CASE(128, 8)
#undef LF_STEP_CASE
    return cudaErrorInvalidValue;
}

}  // namespace lf
