// Instantiations of the decode-step kernel that evict by the accumulated
// attention weight (the last-CTA merge and both rings of the cluster merge), and
// the selection of several slots behind it.
#include "lf_step_kernel.cuh"

namespace lf {
namespace {

// -------------------------------------------------------------- selection --
//
// The k lowest (key, slot) of a unit by one CTA of 32 warps; the step's scan has
// left a key per slot (0xffffffff: no candidate). Latency bound.
constexpr int kSelectThreads = 1024;
constexpr int kHeldKeys = 16;  // keys of a thread in registers
constexpr int kMaxRounds = 8;
constexpr int kSelectKeys = 49152;

// Few slots: 16384 keys at a time in registers, and each round takes the lowest
// (key, slot) left; the k taken stay candidates beside the next 16384. (18 units
// of 9001 slots, us of the whole step: 2 slots 15.0, against 19.7 by the bytes as
// below; 8 slots 18.5 against 20.3; 16 slots 22.1 against 20.9; one sequence of
// 80000, 4 slots, 85.6 against 114.)
__global__ void __launch_bounds__(kSelectThreads, 1) lf_select_few_kernel(const StepParams p) {
    __shared__ uint32_t s_key[2][32], s_slot[2][32];
    allow_dependent_launch();
    grid_dependency_wait();
    const int u = blockIdx.x;
    const int S = p.S;
    const int tid = threadIdx.x;
    const int lane = tid & 31;
    const uint32_t* const keys = p.keys + static_cast<size_t>(u) * S;
    // Thread k's winner of round k so far.
    uint32_t won_key = 0xffffffffu, won_slot = 0;
    for (int j0 = tid; j0 - tid < S; j0 += kHeldKeys * kSelectThreads) {
        uint32_t key[kHeldKeys];
#pragma unroll
        for (int i = 0; i < kHeldKeys; ++i) {
            const int j = j0 + i * kSelectThreads;
            key[i] = j < S ? __ldcg(keys + j) : 0xffffffffu;
        }
        uint32_t old_key = won_key;
        const uint32_t old_slot = won_slot;
        won_key = 0xffffffffu;
        for (int k = 0; k < p.topk; ++k) {
            // The thread's lowest, among equal keys the lowest slot; so the warp's,
            // and the CTA's (every warp works it out).
            uint32_t low = old_key, at = old_slot;
#pragma unroll
            for (int i = 0; i < kHeldKeys; ++i)
                if (key[i] < low) {
                    low = key[i];
                    at = j0 + i * kSelectThreads;
                }
            const uint32_t warp_key = __reduce_min_sync(0xffffffffu, low);
            const uint32_t warp_slot = __reduce_min_sync(0xffffffffu, low == warp_key ? at : 0xffffffffu);
            if (lane == 0) {
                s_key[k & 1][tid >> 5] = warp_key;
                s_slot[k & 1][tid >> 5] = warp_slot;
            }
            __syncthreads();
            const uint32_t a_key = s_key[k & 1][lane];
            const uint32_t best = __reduce_min_sync(0xffffffffu, a_key);
            const uint32_t slot =
                __reduce_min_sync(0xffffffffu, a_key == best ? s_slot[k & 1][lane] : 0xffffffffu);
            if (low == best && at == slot) {  // taken
                if (at == old_slot) old_key = 0xffffffffu;
#pragma unroll
                for (int i = 0; i < kHeldKeys; ++i)
                    if (at == j0 + i * kSelectThreads) key[i] = 0xffffffffu;
            }
            if (tid == k) {
                won_key = best;
                won_slot = slot;
            }
        }
        __syncthreads();  // (an odd k leaves the next round the buffer just read)
    }
    if (tid < p.topk) {
        const bool some = won_key != 0xffffffffu;
        p.next_slot[static_cast<size_t>(u) * p.topk + tid] = some ? static_cast<int>(won_slot) : -1;
        if (some && (p.flags & kFlagMaskEvicted)) p.mask[static_cast<size_t>(u) * S + won_slot] = -1;
    }
}

// More slots: the k-th lowest key by its bytes from the top,
// with a histogram each; among equal keys the lowest slots, likewise, where not
// all of them are taken; then a bitonic sort of the winners. The keys of up to
// kSelectKeys slots are read once into shared memory. (18 units of 9001 slots: 64
// slots 23.0 us a step, 12.1 of them the step that returns one.)
struct Select {
    int hist[256];
    int digit, rank, same, count;
    uint32_t key[kMaxTopK];
    int slot[kMaxTopK];
};

__global__ void __launch_bounds__(kSelectThreads, 1) lf_select_kernel(const StepParams p, bool staged) {
    extern __shared__ uint32_t s_keys[];
    __shared__ Select s;
    allow_dependent_launch();
    grid_dependency_wait();
    const int u = blockIdx.x;
    const int S = p.S;
    const int tid = threadIdx.x;
    const int lane = tid & 31;
    const uint32_t* const keys = p.keys + static_cast<size_t>(u) * S;
    if (tid == 0) s.count = 0;
    __syncthreads();
    // visit(slot, key) for the thread's slots, from memory with eight keys in flight.
    const auto each = [&](bool from_shared, const auto& visit) {
        if (from_shared) {
#pragma unroll 4
            for (int j = tid; j < S; j += kSelectThreads) visit(j, s_keys[j]);
            return;
        }
        constexpr int kBatch = 8;
        for (int j0 = tid; j0 < S; j0 += kBatch * kSelectThreads) {
            uint32_t key[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int j = j0 + i * kSelectThreads;
                key[i] = j < S ? __ldcg(keys + j) : 0xffffffffu;
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (j0 + i * kSelectThreads < S) visit(j0 + i * kSelectThreads, key[i]);
        }
    };
    // The candidates counted (and their keys staged).
    int mine = 0;
    each(false, [&](int j, uint32_t key) {
        if (staged) s_keys[j] = key;
        mine += key != 0xffffffffu;
    });
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0) atomicAdd(&s.count, mine);
    __syncthreads();
    const int keff = min(p.topk, s.count);
    // One byte of the rank-th smallest value(slot, key) that there is whose higher bytes are
    // `prefix`; s.rank becomes the rank left, s.same how many share the byte.
    const auto pass = [&](int shift, uint32_t prefix, uint32_t pmask, const auto& value) {
        for (int i = tid; i < 256; i += kSelectThreads) s.hist[i] = 0;
        __syncthreads();
        each(staged, [&](int j, uint32_t key) {
            uint32_t v;
            if (value(j, key, &v) && (v & pmask) == prefix) atomicAdd(&s.hist[(v >> shift) & 255u], 1);
        });
        __syncthreads();
        if (tid < 32) {
            // Lane i: bins 8 i .. 8 i + 7.
            int n[8], sum = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) sum += n[k] = s.hist[8 * lane + k];
            int upto = sum;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, upto, off);
                if (lane >= off) upto += x;
            }
            const int rank = s.rank;
            __syncwarp();
            int before = upto - sum;
            if (before < rank && upto >= rank) {
                int k = 0;
                while (before + n[k] < rank) before += n[k++];
                s.digit = 8 * lane + k;
                s.rank = rank - before;
                s.same = n[k];
            }
        }
        __syncthreads();
        return static_cast<uint32_t>(s.digit) << shift;
    };
    if (keff > 0) {
        if (tid == 0) s.rank = keff;
        __syncthreads();
        uint32_t T = 0;
        for (int shift = 24; shift >= 0; shift -= 8)
            T |= pass(shift, T, shift == 24 ? 0u : ~0u << (shift + 8), [&](int, uint32_t key, uint32_t* v) {
                *v = key;
                return key != 0xffffffffu;
            });
        // Among keys equal to T, the rank lowest slots: up to slot J.
        uint32_t J = 0xffffffffu;
        if (s.same != s.rank) {
            J = 0;
            for (int shift = 16; shift >= 0; shift -= 8)
                J |= pass(shift, J, shift == 16 ? 0u : ~0u << (shift + 8), [&](int j, uint32_t key, uint32_t* v) {
                    *v = static_cast<uint32_t>(j);
                    return key == T;
                });
        }
        __syncthreads();
        if (tid == 0) s.count = 0;
        __syncthreads();
        each(staged, [&](int j, uint32_t key) {
            if (key < T || (key == T && static_cast<uint32_t>(j) <= J)) {
                const int at = atomicAdd(&s.count, 1);
                s.key[at] = key;  // (keff of them: at < kMaxTopK)
                s.slot[at] = j;
            }
        });
        __syncthreads();
        int n2 = 1;
        while (n2 < keff) n2 <<= 1;
        if (tid >= keff && tid < n2) {
            s.key[tid] = 0xffffffffu;
            s.slot[tid] = 0x7fffffff;
        }
        for (int size = 2; size <= n2; size <<= 1) {
            for (int step = size >> 1; step > 0; step >>= 1) {
                __syncthreads();
                const int i = tid, other = tid ^ step;
                if (i < n2 && other > i) {
                    const bool up = (i & size) == 0;
                    if (key_less(s.key[other], s.slot[other], s.key[i], s.slot[i]) == up) {
                        const uint32_t key = s.key[i];
                        const int slot = s.slot[i];
                        s.key[i] = s.key[other];
                        s.slot[i] = s.slot[other];
                        s.key[other] = key;
                        s.slot[other] = slot;
                    }
                }
            }
        }
        __syncthreads();
    }
    if (tid < p.topk) {
        const int slot = tid < keff ? s.slot[tid] : -1;
        p.next_slot[static_cast<size_t>(u) * p.topk + tid] = slot;
        if (slot >= 0 && (p.flags & kFlagMaskEvicted)) p.mask[static_cast<size_t>(u) * S + slot] = -1;
    }
}

template <int D, int G>
cudaError_t launch_dg(const CUtensorMap& tmK, const CUtensorMap& tmV, const StepParams& p,
                      int units, cudaStream_t stream, int stages, bool cluster, bool pdl) {
    if (!cluster) return launch_t<D, G, 2, kWeights, false>(tmK, tmV, p, units, stream, pdl);
    return stages == kDeepStages
               ? launch_t<D, G, kDeepStages, kWeights, true>(tmK, tmV, p, units, stream, pdl)
               : launch_t<D, G, 2, kWeights, true>(tmK, tmV, p, units, stream, pdl);
}

}  // namespace

static_assert(kMaxTopK <= kSelectThreads, "a thread per winner");
cudaError_t launch_select(const StepParams& p, int units, cudaStream_t stream) {
    const char* env = std::getenv("LF_PDL");
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(units);
    cfg.blockDim = dim3(kSelectThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = (env && std::atoi(env) == 0) ? 0 : 1;
    if (p.topk <= kMaxRounds)
        return cudaLaunchKernelEx(&cfg, lf_select_few_kernel, p);
    const bool staged = p.S <= kSelectKeys;
    cfg.dynamicSmemBytes = staged ? static_cast<size_t>(p.S) * 4 : 0;
    const cudaError_t e = allow_shared<lf_select_kernel>(kSelectKeys * 4);
    return e != cudaSuccess ? e : cudaLaunchKernelEx(&cfg, lf_select_kernel, p, staged);
}

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
