// Instantiations of the decode-step kernel that evict by the accumulated
// attention weight (the last-CTA merge and both rings of the cluster merge), and
// the selection of several slots behind it.
#include "lf_step_kernel.cuh"

namespace lf {
namespace {

// -------------------------------------------------------------- selection --
//
// The k lowest (key, slot) of a unit by one CTA: the step's scan has left a key
// per slot (0xffffffff: no candidate) in the slot's first score term. The k-th
// lowest key by its bytes from the top, with a histogram each; among equal keys
// the lowest slots, likewise, where not all of them are taken; then a bitonic
// sort of the winners. Latency bound: the keys of up to kSelectKeys slots are
// read once into shared memory, 32 warps at it. (The step's last CTA, with four
// warps and the keys in L2 at every pass, took 150 us for 9001 slots; this takes
// 8.)
constexpr int kSelectThreads = 1024;
constexpr int kSelectKeys = 49152;

struct Select {
    int hist[256];
    int digit, rank, same, count;
    uint32_t key[kMaxTopK];
    int slot[kMaxTopK];
};

template <int G>
__global__ void __launch_bounds__(kSelectThreads, 1) lf_select_kernel(const StepParams p, bool staged) {
    extern __shared__ uint32_t s_keys[];
    __shared__ Select s;
    allow_dependent_launch();
    grid_dependency_wait();
    const int u = blockIdx.x;
    const int S = p.S;
    const int tid = threadIdx.x;
    const int lane = tid & 31;
    const uint32_t* keys = reinterpret_cast<const uint32_t*>(p.stash) + static_cast<size_t>(u) * S * G;
    if (tid == 0) s.count = 0;
    __syncthreads();
    // The candidates counted (and their keys staged).
    int mine = 0;
#pragma unroll 8
    for (int j = tid; j < S; j += kSelectThreads) {
        const uint32_t key = __ldcg(keys + static_cast<size_t>(j) * G);
        if (staged) s_keys[j] = key;
        mine += key != 0xffffffffu;
    }
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0) atomicAdd(&s.count, mine);
    __syncthreads();
    const int keff = min(p.topk, s.count);
    const auto key_of = [&](int j) { return staged ? s_keys[j] : __ldcg(keys + static_cast<size_t>(j) * G); };
    // One byte of the rank-th smallest value of those in(j) whose higher bytes are
    // `prefix`; s.rank becomes the rank left, s.same how many share the byte.
    const auto pass = [&](int shift, uint32_t prefix, uint32_t pmask, const auto& value) {
        for (int i = tid; i < 256; i += kSelectThreads) s.hist[i] = 0;
        __syncthreads();
#pragma unroll 4
        for (int j = tid; j < S; j += kSelectThreads) {
            uint32_t v;
            if (value(j, &v) && (v & pmask) == prefix) atomicAdd(&s.hist[(v >> shift) & 255u], 1);
        }
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
            T |= pass(shift, T, shift == 24 ? 0u : ~0u << (shift + 8), [&](int j, uint32_t* v) {
                *v = key_of(j);
                return *v != 0xffffffffu;
            });
        // Among keys equal to T, the rank lowest slots: up to slot J.
        uint32_t J = 0xffffffffu;
        if (s.same != s.rank) {
            J = 0;
            for (int shift = 16; shift >= 0; shift -= 8)
                J |= pass(shift, J, shift == 16 ? 0u : ~0u << (shift + 8), [&](int j, uint32_t* v) {
                    *v = static_cast<uint32_t>(j);
                    return key_of(j) == T;
                });
        }
        __syncthreads();
        if (tid == 0) s.count = 0;
        __syncthreads();
        for (int j = tid; j < S; j += kSelectThreads) {
            const uint32_t key = key_of(j);
            if (key < T || (key == T && static_cast<uint32_t>(j) <= J)) {
                const int at = atomicAdd(&s.count, 1);
                s.key[at] = key;  // (keff of them: at < kMaxTopK)
                s.slot[at] = j;
            }
        }
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

template <int G>
cudaError_t launch_select_t(const StepParams& p, int units, cudaStream_t stream) {
    const bool staged = p.S <= kSelectKeys;
    cudaError_t e = allow_shared<lf_select_kernel<G>>(kSelectKeys * 4);
    if (e != cudaSuccess) return e;
    const char* env = std::getenv("LF_PDL");
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(units);
    cfg.blockDim = dim3(kSelectThreads);
    cfg.dynamicSmemBytes = staged ? static_cast<size_t>(p.S) * 4 : 0;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = (env && std::atoi(env) == 0) ? 0 : 1;
    e = cudaLaunchKernelEx(&cfg, lf_select_kernel<G>, p, staged);
    return e != cudaSuccess ? e : cudaGetLastError();
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
cudaError_t launch_select(int G, const StepParams& p, int units, cudaStream_t stream) {
    switch (G) {
        case 1: return launch_select_t<1>(p, units, stream);
        case 2: return launch_select_t<2>(p, units, stream);
        case 4: return launch_select_t<4>(p, units, stream);
        case 8: return launch_select_t<8>(p, units, stream);
        default: return cudaErrorInvalidValue;
    }
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
