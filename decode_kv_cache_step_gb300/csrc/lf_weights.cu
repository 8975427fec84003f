// Attention weights that a prompt's rows give its keys, summed (sm_103a): what
// eviction by accumulated weight starts from.
//
// w_j = sum over the counted rows i >= j and the heads h of a KV head of
// 2^(s_ihj - r_ih), s = scale * log2(e) * q.k, r_ih = log2 sum_j 2^(s_ihj).
// Two passes over the same products, since a weight needs its whole row's sum
// and a key's weights run across the rows:
//   rows     a CTA holds 128 query rows (128 / g tokens times the g heads that
//            share a KV head) and streams key tiles: each row's running maximum
//            and sum (in pieces of the key axis when rows are few);
//   columns  the products' transpose, so a thread owns a key and adds up its
//            weights in registers, in a fixed order. A CTA holds 128 keys and
//            streams the query tiles that see them; where no sequence has more
//            rows than one tile, it holds that tile and streams the keys.
// Neither pass writes a score. Both are one tensor product per tile, a thread
// issuing them into two accumulators in tensor memory, TMA loads ahead through a
// ring, and four warps that read the accumulators; two CTAs share an SM, so one's
// start and end run under the other's tiles.
#include <math.h>
#include <stdlib.h>

#include <algorithm>

#include "../../include/lf_decode.h"
#include "lf_kernels.h"
#include "lf_tcgen05.cuh"

namespace lf {
namespace {

constexpr int kRows = 128;                // rows of either operand's tile
constexpr int kPanel = kRows * 128;       // bytes of 64 columns of a tile
constexpr int kThreads = 192;             // four warps on the scores, loads, products
constexpr int kRing = 2;                  // tiles of the streamed operand
constexpr uint32_t kTmemCols = 2 * kRows;
constexpr int kMaxShare = 8;              // CTAs that share a tile of keys, a cluster

template <int D>
struct WeightsSmem {
    static constexpr int kTileBytes = kRows * D * 2;
    static constexpr int kRingOff = kTileBytes;
    static constexpr int kBarOff = kRingOff + kRing * kTileBytes;
    // barriers: held, full[], empty[], s_full[2], s_free[2], drain
    static constexpr int kBars = 1 + 2 * kRing + 5;
    static constexpr int kMiscOff = kBarOff + kBars * 8;
    static constexpr int kStatOff = (kMiscOff + 16 + 15) / 16 * 16;  // -r of two query tiles
    static constexpr int kTotalOff = kStatOff + 2 * kRows * 4;  // the cluster's sums
    static constexpr int kAlloc = kTotalOff + kMaxShare * kRows * 4 + 1024;
};

__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y, int z,
                                         uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// 2^x of two packed values.
__device__ __forceinline__ uint64_t ex2_pair(uint64_t x2) {
    float a, b;
    unpack_f32x2(x2, a, b);
    return pack_f32x2(ex2_approx(a), ex2_approx(b));
}

// The counted rows of a sequence: its tokens first .. r.n - 1.
__device__ __forceinline__ int first_row(const PromptWeightsParams& p, const SeqRange& r) {
    return p.rows > 0 ? max(0, r.n - p.rows) : 0;
}
// Index of a counted token among the rows' statistics.
__device__ __forceinline__ int stat_row(const PromptWeightsParams& p, int b, const SeqRange& r, int tok) {
    return p.by_sequence ? b * p.rows + tok - first_row(p, r) : r.q0 + tok;
}

// What a CTA does: its operand's tile, and the tiles streamed past it.
struct Work {
    int b, kvh;
    SeqRange r;
    int at;     // first token of the held rows, or first held key
    int first;  // first streamed key, or token
    int end;    // behind the last
};

// A tile of rows and a piece of the keys they see (rows pass; columns pass with
// few rows).
__device__ __forceinline__ bool rows_work(const PromptWeightsParams& p, int tok, bool report, Work* w) {
    const int item = p.items - 1 - static_cast<int>(blockIdx.x) / p.Hkv;  // longest rows first
    w->kvh = blockIdx.x % p.Hkv;
    // (There are at least as many items as sequences.)
    if (report && item < p.B && w->kvh == 0 && blockIdx.y == 0 && threadIdx.x == 0 &&
        !seq_range(p.q_start, p.kv_len, item, p.T, p.S, true, &w->r))
        atomicOr(p.dev_err, kErrBadLength);
    int rel;
    if (p.by_sequence) {
        const int per = (p.rows + tok - 1) / tok;
        w->b = item / per;
        rel = item % per;
    } else {
        // Sequence b's tiles start at floor(q_start[b] / tok) + b: enough for its
        // rows wherever they start.
        int lo = 0, hi = p.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.q_start[mid] / tok + mid <= item)
                lo = mid;
            else
                hi = mid - 1;
        }
        w->b = lo;
        rel = item - p.q_start[lo] / tok - lo;
    }
    if (!seq_range(p.q_start, p.kv_len, w->b, p.T, p.S, true, &w->r) || rel < 0) return false;
    w->at = first_row(p, w->r) + rel * tok;
    if (w->at >= w->r.n) return false;
    const int keys = w->r.kv - w->r.n + min(w->at + tok, w->r.n);  // the last row's
    const int tiles = (keys + kRows - 1) / kRows;
    const int pieces = gridDim.y;
    w->first = static_cast<int>(static_cast<int64_t>(tiles) * blockIdx.y / pieces) * kRows;
    w->end = min(keys, static_cast<int>(static_cast<int64_t>(tiles) * (blockIdx.y + 1) / pieces) * kRows);
    return true;
}

// 128 keys and this CTA's share of the rows that see one of them (columns pass).
__device__ __forceinline__ bool keys_work(const PromptWeightsParams& p, int tok, Work* w) {
    const int x = blockIdx.x / p.share, rank = blockIdx.x % p.share;
    w->kvh = x % p.Hkv;
    const int y = x / p.Hkv;
    w->b = y % p.B;
    w->at = y / p.B * kRows;
    if (!seq_range(p.q_start, p.kv_len, w->b, p.T, p.S, true, &w->r)) return false;
    if (w->r.n == 0 || w->at >= w->r.kv) return false;
    const int from = max(first_row(p, w->r), w->at - (w->r.kv - w->r.n));
    const int tiles = (w->r.n - from + tok - 1) / tok;
    w->first = from + static_cast<int>(static_cast<int64_t>(tiles) * rank / p.share) * tok;
    w->end = min(w->r.n, from + static_cast<int>(static_cast<int64_t>(tiles) * (rank + 1) / p.share) * tok);
    return true;
}

// The kernel's forms.
constexpr int kRowsPass = 0;
constexpr int kColumnsPass = 1;  // keys held
constexpr int kFewRows = 2;      // the columns pass with the one tile of rows held

template <int D, int kForm>
__global__ void __launch_bounds__(kThreads, 2)
    lf_prompt_weights_kernel(const __grid_constant__ CUtensorMap tmQ,
                             const __grid_constant__ CUtensorMap tmK,
                             const __grid_constant__ PromptWeightsParams p) {
    using L = WeightsSmem<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* held = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
    uint64_t* full = held + 1;
    uint64_t* empty = full + kRing;
    uint64_t* s_full = empty + kRing;
    uint64_t* s_free = s_full + 2;
    uint64_t* drain = s_free + 2;
    volatile uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
    float* stat = reinterpret_cast<float*>(smem + L::kStatOff);  // [2][kRows]
    float* totals = reinterpret_cast<float*>(smem + L::kTotalOff);  // [share][kRows]

    const int tid = threadIdx.x;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int lane = tid & 31;
    allow_dependent_launch();
    grid_dependency_wait();
    const int g = p.Hq / p.Hkv;
    const int gs = __ffs(g) - 1;
    const int tok = kRows >> gs;
    constexpr bool kKeysHeld = kForm == kColumnsPass;
    Work w;
    if (kKeysHeld ? !keys_work(p, tok, &w) : !rows_work(p, tok, kForm == kRowsPass, &w)) return;
    if (kForm != kRowsPass && !p.by_sequence) {
        // The rows pass finds packed tiles by their order: unless q_start ascends
        // nothing is written.
        bool good = true;
        for (int i = tid; i < p.B; i += kThreads) {
            const int from = p.q_start[i], to = p.q_start[i + 1];
            good = good && from >= 0 && from <= to && to <= p.T;
        }
        if (!__syncthreads_and(good)) return;
    }
    // (Every CTA of a cluster has work, or none.)
    const bool shared = kKeysHeld && p.share > 1;
    if (shared) cluster_arrive_relaxed();
    const int step = kKeysHeld ? tok : kRows;
    const int tiles = w.end > w.first ? (w.end - w.first + step - 1) / step : 0;

    if (warp == 5) {
        tmem_alloc(const_cast<uint32_t*>(misc), kTmemCols);
    } else if (warp == 4 && lane == 0) {
        mbar_init(held, 1);
        for (int s = 0; s < kRing; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&s_free[s], 4);
        }
        mbar_init(drain, 1);
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, misc[0], 0);
    const int unit = w.b * p.Hkv + w.kvh;
    const int past = w.r.kv - w.r.n;
    float my_total = 0.f;  // of a shared tile
    const auto store = [&](int j, float total) {
        if (j >= w.r.kv) return;
        float* dst = p.weights + static_cast<size_t>(unit) * p.S + j;
        *dst = j < past ? *dst + total : total;
    };

    if (warp == 4) {
        if (lane == 0 && tiles > 0) {
            // ----------------------------------------------------- loads --
            const auto load_q = [&](uint8_t* dst, int t, uint64_t* bar) {
                for (int c = 0; c < D / 64; ++c)
                    tma_load(dst + c * kPanel, &tmQ, c * 64, w.kvh << gs, w.r.q0 + t, bar);
            };
            const auto load_k = [&](uint8_t* dst, int j, uint64_t* bar) {
                for (int c = 0; c < D / 64; ++c)
                    for (int h = 0; h < 2; ++h)
                        tma_load(dst + c * kPanel + h * (kPanel / 2), &tmK, c * 64, j + h * 64, unit, bar);
            };
            mbar_arrive_expect_tx(held, L::kTileBytes);
            if (kKeysHeld)
                load_k(smem, w.at, held);
            else
                load_q(smem, w.at, held);
            int n = 0;
            for (; n < tiles; ++n) {
                const int st = n % kRing;
                if (!mbar_wait(&empty[st], ((n / kRing) & 1) ^ 1, p.wait_limit_ns)) {
                    atomicOr(p.dev_err, LF_DEVERR_WAIT_TIMEOUT);
                    break;
                }
                mbar_arrive_expect_tx(&full[st], L::kTileBytes);
                uint8_t* dst = smem + L::kRingOff + st * L::kTileBytes;
                if (kKeysHeld)
                    load_q(dst, w.first + n * step, &full[st]);
                else
                    load_k(dst, w.first + n * step, &full[st]);
            }
            // No copy may be in flight when the CTA leaves.
            mbar_wait(held, 0);
            for (int k = max(0, n - kRing); k < n; ++k) mbar_wait(&full[k % kRing], (k / kRing) & 1);
        }
        __syncwarp();
    } else if (warp == 5) {
        if (tiles > 0 && elect_one()) {
            // -------------------------------------------------- products --
            const uint32_t idesc = instr_desc(kRows, kRows, false) | (p.negate ? kInstrNegateA : 0u);
            // The accumulators' lanes are the keys, but for the rows pass: the
            // streamed tile is the first operand where the rows are held.
            const uint64_t hd = smem_desc(smem_u32(smem), 16, 1024);
            bool ok = mbar_wait(held, 0, p.wait_limit_ns);
            for (int n = 0; ok && n < tiles; ++n) {
                const int st = n % kRing, s = n & 1;
                ok = mbar_wait(&full[st], (n / kRing) & 1, p.wait_limit_ns) &&
                     mbar_wait(&s_free[s], ((n >> 1) & 1) ^ 1, p.wait_limit_ns);
                if (!ok) break;
                tc_fence_after();
                const uint64_t sd = smem_desc(smem_u32(smem + L::kRingOff + st * L::kTileBytes), 16, 1024);
                const uint64_t ad = kForm == kFewRows ? sd : hd;
                const uint64_t bd = kForm == kFewRows ? hd : sd;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t off = ((k >> 2) * kPanel + (k & 3) * 32) / 16;
                    mma_ss(tmem + s * kRows, ad + off, bd + off, idesc, k > 0);
                }
                mma_commit(&empty[st]);
                mma_commit(&s_full[s]);
            }
            if (!ok) atomicOr(p.dev_err, LF_DEVERR_WAIT_TIMEOUT);
            // No product may be in flight when tensor memory is freed.
            mma_commit(drain);
            mbar_wait(drain, 0);
        }
        __syncwarp();
    } else {
        // -------------------------------------------------------- scores --
        const uint32_t ts = tmem + (static_cast<uint32_t>(warp) << 21);
        const float c1 = p.scale_log2;
        const uint64_t c2 = pack_f32x2(c1, c1);
        const auto take = [&](int n, uint32_t (&x)[128]) {
            const bool ok = __all_sync(0xffffffffu, mbar_wait(&s_full[n & 1], (n >> 1) & 1, p.wait_limit_ns));
            if (!ok) return false;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 4; ++k) tmem_ld32(ts + (n & 1) * kRows + 32 * k, x + 32 * k);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_free[n & 1]);
            return true;
        };
        bool ok = true;
        // -r of the row of token t, head tid % g: -inf (no weight) without a sum.
        const size_t next_piece = static_cast<size_t>(p.stat_rows) * p.Hq;
        const auto stat_at = [&](int t) {
            return p.stats + static_cast<size_t>(stat_row(p, w.b, w.r, t)) * p.Hq + (w.kvh << gs) + (tid & (g - 1));
        };
        const auto minus_r = [&](float2 v) { return v.y == 0.f ? -INFINITY : -(v.x + __log2f(v.y)); };
        const auto joined = [&](int t) {
            const float2* src = stat_at(t);
            float2 sum = make_float2(-INFINITY, 0.f);
            for (int k = 0; k < p.pieces; ++k) sum.x = fmaxf(sum.x, __ldcg(src + k * next_piece).x);
            if (sum.x == -INFINITY) sum.x = 0.f;
            for (int k = 0; k < p.pieces; ++k) {
                const float2 v = __ldcg(src + k * next_piece);
                sum.y += v.y * exp2f(v.x - sum.x);
            }
            return sum;
        };
        // A key's weights of the tile's 128 rows; columns [lo, hi) see it.
        const auto column_sum = [&](uint32_t (&x)[128], const float* minus, bool some, int lo, int hi) {
            const float4* r4 = reinterpret_cast<const float4*>(minus);
            if (some) {
#pragma unroll
                for (int e = 0; e < 128; ++e) x[e] = e >= lo && e < hi ? x[e] : 0xff800000u;
            }
            uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < 128; e += 4) {
                const float4 r = r4[e >> 2];
                const uint64_t y0 = fma_f32x2(pack_f32x2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), c2,
                                              pack_f32x2(r.x, r.y));
                const uint64_t y1 = fma_f32x2(pack_f32x2(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), c2,
                                              pack_f32x2(r.z, r.w));
                const int q = e >> 1;
                sum[q & 3] = add_f32x2(sum[q & 3], ex2_pair(y0));
                sum[(q + 1) & 3] = add_f32x2(sum[(q + 1) & 3], ex2_pair(y1));
            }
            float a, b;
            unpack_f32x2(add_f32x2(add_f32x2(sum[0], sum[1]), add_f32x2(sum[2], sum[3])), a, b);
            return a + b;
        };
        if (kForm == kRowsPass) {
            // A thread owns the row of token w.at + tid / g, head tid % g.
            const int t = w.at + (tid >> gs);
            const int seen = past + t + 1;  // keys the row sees
            float m = -INFINITY, l = 0.f;
#pragma unroll 1
            for (int n = 0; n < tiles; ++n) {
                uint32_t x[128];
                if (!(ok = take(n, x))) break;
                const int j0 = w.first + n * kRows;
                // Some rows of the tile do not see its last keys.
                if (j0 + kRows > past + w.at + 1) {
#pragma unroll
                    for (int e = 0; e < 128; ++e) x[e] = j0 + e < seen ? x[e] : 0xff800000u;
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < 128; e += 2)
                    mx[(e >> 1) & 3] = fmaxf(fmaxf(mx[(e >> 1) & 3], __uint_as_float(x[e])), __uint_as_float(x[e + 1]));
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c1;
                const float to = fmaxf(m, top);
                const float base = to == -INFINITY ? 0.f : to;
                l *= ex2_approx(m - base);
                m = to;
                const uint64_t b2 = pack_f32x2(-base, -base);
                uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
                for (int q = 0; q < 64; ++q) {
                    const uint64_t y = fma_f32x2(pack_f32x2(__uint_as_float(x[2 * q]), __uint_as_float(x[2 * q + 1])), c2, b2);
                    sum[q & 3] = add_f32x2(sum[q & 3], ex2_pair(y));
                }
                float a, b;
                unpack_f32x2(add_f32x2(add_f32x2(sum[0], sum[1]), add_f32x2(sum[2], sum[3])), a, b);
                l += a + b;
            }
            if (t < w.r.n) const_cast<float2*>(stat_at(t))[blockIdx.y * next_piece] = make_float2(m, l);
        } else if (kForm == kColumnsPass) {
            // A thread owns key w.at + tid; columns are rows of the query tile.
            const int j = w.at + tid;
            // Statistics of the row that is this thread's column of tile n.
            const auto row_of = [&](int n) { return min(w.first + n * step + (tid >> gs), w.r.n - 1); };
            float total = 0.f;
            stat[tid] = minus_r(p.pieces > 1 ? joined(row_of(0)) : __ldcg(stat_at(row_of(0))));
            asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll 1
            for (int n = 0; n < tiles; ++n) {
                // (In flight while the tile is worked.)
                const float2 then = p.pieces > 1 ? joined(row_of(n + 1)) : __ldcg(stat_at(row_of(n + 1)));
                uint32_t x[128];
                // (A warp that has given up keeps to the barriers below.)
                ok = ok && take(n, x);
                const int t0 = w.first + n * step;
                // Column e is a row of token t0 + e / g. From token j - past on
                // they see the key, up to the sequence's last.
                const int there = (w.r.n - t0) << gs;
                const bool some = w.at + kRows > past + t0 + 1 || there < kRows;
                const float sum = column_sum(x, stat + (n & 1) * kRows, some, (j - past - t0) << gs, there);
                if (ok) total += sum;
                stat[((n + 1) & 1) * kRows + tid] = minus_r(then);
                asm volatile("bar.sync 1, 128;" ::: "memory");
            }
            if (shared)
                my_total = total;
            else
                store(j, total);
        } else {
            // Streamed keys; every tile's sums are final.
            stat[tid] = minus_r(joined(min(w.at + (tid >> gs), w.r.n - 1)));
            asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll 1
            for (int n = 0; n < tiles; ++n) {
                uint32_t x[128];
                if (!(ok = take(n, x))) break;
                const int j0 = w.first + n * kRows;
                const int there = (w.r.n - w.at) << gs;
                const bool some = j0 + kRows > past + w.at + 1 || there < kRows;
                store(j0 + tid, column_sum(x, stat, some, (j0 + tid - past - w.at) << gs, there));
            }
        }
        if (!ok && lane == 0) atomicOr(p.dev_err, LF_DEVERR_WAIT_TIMEOUT);
    }
    if (shared) {
        // The cluster's sums to its first CTA, added in the order of the rows.
        cluster_wait();  // its CTAs have all started
        if (tid < kRows) st_cluster(dsmem_addr(totals + cluster_ctarank() * kRows + tid, 0u), my_total);
        cluster_arrive();
        cluster_wait();
        if (cluster_ctarank() == 0 && tid < kRows) {
            float total = 0.f;
            for (int k = 0; k < p.share; ++k) total += totals[k * kRows + tid];
            store(w.at + tid, total);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 5) tmem_dealloc(tmem, kTmemCols);
}

template <int D, int kForm>
cudaError_t launch_pass(const CUtensorMap& tmQ, const CUtensorMap& tmK, const PromptWeightsParams& p,
                        dim3 grid, int cluster, cudaStream_t stream) {
    const auto kernel = lf_prompt_weights_kernel<D, kForm>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         WeightsSmem<D>::kAlloc);
    if (e != cudaSuccess) return e;
    const char* env = std::getenv("LF_PDL");
    cudaLaunchAttribute attr[2];
    int attrs = 0;
    if (!(env && std::atoi(env) == 0)) {
        attr[attrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[attrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[attrs].id = cudaLaunchAttributeClusterDimension;
        attr[attrs].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[attrs].val.clusterDim.y = 1;
        attr[attrs++].val.clusterDim.z = 1;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = WeightsSmem<D>::kAlloc;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = attrs;
    return cudaLaunchKernelEx(&cfg, kernel, tmQ, tmK, p);
}

template <int D>
cudaError_t launch_d(const CUtensorMap& tmQ, const CUtensorMap& tmK, const PromptWeightsParams& p,
                     cudaStream_t stream) {
    const dim3 rows(p.items * p.Hkv, p.pieces);
    const cudaError_t e = launch_pass<D, kRowsPass>(tmQ, tmK, p, rows, 1, stream);
    if (e != cudaSuccess) return e;
    if (p.share == 0) return launch_pass<D, kFewRows>(tmQ, tmK, p, rows, 1, stream);
    const int tiles = (p.S + kRows - 1) / kRows;
    return launch_pass<D, kColumnsPass>(tmQ, tmK, p, dim3(tiles * p.B * p.Hkv * p.share), p.share, stream);
}

}  // namespace

void plan_prompt_weights(PromptWeightsParams* p, int sms) {
    const int tok = kRows / (p->Hq / p->Hkv);
    const int64_t each = p->rows > 0 ? (p->rows + tok - 1) / tok : 0;
    const int64_t packed = p->T / tok + p->B;
    p->by_sequence = p->rows > 0 && each * p->B <= packed && static_cast<int64_t>(p->rows) * p->B < p->T;
    p->items = static_cast<int>(p->by_sequence ? each * p->B : packed);
    p->stat_rows = p->by_sequence ? p->rows * p->B : p->T;
    // Pieces of the keys when the tiles that hold rows leave SMs idle.
    const int64_t rows = p->rows > 0 ? std::min<int64_t>(p->T, static_cast<int64_t>(p->rows) * p->B) : p->T;
    const int64_t busy = std::max<int64_t>(1, (rows + tok - 1) / tok) * p->Hkv;
    const int64_t tiles = (p->S + kRows - 1) / kRows;
    // The columns pass: no tiles of keys (share 0) where no sequence has more rows
    // than a tile holds; else CTAs that share a tile's rows, so that the longest
    // CTA is short beside the whole (six waves of two CTAs an SM).
    const int64_t most = p->rows > 0 ? std::min(p->rows, p->T) : p->T;
    p->share = most <= tok ? 0 : 1;
    while (p->share > 0 && p->share < kMaxShare && p->share * tok * 2 < most &&
           tiles * p->B * p->Hkv * p->share < 12 * sms)
        p->share *= 2;
    p->pieces = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({tiles, 2 * sms / busy, 16})));
}

cudaError_t launch_prompt_weights(int D, const CUtensorMap& tmQ, const CUtensorMap& tmK,
                                  const PromptWeightsParams& p, cudaStream_t stream) {
    if (D == 64) return launch_d<64>(tmQ, tmK, p, stream);
    if (D == 128) return launch_d<128>(tmQ, tmK, p, stream);
    return cudaErrorInvalidValue;
}

}  // namespace lf
