// Attention weights that a prompt's rows give its keys, summed (sm_103a): what
// eviction by accumulated weight starts from.
//
// w_j = sum over the counted rows i >= j and the heads h of a KV head of
// 2^(s_ihj - r_ih), s = scale * log2(e) * q.k, r_ih = log2 sum_j 2^(s_ihj).
// Two passes over the same products, since a weight needs its whole row's sum
// and a key's weights run across the rows:
//   rows     a CTA holds tiles of 128 query rows (128 / g tokens times the g heads
//            that share a KV head) and streams key tiles: each row's running
//            maximum and sum (in pieces of the key axis when rows are few);
//   columns  the products' transpose, so a thread owns a key and adds up its
//            weights in registers, in a fixed order. A CTA holds tiles of 128 keys
//            and streams the query tiles that see them; where no sequence has more
//            rows than one tile, it holds that tile and streams the keys.
// Neither pass writes a score. One thread, or two, issues the tensor products (a held
// tile times the streamed one) into four accumulators in tensor memory, all of it, and
// TMA loads run ahead through a ring. Four warps read an accumulator, each thread
// its lane's 128 scores, so sixteen of the SM's warps hide one another's waits.
// Large calls hold two tiles per CTA (a streamed tile then serves 256 rows) and
// have two accumulators for each; few rows hold one, and its accumulators take
// every fourth tile.
//
// What bounds it: the score warps. A tile of scores is 512 cycles of products, as
// many of exponentials, and some 470 instructions for each of the SM's schedulers;
// alone the products would take 341 us of some 430, the rest alone 420. (Streamed
// tiles of 256 rows, with less to read for the products: 467. Eight score warps with
// two accumulators each: 500. A third of the exponentials as polynomials: slower.
// Waits that poll: the same.) Measured (32 query, 8 KV heads of 128): every row of
// 8192 tokens 430 us in short runs and 436 called without a pause, some 205 and 225 a
// pass, 1270 TFLOP/s of both passes' products; the last 32 rows of 8 prompts of 2000 to
// 8192 tokens 41.4 us, two passes over 113 MB of keys (the second from L2 in part), where
// a CTA's start and the few tiles it streams take the most. One row takes as long.
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
constexpr int kMaxShare = 8;              // CTAs that share tiles of keys, a cluster

// The kernel's forms.
constexpr int kRowsPass = 0;
constexpr int kColumnsPass = 1;  // keys held
constexpr int kFewRows = 2;      // the columns pass with the one tile of rows held

constexpr int kScoreWarps = 16;
constexpr uint32_t kTmemCols = 4 * kRows;

template <int D, int kHeld>
struct WeightsSmem {
    static constexpr int kTurns = 4 / kHeld;  // accumulators of a held tile
    // Warps that issue products, behind the loads' warp: a streamed tile's waits,
    // issue and commits take one warp longer than the products with one held tile
    // (last 32 rows of 8 prompts: 42.9 us with one, 41.0 with two), not with two
    // (8192 tokens: 443 and 453).
    static constexpr int kIssuers = kHeld == 2 ? 1 : 2;
    static constexpr int kThreads = (kScoreWarps + 1 + kIssuers) * 32;
    static constexpr int kRing = D == 64 ? 8 : 4;  // streamed tiles
    // An issuer sees every use of the slots it waits for: it could not tell one
    // round of a barrier from the one after the next.
    static_assert(kRing % kIssuers == 0, "a slot's tiles have one issuer");
    static constexpr int kTileBytes = kRows * D * 2;
    static constexpr int kRingOff = kHeld * kTileBytes;
    static constexpr int kBarOff = kRingOff + kRing * kTileBytes;
    // barriers: held, full[], empty[], stat_full[], stat_free[], s_full[], s_free[],
    // drain[]
    static constexpr int kBars = 1 + 4 * kRing + 8 + kIssuers;
    static constexpr int kMiscOff = kBarOff + kBars * 8;
    static constexpr int kStatOff = (kMiscOff + 16 + 15) / 16 * 16;  // -r of the ring's rows
    static constexpr int kOtherOff = kStatOff + kRing * kRows * 4;  // the other turns' results
    static constexpr int kTotalOff = kOtherOff + (4 - kHeld) * kRows * 8;  // the cluster's sums
    static constexpr int kAlloc = kTotalOff + kMaxShare * kHeld * kRows * 4 + 1024;
    static_assert(kAlloc <= 232448, "shared memory of a CTA");
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

__device__ __forceinline__ uint64_t pair_at(const uint32_t* x) {
    return pack_f32x2(__uint_as_float(x[0]), __uint_as_float(x[1]));
}

// The counted rows of a sequence: its tokens first .. r.n - 1.
__device__ __forceinline__ int first_row(const PromptWeightsParams& p, const SeqRange& r) {
    return p.rows > 0 ? max(0, r.n - p.rows) : 0;
}
// Index of a counted token among the rows' statistics.
__device__ __forceinline__ int stat_row(const PromptWeightsParams& p, int b, const SeqRange& r, int tok) {
    return p.by_sequence ? b * p.rows + tok - first_row(p, r) : r.q0 + tok;
}

// What a CTA does: the tiles it holds, and those streamed past them.
struct Work {
    int b, kvh;
    SeqRange r;
    int at;     // first token of the held rows, or first held key
    int held;   // tiles that hold something
    int first;  // first streamed key, or token
    int end;    // behind the last
};

// Tiles of rows and a piece of the keys they see (rows pass; columns pass with few
// rows). tok: tokens of a tile.
__device__ __forceinline__ bool rows_work(const PromptWeightsParams& p, int tok, int tiles_held, bool report,
                                          Work* w) {
    const int item = p.items - 1 - static_cast<int>(blockIdx.x) / p.Hkv;  // longest rows first
    const int span = tok * tiles_held;
    w->kvh = blockIdx.x % p.Hkv;
    // (There are at least as many items as sequences.)
    if (report && item < p.B && w->kvh == 0 && blockIdx.y == 0 && threadIdx.x == 0 &&
        !seq_range(p.q_start, p.kv_len, item, p.T, p.S, true, &w->r))
        atomicOr(p.dev_err, kErrBadLength);
    int rel;
    if (p.by_sequence) {
        const int per = (p.rows + span - 1) / span;
        w->b = item / per;
        rel = item % per;
    } else {
        // Sequence b's items start at floor(q_start[b] / span) + b: enough for its
        // rows wherever they start.
        int lo = 0, hi = p.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.q_start[mid] / span + mid <= item)
                lo = mid;
            else
                hi = mid - 1;
        }
        w->b = lo;
        rel = item - p.q_start[lo] / span - lo;
    }
    if (!seq_range(p.q_start, p.kv_len, w->b, p.T, p.S, true, &w->r) || rel < 0) return false;
    w->at = first_row(p, w->r) + rel * span;
    if (w->at >= w->r.n) return false;
    const int rows = min(span, w->r.n - w->at);
    w->held = (rows + tok - 1) / tok;
    const int keys = w->r.kv - w->r.n + w->at + rows;  // the last row's
    w->first = blockIdx.y * p.piece_tiles * kRows;
    w->end = min(keys, w->first + p.piece_tiles * kRows);
    return w->first < keys;
}

// Pieces that the rows pass leaves of token t's rows.
__device__ __forceinline__ int row_pieces(const PromptWeightsParams& p, int span, const SeqRange& r, int t) {
    const int first = first_row(p, r);
    const int keys = r.kv - r.n + min(r.n, first + ((t - first) / span + 1) * span);
    return (keys + p.piece_tiles * kRows - 1) / (p.piece_tiles * kRows);
}

// Tiles of keys and this CTA's share of the rows that see one of them (columns pass).
__device__ __forceinline__ bool keys_work(const PromptWeightsParams& p, int tok, int tiles_held, Work* w) {
    const int x = blockIdx.x / p.share, rank = blockIdx.x % p.share;
    w->kvh = x % p.Hkv;
    const int y = x / p.Hkv;
    w->b = y % p.B;
    w->at = y / p.B * (tiles_held * kRows);
    if (!seq_range(p.q_start, p.kv_len, w->b, p.T, p.S, true, &w->r)) return false;
    if (w->r.n == 0 || w->at >= w->r.kv) return false;
    w->held = min(tiles_held, (w->r.kv - w->at + kRows - 1) / kRows);
    const int from = max(first_row(p, w->r), w->at - (w->r.kv - w->r.n));
    const int tiles = (w->r.n - from + tok - 1) / tok;
    w->first = from + static_cast<int>(static_cast<int64_t>(tiles) * rank / p.share) * tok;
    w->end = min(w->r.n, from + static_cast<int>(static_cast<int64_t>(tiles) * (rank + 1) / p.share) * tok);
    return true;
}

template <int D, int kForm, int kHeld>
__global__ void __launch_bounds__(WeightsSmem<D, kHeld>::kThreads, 1)
    lf_prompt_weights_kernel(const __grid_constant__ CUtensorMap tmQ,
                             const __grid_constant__ CUtensorMap tmK,
                             const __grid_constant__ PromptWeightsParams p) {
    using L = WeightsSmem<D, kHeld>;
    constexpr int kTurns = L::kTurns;
    constexpr int kIssuers = L::kIssuers;
    constexpr int kThreads = L::kThreads;
    constexpr bool kKeysHeld = kForm == kColumnsPass;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* held = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
    uint64_t* full = held + 1;
    uint64_t* empty = full + L::kRing;
    uint64_t* stat_full = empty + L::kRing;
    uint64_t* stat_free = stat_full + L::kRing;
    uint64_t* s_full = stat_free + L::kRing;  // [held tile][turn]
    uint64_t* s_free = s_full + 4;
    uint64_t* drain = s_free + 4;
    volatile uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
    float* stat = reinterpret_cast<float*>(smem + L::kStatOff);       // [kRing][kRows]
    float2* other = reinterpret_cast<float2*>(smem + L::kOtherOff);   // [turn - 1][kHeld][kRows]
    float* totals = reinterpret_cast<float*>(smem + L::kTotalOff);    // [share][kHeld][kRows]

    const int tid = threadIdx.x;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int lane = tid & 31;
    allow_dependent_launch();
    grid_dependency_wait();
    const int g = p.Hq / p.Hkv;
    const int gs = __ffs(g) - 1;
    const int tok = kRows >> gs;
    Work w;
    if (kKeysHeld ? !keys_work(p, tok, kHeld, &w) : !rows_work(p, tok, kHeld, kForm == kRowsPass, &w)) return;
    if (kForm != kRowsPass && !p.by_sequence) {
        // The rows pass finds packed rows by their order: unless q_start ascends
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
    const int step = kKeysHeld ? tok : kRows;  // tokens or keys of a streamed tile
    const int tiles = w.end > w.first ? (w.end - w.first + step - 1) / step : 0;

    if (warp == kScoreWarps + 1) {
        tmem_alloc(const_cast<uint32_t*>(misc), kTmemCols);
    } else if (warp == kScoreWarps && lane == 0) {
        mbar_init(held, 1);
        for (int s = 0; s < L::kRing; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], w.held);
            mbar_init(&stat_full[s], 1);
            mbar_init(&stat_free[s], 4 * w.held);
        }
        for (int s = 0; s < 4; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&s_free[s], 4);
        }
        for (int i = 0; i < kIssuers; ++i) mbar_init(&drain[i], 1);
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, misc[0], 0);
    const int unit = w.b * p.Hkv + w.kvh;
    const int past = w.r.kv - w.r.n;

    // (m, l) of the row of token t, head `column` % g: its pieces joined.
    const size_t piece = static_cast<size_t>(p.stat_rows) * p.Hq;
    const auto stat_at = [&](int t, int column) {
        return p.stats + static_cast<size_t>(stat_row(p, w.b, w.r, t)) * p.Hq + (w.kvh << gs) + (column & (g - 1));
    };
    const auto joined = [&](int t, int column) {
        const float2* src = stat_at(t, column);
        float2 sum = __ldcg(src);
        if (!kKeysHeld && p.pieces > 1) {
            const int pieces = row_pieces(p, kHeld * tok, w.r, t);
            float m = sum.x;
            for (int k = 1; k < pieces; ++k) m = fmaxf(m, __ldcg(src + k * piece).x);
            if (m == -INFINITY) m = 0.f;
            float l = 0.f;
            for (int k = 0; k < pieces; ++k) {
                const float2 v = __ldcg(src + k * piece);
                l += v.y * exp2f(v.x - m);
            }
            sum = make_float2(m, l);
        }
        return sum;
    };
    // -r, -inf (no weight) for a row without a sum.
    const auto minus_r = [](float2 v) { return v.y == 0.f ? -INFINITY : -(v.x + __log2f(v.y)); };
    const auto give_up = [&]() { atomicOr(p.dev_err, LF_DEVERR_WAIT_TIMEOUT); };

    float m = -INFINITY, l = 0.f;  // a thread's row; l alone: its key's weights
    if (warp == kScoreWarps) {
        // --------------------------------------------------------- loads --
        const auto load_q = [&](uint8_t* dst, int t, uint64_t* bar) {
            for (int c = 0; c < D / 64; ++c)
                tma_load(dst + c * kPanel, &tmQ, c * 64, w.kvh << gs, w.r.q0 + t, bar);
        };
        const auto load_k = [&](uint8_t* dst, int j, uint64_t* bar) {
            for (int c = 0; c < D / 64; ++c)
                for (int h = 0; h < 2; ++h)
                    tma_load(dst + c * kPanel + h * (kPanel / 2), &tmK, c * 64, j + h * 64, unit, bar);
        };
        if (lane == 0 && tiles > 0) {
            mbar_arrive_expect_tx(held, w.held * L::kTileBytes);
            for (int h = 0; h < w.held; ++h) {
                if (kKeysHeld)
                    load_k(smem + h * L::kTileBytes, w.at + h * kRows, held);
                else
                    load_q(smem + h * L::kTileBytes, w.at + h * tok, held);
            }
        }
        // The statistics of a tile's rows, four a lane, are loaded a tile ahead: a
        // round trip to L2 takes as long as a tile. (A row behind the sequence's
        // last gets that one's; it is masked.)
        float2 now[4], next[4];
        const auto statistics = [&](int n, float2 (&v)[4]) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int column = e * 32 + lane;
                v[e] = joined(min(w.first + n * step + (column >> gs), w.r.n - 1), column);
            }
        };
        if (kKeysHeld) statistics(0, next);
        int n = 0;
        for (; n < tiles; ++n) {
            if (kKeysHeld) {
#pragma unroll
                for (int e = 0; e < 4; ++e) now[e] = next[e];
                statistics(n + 1, next);
            }
            const int st = n % L::kRing;
            const int parity = ((n / L::kRing) & 1) ^ 1;
            bool ok = mbar_wait(&empty[st], parity, p.wait_limit_ns);
            if (kKeysHeld) ok = ok && mbar_wait(&stat_free[st], parity, p.wait_limit_ns);
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0) give_up();
                break;
            }
            if (lane == 0) {
                mbar_arrive_expect_tx(&full[st], L::kTileBytes);
                uint8_t* dst = smem + L::kRingOff + st * L::kTileBytes;
                if (kKeysHeld)
                    load_q(dst, w.first + n * step, &full[st]);
                else
                    load_k(dst, w.first + n * step, &full[st]);
            }
            if (kKeysHeld) {
#pragma unroll
                for (int e = 0; e < 4; ++e) stat[st * kRows + e * 32 + lane] = minus_r(now[e]);
                __syncwarp();
                if (lane == 0) mbar_arrive(&stat_full[st]);
            }
        }
        // No copy may be in flight when the CTA leaves.
        if (lane == 0 && tiles > 0) {
            mbar_wait(held, 0);
            for (int k = max(0, n - L::kRing); k < n; ++k) mbar_wait(&full[k % L::kRing], (k / L::kRing) & 1);
        }
        __syncwarp();
    } else if (warp > kScoreWarps) {
        if (tiles > 0 && elect_one()) {
            // -------------------------------------------------- products --
            // The accumulators' lanes are the keys, but for the rows pass: the
            // streamed tile is the first operand where the rows are held.
            const uint32_t idesc = instr_desc(kRows, kRows, false) | (p.negate ? kInstrNegateA : 0u);
            const int issuer = warp - kScoreWarps - 1;
            bool ok = mbar_wait(held, 0, p.wait_limit_ns);
            for (int n = issuer; ok && n < tiles; n += kIssuers) {
                const int st = n % L::kRing, s = n % kTurns;
                ok = mbar_wait(&full[st], (n / L::kRing) & 1, p.wait_limit_ns);
                if (!ok) break;
                const uint64_t sd = smem_desc(smem_u32(smem + L::kRingOff + st * L::kTileBytes), 16, 1024);
                for (int h = 0; ok && h < w.held; ++h) {
                    ok = mbar_wait(&s_free[kTurns * h + s], ((n / kTurns) & 1) ^ 1, p.wait_limit_ns);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t hd = smem_desc(smem_u32(smem + h * L::kTileBytes), 16, 1024);
                    const uint64_t ad = kForm == kFewRows ? sd : hd;
                    const uint64_t bd = kForm == kFewRows ? hd : sd;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint64_t off = ((k >> 2) * kPanel + (k & 3) * 32) / 16;
                        mma_ss(tmem + (kTurns * h + s) * kRows, ad + off, bd + off, idesc, k > 0);
                    }
                    mma_commit(&s_full[kTurns * h + s]);
                }
            }
            if (!ok) give_up();
            // No product may be in flight when tensor memory is freed.
            mma_commit(&drain[issuer]);
            mbar_wait(&drain[issuer], 0);
        }
        __syncwarp();
    } else if ((warp >> 2) % kHeld < w.held) {
        // -------------------------------------------------------- scores --
        const int h = (warp >> 2) % kHeld;      // held tile
        const int s = (warp >> 2) / kHeld;      // its turn of the streamed tiles
        const int at = (warp & 3) * 32 + lane;  // the thread's lane of the accumulator
        const uint32_t ts = tmem + (static_cast<uint32_t>(warp & 3) << 21) + (kTurns * h + s) * kRows;
        const float c1 = p.scale_log2;
        const uint64_t c2 = pack_f32x2(c1, c1);
        const auto arrived = [&](uint64_t* bar, int parity) {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, p.wait_limit_ns)) != 0;
        };
        // Half of a tile's 128 scores; behind the last the accumulator is free.
        const auto take = [&](int half, bool last, uint32_t (&x)[64]) {
            tmem_ld32(ts + half * 64, x);
            tmem_ld32(ts + half * 64 + 32, x + 32);
            tmem_wait_ld();
            if (last) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_free[kTurns * h + s]);
            }
        };
        const auto sum4 = [](const uint64_t (&sum)[4]) {
            float a, b;
            unpack_f32x2(add_f32x2(add_f32x2(sum[0], sum[1]), add_f32x2(sum[2], sum[3])), a, b);
            return a + b;
        };
        // A key's weights of a tile's rows; columns [lo, hi) see it.
        const auto column_sum = [&](const float* minus, bool some, int lo, int hi) {
            float total = 0.f;
            // A masked logit of -infinity and a row's statistic that is NaN give NaN: where
            // such a row lies in a tile that not all its keys see, columns are left out instead.
            // (The test costs nothing: 8192 tokens 430 us with it and without.)
            const float4 v = some ? reinterpret_cast<const float4*>(minus)[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
            if (some && __any_sync(0xffffffffu, isnan(v.x) || isnan(v.y) || isnan(v.z) || isnan(v.w))) {
#pragma unroll 1
                for (int e0 = 0; e0 < kRows; e0 += 16) {
                    uint32_t x[16];
                    tmem_ld16(ts + e0, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float w = ex2_approx(fmaf(__uint_as_float(x[e]), c1, minus[e0 + e]));
                        total += e0 + e >= lo && e0 + e < hi ? w : 0.f;
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_free[kTurns * h + s]);
                return total;
            }
            // (Few rows may leave the second half without a row: 8 rows 40.8 us for 48.9.)
            const int halves = kForm == kFewRows && hi <= kRows / 2 ? 1 : 2;
            // (Both halves' code, 20 us less of 450 for 8192 tokens; a few rows spill.)
#pragma unroll(kForm == kColumnsPass ? 2 : 1)
            for (int half = 0; half < halves; ++half) {
                uint32_t x[64];
                take(half, half + 1 == halves, x);
                if (some) {
#pragma unroll
                    for (int e = 0; e < 64; ++e) x[e] = half * 64 + e >= lo && half * 64 + e < hi ? x[e] : 0xff800000u;
                }
                const float4* r4 = reinterpret_cast<const float4*>(minus + half * 64);
                uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
                for (int e = 0; e < 64; e += 4) {
                    const float4 r = r4[e >> 2];
                    uint64_t& s0 = sum[(e >> 1) & 3];
                    uint64_t& s1 = sum[((e >> 1) + 1) & 3];
                    s0 = add_f32x2(s0, ex2_pair(fma_f32x2(pair_at(x + e), c2, pack_f32x2(r.x, r.y))));
                    s1 = add_f32x2(s1, ex2_pair(fma_f32x2(pair_at(x + e + 2), c2, pack_f32x2(r.z, r.w))));
                }
                total += sum4(sum);
            }
            return total;
        };
        bool ok = true;
        if (kForm == kFewRows) {
            // The streamed tiles are keys; their sums are final.
            if (s == 0) stat[at] = minus_r(joined(min(w.at + (at >> gs), w.r.n - 1), at));
            asm volatile("bar.sync 1, 512;" ::: "memory");
        }
#pragma unroll 1
        for (int n = s; n < tiles; n += kTurns) {
            if (!(ok = arrived(&s_full[kTurns * h + s], (n / kTurns) & 1))) break;
            tc_fence_after();
            // (The streamed tile's products with this held one are done.)
            if ((warp & 3) == 0 && lane == 0) mbar_arrive(&empty[n % L::kRing]);
            if (kForm == kRowsPass) {
                // A thread owns the row of token w.at + h * tok + at / g, head at % g.
                const int t0 = w.at + h * tok;
                const int j0 = w.first + n * kRows;
                const int seen = past + t0 + (at >> gs) + 1 - j0;  // of the tile's keys
                const bool some = j0 + kRows > past + t0 + 1;
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    uint32_t x[64];
                    take(half, half == 1, x);
                    if (some) {
#pragma unroll
                        for (int e = 0; e < 64; ++e) x[e] = half * 64 + e < seen ? x[e] : 0xff800000u;
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < 64; e += 2)
                        mx[(e >> 1) & 3] =
                            fmaxf(fmaxf(mx[(e >> 1) & 3], __uint_as_float(x[e])), __uint_as_float(x[e + 1]));
                    const float to = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c1);
                    const float base = to == -INFINITY ? 0.f : to;
                    l *= ex2_approx(m - base);
                    m = to;
                    const uint64_t b2 = pack_f32x2(-base, -base);
                    uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int e = 0; e < 64; e += 2)
                        sum[(e >> 1) & 3] = add_f32x2(sum[(e >> 1) & 3], ex2_pair(fma_f32x2(pair_at(x + e), c2, b2)));
                    l += sum4(sum);
                }
            } else if (kForm == kColumnsPass) {
                // A thread owns key j; column e is a row of token t0 + e / g. From
                // token j - past on they see the key, up to the sequence's last.
                const int st = n % L::kRing;
                if (!(ok = arrived(&stat_full[st], (n / L::kRing) & 1))) break;
                const int j0 = w.at + h * kRows;
                const int t0 = w.first + n * step;
                const int there = (w.r.n - t0) << gs;
                const bool some = j0 + kRows > past + t0 + 1 || there < kRows;
                l += column_sum(stat + st * kRows, some, (j0 + at - past - t0) << gs, there);
                __syncwarp();
                if (lane == 0) mbar_arrive(&stat_free[st]);
            } else {
                const int j0 = w.first + n * kRows;
                const int there = (w.r.n - w.at) << gs;
                const bool some = j0 + kRows > past + w.at + 1 || there < kRows;
                const float total = column_sum(stat, some, (j0 + at - past - w.at) << gs, there);
                if (j0 + at < w.r.kv) {
                    float* dst = p.weights + static_cast<size_t>(unit) * p.S + j0 + at;
                    *dst = j0 + at < past ? *dst + total : total;
                }
            }
        }
        if (!ok && lane == 0) give_up();
        if (s > 0) other[((s - 1) * kHeld + h) * kRows + at] = make_float2(m, l);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kScoreWarps + 1) tmem_dealloc(tmem, kTmemCols);
    if (kForm == kFewRows) return;
    // The first turn's threads take the others' results.
    const int h = warp >> 2;
    const int at = tid & (kRows - 1);
    const bool mine = h < kHeld && h < w.held;
    if (mine) {
#pragma unroll
        for (int s = 1; s < kTurns; ++s) {
            const float2 v = other[((s - 1) * kHeld + h) * kRows + at];
            if (kForm == kRowsPass) {
                const float to = fmaxf(m, v.x);
                const float base = to == -INFINITY ? 0.f : to;
                l = l * ex2_approx(m - base) + v.y * ex2_approx(v.x - base);
                m = to;
            } else {
                l += v.y;
            }
        }
        const int t = w.at + h * tok + (at >> gs);
        if (kForm == kRowsPass && t < w.r.n)
            const_cast<float2*>(stat_at(t, at))[blockIdx.y * piece] = make_float2(m, l);
    }
    if (kForm == kColumnsPass) {
        if (shared) {
            // The cluster's sums to its first CTA, added in the order of the rows.
            cluster_wait();  // its CTAs have all started
            if (mine) st_cluster(dsmem_addr(totals + (cluster_ctarank() * kHeld + h) * kRows + at, 0u), l);
            cluster_arrive();
            cluster_wait();
            if (cluster_ctarank() != 0) return;
            if (mine) {
                l = 0.f;
                for (int k = 0; k < p.share; ++k) l += totals[(k * kHeld + h) * kRows + at];
            }
        }
        const int j = w.at + h * kRows + at;
        if (mine && j < w.r.kv) {
            float* dst = p.weights + static_cast<size_t>(unit) * p.S + j;
            *dst = j < past ? *dst + l : l;
        }
    }
}

// The rows' pieces joined in place of the first, for the columns pass, which reads
// them for every tile of keys (where it joins two of them itself, 1024 tokens take 48
// us instead of 29). Few rows are read once, by the threads that join them.
constexpr int kMaxPieces = 16;
constexpr int kJoinTiles = 6;  // tiles that take as long as the join
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads) lf_join_statistics_kernel(const PromptWeightsParams p, int span) {
    allow_dependent_launch();
    grid_dependency_wait();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kJoinThreads + threadIdx.x;
    const int row = static_cast<int>(i / p.Hq);
    if (row >= p.stat_rows) return;
    const int b = p.by_sequence ? row / p.rows : seq_of_row(p.q_start, p.B, row);
    SeqRange r;
    if (!seq_range(p.q_start, p.kv_len, b, p.T, p.S, true, &r)) return;
    const int t = p.by_sequence ? first_row(p, r) + row % p.rows : row - r.q0;
    if (t < first_row(p, r) || t >= r.n) return;
    const int pieces = row_pieces(p, span, r, t);
    if (pieces == 1) return;
    const size_t piece = static_cast<size_t>(p.stat_rows) * p.Hq;
    float2 v[kMaxPieces];
    float m = -INFINITY, l = 0.f;
#pragma unroll
    for (int k = 0; k < kMaxPieces; ++k) {
        v[k] = k < pieces ? __ldcg(p.stats + k * piece + i) : make_float2(-INFINITY, 0.f);
        m = fmaxf(m, v[k].x);
    }
    if (m == -INFINITY) m = 0.f;
#pragma unroll
    for (int k = 0; k < kMaxPieces; ++k)
        if (k < pieces) l += v[k].y * exp2f(v[k].x - m);
    p.stats[i] = make_float2(m, l);
}

cudaError_t launch_join(const PromptWeightsParams& p, cudaStream_t stream) {
    const char* env = std::getenv("LF_PDL");
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const int64_t n = static_cast<int64_t>(p.stat_rows) * p.Hq;
    cfg.gridDim = dim3(static_cast<unsigned>((n + kJoinThreads - 1) / kJoinThreads));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = (env && std::atoi(env) == 0) ? 0 : 1;
    return cudaLaunchKernelEx(&cfg, lf_join_statistics_kernel, p, 2 * kRows / (p.Hq / p.Hkv));
}

template <int D, int kForm, int kHeld>
cudaError_t launch_pass(const CUtensorMap& tmQ, const CUtensorMap& tmK, const PromptWeightsParams& p,
                        dim3 grid, int cluster, cudaStream_t stream) {
    using L = WeightsSmem<D, kHeld>;
    constexpr auto kernel = lf_prompt_weights_kernel<D, kForm, kHeld>;
    const cudaError_t e = allow_shared<kernel>(L::kAlloc);
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
    cfg.blockDim = dim3(L::kThreads);
    cfg.dynamicSmemBytes = L::kAlloc;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = attrs;
    return cudaLaunchKernelEx(&cfg, kernel, tmQ, tmK, p);
}

template <int D>
cudaError_t launch_d(const CUtensorMap& tmQ, const CUtensorMap& tmK, const PromptWeightsParams& p,
                     cudaStream_t stream) {
    const dim3 rows(p.items * p.Hkv, p.pieces);
    if (p.share == 0) {
        const cudaError_t e = launch_pass<D, kRowsPass, 1>(tmQ, tmK, p, rows, 1, stream);
        return e != cudaSuccess ? e : launch_pass<D, kFewRows, 1>(tmQ, tmK, p, rows, 1, stream);
    }
    cudaError_t e = launch_pass<D, kRowsPass, 2>(tmQ, tmK, p, rows, 1, stream);
    if (e == cudaSuccess && p.pieces > 1) e = launch_join(p, stream);
    if (e != cudaSuccess) return e;
    const int tiles = (p.S + 2 * kRows - 1) / (2 * kRows);
    return launch_pass<D, kColumnsPass, 2>(tmQ, tmK, p, dim3(tiles * p.B * p.Hkv * p.share), p.share, stream);
}

}  // namespace

void plan_prompt_weights(PromptWeightsParams* p, int sms) {
    const int tok = kRows / (p->Hq / p->Hkv);
    // Where no sequence has more rows than a tile holds: one tile per CTA and no
    // tiles of keys (share 0).
    const int64_t most = p->rows > 0 ? std::min(p->rows, p->T) : p->T;
    const bool few = most <= tok;
    const int span = few ? tok : 2 * tok;
    const int64_t each = p->rows > 0 ? (p->rows + span - 1) / span : 0;
    const int64_t packed = p->T / span + p->B;
    p->by_sequence = p->rows > 0 && each * p->B <= packed && static_cast<int64_t>(p->rows) * p->B < p->T;
    p->items = static_cast<int>(p->by_sequence ? each * p->B : packed);
    p->stat_rows = p->by_sequence ? p->rows * p->B : p->T;
    // Pieces of the keys, 16 at most, when the items that hold rows leave SMs idle. Few
    // rows: of so many tiles that full caches are one wave of CTAs, whose start takes
    // as long as several tiles (64 items of 2000 to 8192 keys, us of both passes, 27
    // tiles a piece 33, 22: 29, 16: 33, 11: 36, 8: 41, 32: 36); exactly where there are
    // few items (16 of 8192 keys: 8 tiles, 128 CTAs, 17; 7 tiles, 160 CTAs, 22), while
    // with many the ragged ends of a second wave fit in. More rows: only where a wave
    // holds two pieces of all items, and if they save more than the join's launch.
    // (Items: a sequence's rows share no tile with another's, so those of each sequence
    // take one at least. Counted as if their rows were packed, 8 rows of 8 prompts with
    // groups of 4 took 63 us for 41, one row 87.)
    const int64_t held = p->by_sequence ? each * p->B
                                        : std::max<int64_t>(std::min(p->B, p->T), (p->T + span - 1) / span);
    const int64_t busy = held * p->Hkv;
    const int64_t tiles = (p->S + kRows - 1) / kRows;
    const int64_t least = (tiles + kMaxPieces - 1) / kMaxPieces;
    int64_t per = tiles;
    if (busy * (few ? 5 : 2) <= sms)
        per = std::max(least, (tiles + sms / busy - 1) / (sms / busy));
    else if (few)
        per = std::min(tiles, std::max(least, (tiles * busy + sms - 1) / sms));
    if (!few && tiles - per < kJoinTiles) per = tiles;
    p->piece_tiles = static_cast<int>(per);
    p->pieces = static_cast<int>((tiles + per - 1) / per);
    // CTAs that share two held tiles of keys, a cluster: the first keys are seen by
    // every row, the last by few, so a call takes at least as long as its first tiles
    // unless those are shared; but a start takes as long as several tiles, and larger
    // clusters leave SMs of their group idle. (us, shared by 1, 2, 4, 8; pairs of tiles:
    // 256 (8192 tokens, 8 KV heads) 430, 429, 469, 595; 192: 287, 257, 276, 353; 96: 130,
    // 91, 96, 126; 80: 351, 225, 197, 229; 64: 86, 60, 55, 76; 32: 48, 35, 29, 37; 16:
    // 75, 49, 36, 27 with 63 tiles of rows, 31, 25, 20, 22 with 16.)
    const int64_t pairs = (tiles + 1) / 2 * p->B * p->Hkv;
    const int64_t most_pairs[] = {sms * 4 / 3, sms * 4 / 7, sms / 6};
    const int least_rows[] = {2, 4, 32};  // tiles of a sequence's rows
    const int64_t mean = std::min<int64_t>(most, (p->T + p->B - 1) / p->B);
    p->share = few ? 0 : 1;
    for (int i = 0; i < 3 && p->share > 0; ++i) {
        if (pairs > most_pairs[i] || mean <= static_cast<int64_t>(least_rows[i]) * tok) break;
        p->share *= 2;
    }
}

cudaError_t launch_prompt_weights(int D, const CUtensorMap& tmQ, const CUtensorMap& tmK,
                                  const PromptWeightsParams& p, cudaStream_t stream) {
    if (D == 64) return launch_d<64>(tmQ, tmK, p, stream);
    if (D == 128) return launch_d<128>(tmQ, tmK, p, stream);
    return cudaErrorInvalidValue;
}

}  // namespace lf
