// Attention of packed query rows over in-order caches (sm_103a): the sliding
// window with visible first tokens, and the shared prefix of a decode batch.
//
// One pass over a row's visible keys with the running reference m and sum l
// of its softmax (log2 domain): s = scale * q.k, p = 2^(s - m), O += p v.
// The row's output is O / l; with pieces, (m, l) and the unnormalised O are
// written instead and a later kernel joins them.
//
// Tensor cores do both products. A tile has 128 query rows: 128 / g tokens
// times the g query heads that share a KV head, so a K/V tile in shared
// memory serves the whole group, for single tokens as for prompts. Two
// streams run against each other, each with its own S and O accumulators in
// tensor memory and its own four softmax warps, so one stream's products run
// under the other's exponentials:
//   rows mode  the streams are two query tiles over the same K/V tiles (each
//              K/V tile is read from L2 once per 256 rows);
//   keys mode  (at most 128 rows per sequence on average) the streams are
//              the even and odd K/V tiles of one query tile; at its end the
//              warps of stream 0 read both O and join them.
// A CTA (one per SM: 224 KB of shared memory, all of TMEM) keeps taking work
// items until the grid has none left (cluster launch control hands it the
// index of a CTA that has not started), so one item's loads and products run
// under the epilogue of the one before. Its warps:
//   warps 0-3, 4-7  softmax of stream 0, 1; a thread owns a row: S from
//                   tensor memory, m, l, P (bf16) back over S, at the end O
//   warp 8          one thread issues S = Q K^T (both in shared memory) and
//                   O += P V (P in tensor memory, V as it lies in the cache)
//   warp 9          TMA loads: K and V tiles through a ring
//   warp 10         next work item: cancels a pending CTA, finds the item's
//                   sequence, rows and tiles, hands it to the others; loads Q
//   warp 11         zeroes the rows of V tiles behind a range's last key, and
//                   first the counters of the step that follows a prefix
// A tensor product of 128 x 128 x 128 takes 512 cycles; a pair of tiles needs
// four of them per 128 keys, and the two streams' softmax must fit in between.
// So the chain from S to P is kept short: the exponentials start on the first
// 32 columns of S, with the reference m left by the tiles before. m moves only
// after a tile whose weights add up to more than 2^10, by the logarithm of that
// sum (O and l are rescaled before the next tile's P), which is rare: any
// reference serves, so the tile's maximum is not looked for. Until then the
// weights stay as they are, relative precision and all: bf16 and fp32 hold up
// to 2^127, and a row that outgrows 2^100 within one tile is computed again.
// P is handed over in two halves, the first while the second is still in the
// making.
// P is rounded to bf16 (at most 2^-8 of each weight) because the tensor cores
// take it; l sums the rounded weights, so what the rounding does to a weight
// that dominates the row cancels: 0.0018 of the exact outputs' norm, where the
// unrounded sum gave 0.0023 and rounding exact outputs gives 0.0016. (The sum
// adds bf16 to fp32 in one instruction a weight; widened first, two by two, a
// causal prompt of 16384 tokens took 2% longer, with a maximum beside it 10%.)
// A shared prefix keeps the sum of its unrounded weights as well, which is its
// share of the softmax that the step's slots, outputs and scores see.
//
// What bounds it, and what it measured (32 query and 8 KV heads of 128):
//   a causal prompt of 16384 tokens 1.49 ms, 1470 TFLOP/s, and 1.56 ms a call in
//   a loop of seconds, where the board's power cap takes the clock from 2.07 to
//   1.96 GHz. The softmax warps' arithmetic: without the weights' sum it takes
//   1.32 ms, without any arithmetic 1.33, and 1.27 ms would be the sustained
//   rate of a large plain matrix product (1726 TFLOP/s);
//   eight prompts of 1200 to 2400 tokens, window 1024: 174 us, 947 TFLOP/s
//   of visible pairs; 9 tiles are worked for 8 tiles' worth of pairs, and a
//   tile with a mask costs about 1.5 times one without;
//   128 single tokens, window 1024: 92 us, 5.7 TB/s (the loads, in halves of
//   64 keys, are 4.5% more than the keys seen); 32 single tokens over 16384
//   keys each: 312 us, 6.88 TB/s, the measured copy rate.
//
// Keys a row does not see are removed by select before the exponentials, and
// what a V tile holds behind the range's last key is zeroed in shared memory,
// so it does not matter what lies there. A NaN or infinity in a row that
// others of the tile do see would still reach this row's O as 0 * NaN: a row
// whose result is not finite is computed again by attn_row, key by key. So is
// one left without a reference (m = -infinity) by a tile that holds finite logits.
#include <math.h>
#include <stdlib.h>

#include <algorithm>

#include "../../include/lf_decode.h"
#include "lf_kernels.h"
#include "lf_tcgen05.cuh"

namespace lf {
namespace {

constexpr int kRows = 128;    // query rows of a tile
constexpr int kKeys = 128;    // keys of a tile
constexpr int kSoftmaxThreads = 256;
constexpr int kAttnThreads = kSoftmaxThreads + 128;
// Registers: 384 threads launch with 168 each (64512 in all); the softmax
// warps, which hold a row's 128 scores, then take 224 and the others 56
// (256 * 224 + 128 * 56 = 64512).
constexpr int kSoftmaxRegs = 224;
constexpr int kOtherRegs = 56;
constexpr int kPanel = kRows * 128;  // bytes of 64 columns of a tile
constexpr float kRescale = 1024.f;      // a tile's sum of weights that moves m
constexpr float kMaxGrowth = 1.27e30f;  // 2^100: the largest sum that l and O are trusted with

constexpr int kItemSlots = 3;        // items in flight between the warps
constexpr int kAskTiles = 4;         // K/V tiles of an item left to load when the next is asked for

// What the warps work on.
struct Item {
    int seq, tok0, ntok;  // sequence, first packed row (token) of the tile, its tokens
    int pos0;             // position of the first token (causal)
    int lo, hi;           // keys some row sees: [lo, hi) and below sinks
    int sinks;
    int nsink;            // tiles of the list that hold first keys only
    int joined;           // the tile whose second half holds the first keys, or -1
    int first, count;     // this item's part of the list
    int kvh, split;
    int stop;             // no more work
};

template <int D>
struct AttnSmem {
    static constexpr int kTileBytes = kRows * D * 2;
    static constexpr int kStages = D == 128 ? 5 : 10;
    static constexpr int kRingOff = 2 * kTileBytes;  // after the two Q tiles
    static constexpr int kBarOff = kRingOff + kStages * kTileBytes;
    // barriers: q_full[2], q_empty[2], full[], empty[], s_full[2], p_half[2],
    // p_full[2], o_done[2], o_free[2], item_full[], item_empty[], v_ask,
    // v_clean, drain, next, want, other
    static constexpr int kBars = 4 + 2 * kStages + 10 + 2 * kItemSlots + 6;
    static constexpr int kItemOff = kBarOff + kBars * 8;
    static constexpr int kNextOff = (kItemOff + kItemSlots * static_cast<int>(sizeof(Item)) + 15) / 16 * 16;
    static constexpr int kMiscOff = kNextOff + 16;  // TMEM base; V tile to clean, its rows to keep
    static constexpr int kOtherOff = kMiscOff + 16;  // stream 1's (m, l) [128], keys mode
    static constexpr int kAlloc = kOtherOff + kRows * 8 + 1024;
    static_assert(kAlloc <= 232448, "shared memory of a CTA");
};

// Half h (64 keys) of tile i of the list: its first key and the end of what it
// may hold. Below nsink: the keys from 0 to sinks; then those from lo to hi.
// Few first keys fit into the last tile's second half when the window leaves
// it empty: a tile less.
struct Half {
    int start, end;
};
__device__ __forceinline__ Half tile_half(const Item& it, int i, int h) {
    if (i < it.nsink) return {i * kKeys + h * 64, it.sinks};
    if (h && i == it.joined) return {0, it.sinks};
    return {it.lo + (i - it.nsink) * kKeys + h * 64, it.hi};
}
__device__ __forceinline__ int half_keys(Half x) { return max(0, min(64, x.end - x.start)); }

struct AttnPlan {
    bool rows_mode;
    int tok_shift;  // log2 tokens of a work item
    int nsplit;     // work items over a query tile's K/V tiles
    int items;
};

AttnPlan attn_plan(int T, int N, int Hq, int Hkv, int S, bool causal, int window, int sinks,
                   int sms) {
    const int g = Hq / Hkv;
    int gs = 0;
    while ((1 << gs) < g) ++gs;
    AttnPlan pl;
    // Two query tiles per CTA once sequences have more than one on average.
    // Measured at 4096 keys, keys against rows mode, us: 64 sequences with
    // 128 / 192 / 256 rows each 189 / 299 / 302 against 215 / 232 / 236,
    // 8 sequences 35 / 48 / 48 against 38 / 42 / 45.
    const long long avg = (static_cast<long long>(T) + N - 1) / N;
    pl.rows_mode = avg * g > kRows;
    pl.tok_shift = (pl.rows_mode ? 8 : 7) - gs;
    const int tok = 1 << pl.tok_shift;
    pl.items = (T >> pl.tok_shift) + N;
    // Split the keys when the items (about this many hold rows) leave SMs
    // idle, while all parts still run at once. Measured on single tokens over
    // 16384 keys, us by parts 1 / 2 / 4 / 8 / 16: one sequence (8 items) 140 /
    // 75 / 42 / 25 / 18, eight sequences (64 items, the rule takes 2) 141 /
    // 83 / 93 / 101 / 104, sixteen (128 items, 1) 152 / 168 / 177 / 170 / 179.
    // A part has at least two tiles (one per stream): 1024 keys of one
    // sequence take 10.1 us in 4 parts and no less in more.
    const long long busy = std::min<long long>(pl.items, N * ((avg + tok - 1) / tok)) * Hkv;
    long long keys = S;
    if (causal && window > 0)
        keys = std::min<long long>(S, static_cast<long long>(window) + std::min<long long>(tok, avg) + sinks);
    const long long tiles = (keys + kKeys - 1) / kKeys;
    const long long most = std::max<long long>(1, tiles / 2);
    pl.nsplit = static_cast<int>(
        std::max<long long>(1, std::min<long long>({most, sms / std::max<long long>(busy, 1), 16})));
    return pl;
}

// One warp, one query row, keys visible by select: lane i scores key j0 + i of
// each 32, then the lanes share the values' columns. (m, l) and the lane's
// columns lane * D / 32 ... of O.
template <int D>
__device__ void attn_row(const __nv_bfloat16* q, const __nv_bfloat16* k, const __nv_bfloat16* v,
                         int j_lo, int j_hi, int lo, int hi, int sinks, float scale_log2, float& m,
                         float& l, float (&o)[D / 32]) {
    const int lane = threadIdx.x & 31;
    constexpr int kC = D / 32;
#pragma unroll 1
    for (int j0 = j_lo; j0 < j_hi; j0 += 32) {
        const int j = j0 + lane;
        const bool vis = j < j_hi && j < hi && (j >= lo || j < sinks);
        const unsigned any = __ballot_sync(0xffffffffu, vis);
        if (!any) continue;
        float s = -INFINITY;
        if (vis) {
            const uint4* kr = reinterpret_cast<const uint4*>(k + static_cast<size_t>(j) * D);
            const uint4* qr = reinterpret_cast<const uint4*>(q);
            float a = 0.f;
#pragma unroll 4
            for (int c = 0; c < D / 8; ++c) {
                const uint4 kk = __ldg(kr + c), qq = __ldg(qr + c);
                const __nv_bfloat162* kb = reinterpret_cast<const __nv_bfloat162*>(&kk);
                const __nv_bfloat162* qb = reinterpret_cast<const __nv_bfloat162*>(&qq);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 x = __bfloat1622float2(kb[e]), y = __bfloat1622float2(qb[e]);
                    a += x.x * y.x;
                    a += x.y * y.y;
                }
            }
            s = a * scale_log2;
        }
        float mx = s;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        mx = fmaxf(mx, m);
        const float base = mx == -INFINITY ? 0.f : mx;
        const float keep = m == -INFINITY ? 0.f : exp2f(m - base);
        const float p = vis ? exp2f(s - base) : 0.f;
        float sum = p;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        l = l * keep + sum;
        m = mx;
#pragma unroll
        for (int c = 0; c < kC; ++c) o[c] = keep == 0.f ? 0.f : o[c] * keep;
        // Eight keys' values in flight: 2.9 us for a key of the warp's 32 rows
        // at d = 64 with every warp of the GPU at it (one key's: 13.5 us).
#pragma unroll 1
        for (int i0 = 0; i0 < 32; i0 += 8) {
            if (!(any >> i0 & 0xffu)) continue;
            uint32_t w[8][kC / 2];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
#pragma unroll
                for (int c = 0; c < kC / 2; ++c) w[i][c] = 0u;
                if (any >> (i0 + i) & 1u) {
                    const __nv_bfloat16* vr = v + static_cast<size_t>(j0 + i0 + i) * D + lane * kC;
#pragma unroll
                    for (int c = 0; c < kC / 2; ++c) w[i][c] = __ldg(reinterpret_cast<const uint32_t*>(vr) + c);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float pj = __shfl_sync(0xffffffffu, p, i0 + i);
                // (A key that is not seen: 0 * 0.)
#pragma unroll
                for (int c = 0; c < kC / 2; ++c) {
                    const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i][c]));
                    o[2 * c] += pj * x.x;
                    o[2 * c + 1] += pj * x.y;
                }
            }
        }
    }
}

// An item's row again, over all its tiles; the warp writes the result.
template <int D>
__device__ __noinline__ void redo_row(const AttnParams& p, const Item& it, size_t row,
                                      size_t cache, int lo, int hi) {
    const int lane = threadIdx.x & 31;
    float m = -INFINITY, l = 0.f, o[D / 32];
#pragma unroll
    for (int c = 0; c < D / 32; ++c) o[c] = 0.f;
#pragma unroll 1
    for (int i = 0; i < it.count; ++i) {
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            const Half x = tile_half(it, it.first + i, h);
            attn_row<D>(p.q + row * D, p.k + cache, p.v + cache, x.start, x.start + half_keys(x), lo, hi,
                        it.sinks, p.negate ? -p.scale_log2 : p.scale_log2, m, l, o);
        }
    }
    if (p.pieces == 0) {
        const float il = 1.f / l;
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
            p.out[row * D + lane * (D / 32) + c] = __float2bfloat16_rn(l == 0.f ? 0.f : o[c] * il);
    } else {
        const size_t at = static_cast<size_t>(it.split) * p.T * p.Hq + row;
        if (lane == 0) p.part_ml[at] = make_float2(m, l);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) p.part_o[at * D + lane * (D / 32) + c] = o[c];
    }
}

// TMA load without an L2 hint: K and V tiles are read again by other CTAs.
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y, int z,
                                         uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// Waits for a barrier's phase; false after limit_ns. (Small code: a CTA has
// some twenty waits, and its roles share the instruction cache. A wait may
// last as long as an item, hundreds of microseconds, so its limit is a time:
// the hardware ends a suspension when it likes.)
constexpr uint64_t kDrainNs = 1000000000;
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
    const uint32_t hint = limit_ns < 10000000 ? static_cast<uint32_t>(limit_ns) : 10000000u;
    uint64_t t0 = 0;
    for (;;) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity), "r"(hint)
            : "memory");
        if (ok) return true;
        const uint64_t t = global_timer_ns();
        if (t0 == 0) t0 = t;
        if (t - t0 > limit_ns) return false;
    }
}

// One warp: the sequence and rows of query tile x, and its part of the K/V
// tiles. Sequence b's tiles start at index floor(q_start[b] / tok) + b: enough
// for its rows wherever they start, so no prefix sum over the sequences is
// needed. False where the tile holds no rows (report_sequence tells why).
__device__ bool find_item(const AttnParams& p, const AttnPlan& pl, int2 work, Item* it) {
    const int lane = threadIdx.x & 31;
    // The last tiles (the longest rows of a causal prompt) come first, a
    // tile's KV heads together (they share its rows of Q and out).
    const int x = pl.items - 1 - work.x / p.Hkv;
    int b = 0, len = p.N;
#pragma unroll 1
    while (len > 32) {
        const int step = (len + 31) >> 5;
        const int i = b + lane * step;
        const bool le = lane * step < len && (p.q_start[i] >> pl.tok_shift) + i <= x;
        const unsigned hit = __ballot_sync(0xffffffffu, le);
        const int top = hit ? 31 - __clz(hit) : 0;
        b += top * step;
        len = min(step, len - top * step);
    }
    // The last 32 sequences: their ranges and lengths in one round trip.
    SeqRange r;
    const int i = b + min(lane, len - 1);
    const bool good = seq_range(p.q_start, p.kv_len, i, p.T, p.S, p.causal, &r);
    const unsigned hit =
        __ballot_sync(0xffffffffu, lane < len && (r.q0 >> pl.tok_shift) + i <= x);
    const int top = hit ? 31 - __clz(hit) : 0;
    b += top;
    r.q0 = __shfl_sync(0xffffffffu, r.q0, top);
    r.n = __shfl_sync(0xffffffffu, r.n, top);
    r.kv = __shfl_sync(0xffffffffu, r.kv, top);
    if (!__shfl_sync(0xffffffffu, good, top)) return false;
    const int rel = (x - (r.q0 >> pl.tok_shift) - b) << pl.tok_shift;
    if (rel < 0 || rel >= r.n) return false;
    it->seq = b;
    it->tok0 = r.q0 + rel;
    it->ntok = min(1 << pl.tok_shift, r.n - rel);
    it->pos0 = r.kv - r.n + rel;
    it->hi = p.causal ? it->pos0 + it->ntok : r.kv;
    it->lo = (p.causal && p.window > 0) ? max(0, it->pos0 + 1 - p.window) : 0;
    it->sinks = p.causal ? p.sinks : 0;
    it->nsink = 0;
    it->joined = -1;
    if (it->sinks >= it->lo) it->lo = 0;  // one range
    int tiles = (it->hi - it->lo + kKeys - 1) / kKeys;
    if (it->sinks < it->lo && it->sinks > 0) {
        if (it->sinks <= 64 && it->hi - it->lo - (tiles - 1) * kKeys <= 64)
            it->joined = tiles - 1;
        else
            it->nsink = (it->sinks + kKeys - 1) / kKeys;
        tiles += it->nsink;
    }
    it->first = tiles * work.y / pl.nsplit;
    it->count = tiles * (work.y + 1) / pl.nsplit - it->first;
    it->kvh = work.x % p.Hkv;
    it->split = work.y;
    it->stop = 0;
    return true;
}

// One thread: reports sequence work.x if it does not fit. There are at least as
// many items as sequences, and the search above may miss a sequence whose rows
// end before they start.
__device__ __forceinline__ void report_sequence(const AttnParams& p, int2 work) {
    SeqRange r;
    if (work.y == 0 && work.x < p.N &&
        !seq_range(p.q_start, p.kv_len, work.x, p.T, p.S, p.causal, &r))
        atomicOr(p.dev_err, kErrBadLength);
}

// Stores 64 bytes of each lane's row (v: the lane's own row) at byte `off` of
// the rows. A lane's row lies far from its neighbours', so plain 16-byte
// stores would touch 32 lines each; four lanes exchange their pieces first
// and store 64 bytes of one row together: a quarter of the lines. dst[i] is
// the address of row i of the lane's group of four, or null (not stored).
// With few rows to store in the warp (own: the lane's, or null) the plain
// stores are as quick and spare the exchange.
__device__ __forceinline__ void store_rows(uint4 (&v)[4], char* const (&dst)[4], char* own, bool few,
                                           int off) {
    if (few) {
        if (own) {
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(own + off + i * 16) = v[i];
        }
        return;
    }
    const int q = threadIdx.x & 3;
    auto swap = [&](uint4& a, uint4& b, int bit) {
        // Lanes with the bit set give a and get b of the other, and so on.
        const bool up = (q & bit) != 0;
        const uint4 give = up ? a : b;
        uint4 got;
        got.x = __shfl_xor_sync(0xffffffffu, give.x, bit);
        got.y = __shfl_xor_sync(0xffffffffu, give.y, bit);
        got.z = __shfl_xor_sync(0xffffffffu, give.z, bit);
        got.w = __shfl_xor_sync(0xffffffffu, give.w, bit);
        if (up)
            a = got;
        else
            b = got;
    };
    // 4 x 4 transpose of 16-byte pieces: v[i] becomes piece q of row i.
    swap(v[0], v[1], 1);
    swap(v[2], v[3], 1);
    swap(v[0], v[2], 2);
    swap(v[1], v[3], 2);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (dst[i]) *reinterpret_cast<uint4*>(dst[i] + off + q * 16) = v[i];
}

// Bits [0, n) of a 32-key chunk.
__device__ __forceinline__ uint32_t below(int n) {
    return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}

template <int D, bool kRowsMode, bool kCausal>
__global__ void __launch_bounds__(kAttnThreads, 1)
    lf_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ AttnParams p,
                   const __grid_constant__ AttnPlan pl) {
    using L = AttnSmem<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
    uint64_t* q_empty = q_full + 2;
    uint64_t* full = q_empty + 2;
    uint64_t* empty = full + L::kStages;
    uint64_t* s_full = empty + L::kStages;
    uint64_t* p_half = s_full + 2;
    uint64_t* p_full = p_half + 2;
    uint64_t* o_done = p_full + 2;
    uint64_t* o_free = o_done + 2;
    uint64_t* item_full = o_free + 2;
    uint64_t* item_empty = item_full + kItemSlots;
    uint64_t* v_ask = item_empty + kItemSlots;
    uint64_t* v_clean = v_ask + 1;
    uint64_t* drain = v_clean + 1;
    uint64_t* next = drain + 1;
    uint64_t* want = next + 1;
    uint64_t* other = want + 1;
    float2* const other_ml = reinterpret_cast<float2*>(smem + L::kOtherOff);
    Item* items = reinterpret_cast<Item*>(smem + L::kItemOff);
    volatile uint32_t* misc = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);

    const int tid = threadIdx.x;
    // From one lane, so the compiler knows that a warp's role is uniform.
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int lane = tid & 31;

    // Everything before this wait may run while the previous kernel of the
    // stream ends. (Warp 10 waits first: it reads the lengths.)
    Item it0;
    bool found0 = false;
    if (warp == 10) {
        grid_dependency_wait();
        found0 = find_item(p, pl, make_int2(blockIdx.x, blockIdx.y), &it0);
    } else if (warp == 8) {
        tmem_alloc(reinterpret_cast<uint32_t*>(smem + L::kMiscOff), 512);
    } else if (warp == 9 && lane == 0) {
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&q_full[s], 1);
            mbar_init(&q_empty[s], 1);
            mbar_init(&s_full[s], 1);
            mbar_init(&p_half[s], 4);
            mbar_init(&p_full[s], 4);
            mbar_init(&o_done[s], 1);
            mbar_init(&o_free[s], 4);
        }
        for (int s = 0; s < kItemSlots; ++s) {
            mbar_init(&item_full[s], 1);
            mbar_init(&item_empty[s], 10);  // producer, products, eight softmax warps
        }
        mbar_init(v_ask, 1);
        mbar_init(v_clean, 1);
        mbar_init(drain, 1);
        mbar_init(next, 1);
        mbar_init(want, 1);
        mbar_init(other, 4);
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // The next kernel may start once every CTA is past its wait (not before:
    // the decode step with a prefix reads its own inputs without waiting for
    // this grid, relying on the kernels before it being over, and counts in
    // words that every CTA sets to 0 before that). A CTA counts as having let
    // it start with the first of its threads that says so, so one warp alone
    // does, the one that stores the zeros, after its fence.
    grid_dependency_wait();
    if (warp == 11) {
        if (p.zero != nullptr) {
            // Device-scope stores, fenced: the step's atomics meet them in L2.
            for (int i = lane; i < p.zero_quads; i += 32)
                asm volatile("st.relaxed.gpu.global.v4.u32 [%0], {%1, %1, %1, %1};" ::"l"(p.zero + i), "r"(0u)
                             : "memory");
            __threadfence();
        }
        __syncwarp();  // every lane's zeros
        allow_dependent_launch();
    }
    const uint32_t tmem = __shfl_sync(0xffffffffu, misc[0], 0);
    // Work units of the streams: unit j of an item belongs to stream j & 1 and
    // reads K/V tile j >> 1 (rows mode) or j (keys mode) of the item's part of
    // the list.
    constexpr bool rows = kRowsMode;
    const int gs = __ffs(p.Hq / p.Hkv) - 1;

    // A wait of a whole warp: every lane learns whether all of them saw the
    // barrier complete.
    auto warp_wait = [&](uint64_t* bar, int parity) {
        return __all_sync(0xffffffffu, wait_phase(bar, parity, p.wait_limit_ns)) != 0;
    };
    auto give_up = [&]() { atomicOr(p.dev_err, LF_DEVERR_WAIT_TIMEOUT); };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 9 && lane == 0) {
            // --------------------------------------------------- producer --
            int n = 0;  // ring entries issued
            bool ok = true;
            for (int w = 0;; ++w) {
                const int slot = w % kItemSlots;
                ok = wait_phase(&item_full[slot], (w / kItemSlots) & 1, p.wait_limit_ns);
                if (!ok) break;
                const Item& it = items[slot];
                if (it.stop) break;
                const int units = rows ? 2 * it.count : it.count;
                if (units > 0) {
                    const int unit = it.seq * p.Hkv + it.kvh;
                    // Late enough that another CTA may still be the one to take
                    // the next item, early enough that it is found in time.
                    const int ask = max(0, units - (rows ? 2 * kAskTiles : kAskTiles));
                    // The order in which the products take the tiles: K of
                    // unit t after V of unit t - 2 (in rows mode, two units
                    // share the tile of the even one).
                    const int step = rows ? 2 : 1;
                    for (int t = 0; ok && t < units + 2; t += step) {
                        if (t == ask) mbar_arrive(want);
#pragma unroll 1
                        for (int kv = t >= 2 ? 0 : 1; kv < (t < units ? 2 : 1); ++kv) {
                            const int st = n % L::kStages;
                            ok = wait_phase(&empty[st], ((n / L::kStages) & 1) ^ 1, p.wait_limit_ns);
                            if (!ok) break;
                            const int i = it.first + (kv ? t : t - 2) / step;
                            // The second half only where it holds a key.
                            const int halves = half_keys(tile_half(it, i, 1)) > 0 ? 2 : 1;
                            mbar_arrive_expect_tx(&full[st], halves * (L::kTileBytes / 2));
                            uint8_t* dst = smem + L::kRingOff + st * L::kTileBytes;
#pragma unroll 1
                            for (int h = 0; h < halves; ++h) {
                                const int y = tile_half(it, i, h).start;
                                for (int c = 0; c < D / 64; ++c)
                                    tma_load(dst + c * kPanel + h * (kPanel / 2), kv ? &tmK : &tmV,
                                             c * 64, y, unit, &full[st]);
                            }
                            ++n;
                        }
                    }
                    if (!ok) break;
                } else {
                    mbar_arrive(want);
                }
                mbar_arrive(&item_empty[slot]);
            }
            if (!ok) give_up();
            // No copy may be in flight when the CTA leaves (there is one here
            // only after some wait has run out).
            for (int k = max(0, n - L::kStages); k < n; ++k)
                wait_phase(&full[k % L::kStages], (k / L::kStages) & 1, kDrainNs);
        } else if (warp == 8 && elect_one()) {
            // -------------------------------------------- matrix products --
            // All of it in one thread: with the whole warp in the loop and
            // only the products elected, 8 of them took 700 to 1000 cycles to
            // issue instead of 300 (the queue's depth) to 500 (their rate).
            const uint32_t idesc_s = instr_desc(kRows, kKeys, false) | (p.negate ? kInstrNegateA : 0u);
            constexpr uint32_t idesc_o = instr_desc(kRows, D, true);
            const uint32_t ring = smem_u32(smem + L::kRingOff);
            int n = 0;                  // ring entries taken
            int done = 0;               // items with work
            int cleaned = 0;            // V tiles that had rows to zero
            int pdone[2] = {0, 0};      // units of each stream whose P was taken
            int odone[2] = {0, 0};      // items in which each stream had units
            int kst = 0, vst = 0;       // stages of the current K and V tiles
            bool clean = false;         // the V tile has rows to zero
            bool ok = true;
            auto wait = [&](uint64_t* bar, int parity) {
                return wait_phase(bar, parity, p.wait_limit_ns);
            };
            for (int w = 0;; ++w) {
                const int slot = w % kItemSlots;
                ok = wait(&item_full[slot], (w / kItemSlots) & 1);
                if (!ok) break;
                const Item& it = items[slot];
                if (it.stop) break;
                const int units = rows ? 2 * it.count : it.count;
                if (units > 0) {
                    const int qb = rows ? 0 : done & 1;
                    const uint32_t qs = smem_u32(smem) + qb * L::kTileBytes;
                    ok = wait(&q_full[qb], (rows ? done : done >> 1) & 1);
                    auto take = [&](int* st) {
                        *st = n % L::kStages;
                        const bool got = wait(&full[*st], (n / L::kStages) & 1);
                        ++n;
                        return got;
                    };
                    // O of unit t - 2, then S of unit t: a stream's next S
                    // follows the product that read its P.
#pragma unroll 1
                    for (int t = 0; ok && t < units + 2; ++t) {
                        const int s = t & 1;
                        if (t >= 2) {
                            if (!(rows && s)) {
                                ok = take(&vst);
                                if (!ok) break;
                                const int i = it.first + (rows ? (t - 2) >> 1 : t - 2);
                                const int keep0 = half_keys(tile_half(it, i, 0));
                                const int keep1 = half_keys(tile_half(it, i, 1));
                                clean = keep0 + keep1 < kKeys;
                                if (clean) {
                                    misc[1] = vst;
                                    misc[2] = keep0 | keep1 << 8;
                                    mbar_arrive(v_ask);
                                }
                            }
                            if (t < 4) {
                                // The stream's previous O has been read.
                                ok = odone[s] == 0 || wait(&o_free[s], (odone[s] - 1) & 1);
                                if (!ok) break;
                                ++odone[s];
                            }
                            if (clean && !(rows && s)) {
                                ok = wait(v_clean, cleaned & 1);
                                if (!ok) break;
                                ++cleaned;
                            }
                            const uint64_t vd = smem_desc(ring + vst * L::kTileBytes, kPanel, 1024);
                            const uint32_t od = tmem + 2 * kKeys + s * D;
#pragma unroll 1
                            for (int half = 0; half < 2; ++half) {
                                ok = wait(half ? &p_full[s] : &p_half[s], pdone[s] & 1);
                                if (!ok) break;
                                tc_fence_after();
                                const uint32_t pa = tmem + s * kKeys + half * (kKeys / 4);
                                const uint64_t vh = vd + half * (kKeys / 2 * 128 / 16);
#pragma unroll
                                for (int k = 0; k < kKeys / 32; ++k)
                                    mma_ts(od, pa + k * 8, vh + k * (2048 / 16), idesc_o,
                                           t > 3 || half > 0 || k > 0);
                            }
                            if (!ok) break;
                            ++pdone[s];
                            mma_commit(&o_done[s]);
                            if (!rows || s) mma_commit(&empty[vst]);
                        }
                        if (t < units) {
                            if (!(rows && s)) {
                                ok = take(&kst);
                                if (!ok) break;
                            }
                            tc_fence_after();
                            const uint64_t qd = smem_desc(qs + (rows && s ? L::kTileBytes : 0), 16, 1024);
                            const uint64_t kd = smem_desc(ring + kst * L::kTileBytes, 16, 1024);
#pragma unroll
                            for (int k = 0; k < D / 16; ++k) {
                                const uint64_t off = ((k >> 2) * kPanel + (k & 3) * 32) / 16;
                                mma_ss(tmem + s * kKeys, qd + off, kd + off, idesc_s, k > 0);
                            }
                            mma_commit(&s_full[s]);
                            if (!rows || s) mma_commit(&empty[kst]);
                            if (t == units - 1) mma_commit(&q_empty[qb]);
                        }
                    }
                    if (!ok) break;
                    ++done;
                }
                mbar_arrive(&item_empty[slot]);
            }
            if (!ok) give_up();
            // No product may be in flight when tensor memory is freed.
            mma_commit(drain);
            wait_phase(drain, 0, kDrainNs);
            misc[1] = L::kStages;  // no more V tiles
            mbar_arrive(v_ask);
        } else if (warp == 11) {
            // ------------------------------------------------- V tile rows --
            // On demand of the products' thread, which has seen the tile land.
            // Requests may be far apart: this wait alone has a longer limit.
            for (int n = 0;; ++n) {
                if (!__all_sync(0xffffffffu, wait_phase(v_ask, n & 1, 100 * p.wait_limit_ns))) break;
                const int st = static_cast<int>(misc[1]);
                if (st >= L::kStages) break;
                uint8_t* vt = smem + L::kRingOff + st * L::kTileBytes;
                const uint32_t keep = misc[2];
#pragma unroll 1
                for (int c = 0; c < 2 * (D / 64); ++c)  // panel c >> 1, half c & 1
#pragma unroll 1
                    for (int e = ((keep >> (c & 1) * 8) & 255) * 8 + lane; e < 64 * 8; e += 32)
                        *reinterpret_cast<uint4*>(vt + c * (kPanel / 2) + e * 16) =
                            make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(v_clean);
            }
        } else if (warp == 10) {
            // ------------------------------------------------- next items --
            int w = 0;     // items handed out
            int done = 0;  // items with work
            bool ok = true;
            Item it = it0;
            it.stop = found0 ? 0 : -1;  // -1: no rows there, ask again
            int2 work = make_int2(blockIdx.x, blockIdx.y);
            for (int round = 0;; ++round) {
                if (it.stop >= 0) {
                    const int slot = w % kItemSlots;
                    ok = warp_wait(&item_empty[slot], ((w / kItemSlots) & 1) ^ 1);
                    if (!ok) break;
                    if (lane == 0) {
                        items[slot] = it;
                        mbar_arrive(&item_full[slot]);
                    }
                    __syncwarp();
                    if (it.stop) break;
                    if (it.count > 0) {
                        // Q: both tiles in rows mode, alternating buffers in keys mode.
                        const int qb = rows ? 0 : done & 1;
                        const int use = rows ? done : done >> 1;
                        ok = warp_wait(&q_empty[qb], (use & 1) ^ 1);
                        if (!ok) break;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&q_full[qb], (rows ? 2 : 1) * L::kTileBytes);
                            for (int s = 0; s < (rows ? 2 : 1); ++s)
                                for (int c = 0; c < D / 64; ++c)
                                    tma_load(smem + (s + qb) * L::kTileBytes + c * kPanel, &tmQ, c * 64,
                                             it.kvh << gs, it.tok0 + s * (kRows >> gs), &q_full[qb]);
                        }
                        __syncwarp();
                        ++done;
                    }
                    ok = warp_wait(want, w & 1);
                    if (!ok) break;
                    ++w;
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(next, 16);
                    cancel_next_cta(smem + L::kNextOff, next);
                    report_sequence(p, work);  // under the answer's round trip
                }
                ok = warp_wait(next, round & 1);
                if (!ok) break;
                work = cancelled_cta(smem + L::kNextOff);
                fence_proxy_async_smem();  // the answer is read before the next one lands
                __syncwarp();
                if (work.x < 0)
                    it.stop = 1;
                else
                    it.stop = find_item(p, pl, work, &it) ? 0 : -1;
            }
            if (!ok && lane == 0) give_up();
            // Neither Q's copies nor, after a wait that ran out, an answer.
            // (The last use of each buffer.)
            for (int k = max(0, done - (rows ? 1 : 2)); k < done; ++k)
                wait_phase(&q_full[rows ? 0 : k & 1], (rows ? k : k >> 1) & 1, kDrainNs);
            if (!ok) {
                wait_phase(next, 0, 1000000);
                wait_phase(next, 1, 1000000);
            }
        }
    } else {
        // --------------------------------------------------------- softmax --
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int s = warp >> 2;
        const int r = tid & (kRows - 1);
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // the warp's lanes
        const uint32_t ts = tmem + lanes + s * kKeys;
        const uint32_t to = tmem + lanes + 2 * kKeys + s * D;
        const int tt = (rows && s ? kRows >> gs : 0) + (r >> gs);  // token of the item
        const float c = p.scale_log2;
        const uint64_t c2 = pack_f32x2(c, c);
        int n = 0;       // units of this stream so far
        int others = 0;  // results of stream 1 joined
        bool ok = true;
        for (int w = 0;; ++w) {
            const int slot = w % kItemSlots;
            ok = warp_wait(&item_full[slot], (w / kItemSlots) & 1);
            if (!ok) break;
            const Item& it = items[slot];
            if (it.stop) break;
            const int units = rows ? 2 * it.count : it.count;
            const bool valid = tt < it.ntok;
            const bool any_valid = __any_sync(0xffffffffu, valid);
            const int row_hi = kCausal ? it.pos0 + tt + 1 : it.hi;
            const int row_lo = (kCausal && p.window > 0) ? max(0, row_hi - p.window) : 0;
            // Keys every row of the warp sees: [all_lo, all_hi), and below sinks.
            const int all_hi = __shfl_sync(0xffffffffu, row_hi, 0);
            const int all_lo = __shfl_sync(0xffffffffu, row_lo, 31);
            float m = -INFINITY, l = 0.f;  // l: of the rounded weights
            float l_all = 0.f;             // of the weights themselves (prefix)
            float grown = 0.f;             // of the last tile's weights
            for (int j = s; j < units; j += 2, ++n) {
                if (!warp_wait(&s_full[s], n & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (any_valid) {
                    const int i = it.first + (rows ? j >> 1 : j);
                    const Half h0 = tile_half(it, i, 0), h1 = tile_half(it, i, 1);
                    const bool partial =
                        i == it.joined || !(h0.start + kKeys <= min(all_hi, h0.end) &&
                                            (h0.start >= all_lo || h0.start + kKeys <= it.sinks));
                    uint32_t x[2][32];
                    // Keys the row does not see: weight 0. Most 32-key chunks
                    // of a partial tile hold none.
                    auto hide = [&](int k, uint32_t* v) {
                        const Half x = k < 64 ? h0 : h1;
                        const int j0 = x.start + (k & 32);
                        const uint32_t vis = below(min(row_hi, x.end) - j0) &
                                             (~below(row_lo - j0) | below(it.sinks - j0));
                        if (__any_sync(0xffffffffu, vis != 0xffffffffu)) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                v[e] = (vis & (1u << e)) ? v[e] : 0xff800000u;
                        }
                    };
                    auto largest = [&](const uint32_t* v) {
                        float t[2] = {-INFINITY, -INFINITY};
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            t[(e >> 1) & 1] = fmaxf(t[(e >> 1) & 1], fmaxf(__uint_as_float(v[e]),
                                                                          __uint_as_float(v[e + 1])));
                        return fmaxf(t[0], t[1]);
                    };
                    // The reference moves where the last tile outgrew it.
                    if (__any_sync(0xffffffffu, grown > kRescale)) {
                        const float to_m = grown > kRescale ? m + __log2f(grown) : m;
                        const float f = grown > kRescale ? ex2_approx(m - to_m) : 1.f;
                        m = to_m;
                        // Beyond 2^100 in one tile: the row is computed again.
                        l = grown > kMaxGrowth ? NAN : l * f;
                        if (!kCausal) l_all *= f;
                        // The product that S waited for came after the one
                        // that last wrote O.
#pragma unroll 1
                        for (int k = 0; k < D; k += 16) {
                            uint32_t o[16];
                            tmem_ld16(to + k, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st16(to + k, o);
                        }
                        tmem_wait_st();
                    }
                    uint64_t b2 = 0;
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
                    uint64_t all[2] = {0ull, 0ull};
                    // Weights of 32 keys: exponentials, P, its sum.
                    auto weigh = [&](int k, const uint32_t* v) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float a, b;
                            unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(v[e]),
                                                              __uint_as_float(v[e + 1])), c2, b2), a, b);
                            a = ex2_approx(a);
                            b = ex2_approx(b);
                            if (!kCausal) all[(e >> 1) & 1] = add_f32x2(all[(e >> 1) & 1], pack_f32x2(a, b));
                            pk[e >> 1] = pack_bf16x2(a, b);
                            add_bf16x2(sum[e & 2], sum[(e & 2) + 1], pk[e >> 1]);
                        }
                        tmem_st16(ts + (k >> 1), pk);
                    };
                    auto hand_over = [&]() {
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&p_half[s]);
                    };
                    auto refer = [&]() {
                        const float base = m == -INFINITY ? 0.f : -m;
                        b2 = pack_f32x2(base, base);
                    };
                    if (!partial) {
                        tmem_ld32(ts, x[0]);
                        if (__any_sync(0xffffffffu, m == -INFINITY)) {
                            // No reference yet: the largest of the first 32.
                            tmem_wait_ld();
                            const float t = largest(x[0]) * c;
                            if (m == -INFINITY) {
                                m = t;
                                // -infinity all: no reference for the others.
                                if (t == -INFINITY) l = NAN;
                            }
                        }
                        refer();
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            tmem_wait_ld();
                            if (q < 3) tmem_ld32(ts + 32 * (q + 1), x[(q + 1) & 1]);
                            weigh(32 * q, x[q & 1]);
                            if (q == 1) hand_over();
                        }
                    } else {
                        uint32_t v[4][32];
#pragma unroll
                        for (int q = 0; q < 4; ++q) tmem_ld32(ts + 32 * q, v[q]);
                        tmem_wait_ld();
#pragma unroll
                        for (int q = 0; q < 4; ++q) hide(32 * q, v[q]);
                        if (__any_sync(0xffffffffu, m == -INFINITY)) {
                            const float t = fmaxf(fmaxf(largest(v[0]), largest(v[1])),
                                                  fmaxf(largest(v[2]), largest(v[3]))) * c;
                            if (m == -INFINITY) m = t;
                        }
                        refer();
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            weigh(32 * q, v[q]);
                            if (q == 1) hand_over();
                        }
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_full[s]);
                    grown = (sum[0] + sum[2]) + (sum[1] + sum[3]);
                    l += grown;
                    if (!kCausal) {
                        float a, b;
                        unpack_f32x2(add_f32x2(all[0], all[1]), a, b);
                        l_all += a + b;
                    }
                } else {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&p_half[s]);
                        mbar_arrive(&p_full[s]);
                    }
                }
            }
            if (!ok) break;
            // A prefix's share of the softmax is that of its unrounded weights: with
            // the base moved by the sums' quotient, l_all 2^m = l 2^m', O stays O / l.
            if (!kCausal && l > 0.f) m += __log2f(l_all / l);
            const bool worked = units > s;  // the stream had a unit
            if (worked) {
                ok = warp_wait(&o_done[s], (n - 1) & 1);
                if (!ok) break;
                tc_fence_after();
            }
            if (!rows && s) {
                // Stream 0 joins this stream's result with its own. (The next
                // one waits for O to be read, and this with it.)
                if (worked) {
                    other_ml[r] = make_float2(m, l);
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) {
                    if (worked) mbar_arrive(other);
                    mbar_arrive(&item_empty[slot]);
                }
                continue;
            }
            const bool two = !rows && units > 1;
            // 0 unless a value is not finite or grew out of hand.
            float bad = l < 1e30f ? 0.f : NAN;
            float f0 = 1.f, f1 = 0.f;  // weights of the two O
            if (two) {
                ok = warp_wait(other, others++ & 1);
                if (!ok) break;
                tc_fence_after();
                const float2 v = other_ml[r];
                bad = v.y < 1e30f ? bad : NAN;
                const float top = fmaxf(l == 0.f ? -INFINITY : m, v.y == 0.f ? -INFINITY : v.x);
                f0 = l == 0.f ? 0.f : exp2f(m - top);
                f1 = v.y == 0.f ? 0.f : exp2f(v.x - top);
                l = l * f0 + v.y * f1;
                m = top;
            }
            const size_t row = static_cast<size_t>(it.tok0 + tt) * p.Hq + (it.kvh << gs) +
                               (r & ((1 << gs) - 1));
            const size_t at = static_cast<size_t>(it.split) * p.T * p.Hq + row;
            const bool some = valid && l != 0.f;
            if (any_valid) {
                if (p.pieces == 0) {
                    const float il = some ? 1.f / l : 0.f;
                    f0 *= il;
                    f1 *= il;
                }
                const bool use0 = some && f0 != 0.f, use1 = some && f1 != 0.f;
                // Rows to store, of the lane's group of four.
                char* const mine = (p.pieces == 0 ? reinterpret_cast<char*>(p.out) + row * D * 2
                                                  : reinterpret_cast<char*>(p.part_o) + at * D * 4);
                const uint64_t addr =
                    (p.pieces == 0 ? valid : some) ? reinterpret_cast<uint64_t>(mine) : 0ull;
                char* const own = reinterpret_cast<char*>(addr);
                const bool few = __popc(__ballot_sync(0xffffffffu, addr != 0)) <= 8;
                char* dst[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    dst[i] = reinterpret_cast<char*>(__shfl_sync(0xffffffffu, addr, i, 4));
#pragma unroll 1
                for (int k = 0; k < D; k += 32) {
                    uint32_t o[32];
                    if (worked) {
                        tmem_ld32(to + k, o);
                        tmem_wait_ld();
                    }
                    // (An O without a key has weight 0 and is not looked at.)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = use0 ? __float_as_uint(__uint_as_float(o[e]) * f0) : 0u;
                    if (two) {
                        uint32_t o1[32];
                        tmem_ld32(to + D + k, o1);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (use1)
                                o[e] = __float_as_uint(fmaf(__uint_as_float(o1[e]), f1, __uint_as_float(o[e])));
                    }
                    float odd[4] = {bad, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int e = 0; e < 32; ++e) odd[e & 3] = fmaf(__uint_as_float(o[e]), 0.f, odd[e & 3]);
                    bad = (odd[0] + odd[1]) + (odd[2] + odd[3]);
                    uint4 v[4];
                    if (p.pieces == 0) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t* w = o + 8 * i;
                            v[i].x = pack_bf16x2(__uint_as_float(w[0]), __uint_as_float(w[1]));
                            v[i].y = pack_bf16x2(__uint_as_float(w[2]), __uint_as_float(w[3]));
                            v[i].z = pack_bf16x2(__uint_as_float(w[4]), __uint_as_float(w[5]));
                            v[i].w = pack_bf16x2(__uint_as_float(w[6]), __uint_as_float(w[7]));
                        }
                        store_rows(v, dst, own, few, k * 2);
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                v[i] = make_uint4(o[16 * h + 4 * i], o[16 * h + 4 * i + 1],
                                                  o[16 * h + 4 * i + 2], o[16 * h + 4 * i + 3]);
                            store_rows(v, dst, own, few, k * 4 + h * 64);
                        }
                    }
                }
                if (valid && p.pieces > 0) p.part_ml[at] = make_float2(m, l);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (worked) mbar_arrive(&o_free[s]);
                if (two) mbar_arrive(&o_free[1]);
            }
            for (unsigned redo = __ballot_sync(0xffffffffu, some && !(bad == 0.f)); redo;
                 redo &= redo - 1) {
                const int from = __ffs(redo) - 1;
                const size_t rr =
                    static_cast<size_t>(__shfl_sync(0xffffffffu, static_cast<unsigned>(row >> 32), from))
                        << 32 |
                    __shfl_sync(0xffffffffu, static_cast<unsigned>(row), from);
                redo_row<D>(p, it, rr, (static_cast<size_t>(it.seq) * p.Hkv + it.kvh) * p.S * D,
                            __shfl_sync(0xffffffffu, row_lo, from),
                            __shfl_sync(0xffffffffu, row_hi, from));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_empty[slot]);
        }
        if (!ok && lane == 0) give_up();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

// Joins the pieces of the key axis: one warp per query row.
constexpr int kMergeWarps = 4;
constexpr int kMaxPieces = 32;

template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) lf_attn_merge_kernel(const AttnParams p) {
    const int lane = threadIdx.x & 31;
    const size_t rows = static_cast<size_t>(p.T) * p.Hq;
    const size_t at = static_cast<size_t>(blockIdx.x) * kMergeWarps + (threadIdx.x >> 5);
    allow_dependent_launch();
    const size_t row = at < rows ? at : rows - 1;
    const int t = static_cast<int>(row / p.Hq);
    // Every thread waits, so this grid ends after the attention grid.
    grid_dependency_wait();
    // A batch of single tokens has its row t in sequence t.
    int n = min(t, p.N - 1);
    if (!(p.q_start[n] <= t && t < p.q_start[n + 1])) n = seq_of_row(p.q_start, p.N, t);
    SeqRange r;
    const bool mine = seq_range(p.q_start, p.kv_len, n, p.T, p.S, p.causal, &r) && t >= r.q0 && t < r.q0 + r.n && at < rows;
    if (!mine) return;
    const float2 ml = lane < p.pieces ? __ldcg(&p.part_ml[lane * rows + row])
                                      : make_float2(-INFINITY, 0.f);
    float m = ml.y != 0.f ? ml.x : -INFINITY;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    float w = ml.y != 0.f ? exp2f(ml.x - m) : 0.f;
    float l = ml.y * w;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    w = l == 0.f ? 0.f : w / l;
    // The pieces' outputs, eight loads in flight; one without a visible key
    // was not written and is not read.
    constexpr int kC = D / 32;
    constexpr int kBatch = 8;
    float o[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) o[c] = 0.f;
    const float* po = p.part_o + row * D + lane * kC;
    for (int i0 = 0; i0 < p.pieces; i0 += kBatch) {
        float wi[kBatch], v[kBatch][kC];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            wi[i] = __shfl_sync(0xffffffffu, w, (i0 + i) & 31);
            if (i0 + i >= p.pieces) wi[i] = 0.f;
#pragma unroll
            for (int c = 0; c < kC; c += 2) {
                float2 x = make_float2(0.f, 0.f);
                if (wi[i] != 0.f)
                    x = __ldcg(reinterpret_cast<const float2*>(po + (i0 + i) * rows * D + c));
                v[i][c] = x.x;
                v[i][c + 1] = x.y;
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
#pragma unroll
            for (int c = 0; c < kC; ++c) o[c] += wi[i] * v[i][c];
    }
#pragma unroll
    for (int c = 0; c < kC; c += 2)
        *reinterpret_cast<uint32_t*>(p.out + row * D + lane * kC + c) = pack_bf16x2(o[c], o[c + 1]);
}

template <int D, bool kRowsMode, bool kCausal>
cudaError_t launch_attention_t(const CUtensorMap& tmQ, const CUtensorMap& tmK,
                               const CUtensorMap& tmV, const AttnParams& p, const AttnPlan& pl,
                               cudaStream_t stream) {
    using L = AttnSmem<D>;
    auto kernel = lf_attn_kernel<D, kRowsMode, kCausal>;
    static int configured_for = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (configured_for != dev) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
        if (e != cudaSuccess) return e;
        configured_for = dev;
    }
    const dim3 grid(static_cast<unsigned>(pl.items) * p.Hkv, static_cast<unsigned>(pl.nsplit));
    const char* env = std::getenv("LF_PDL");
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kAttnThreads);
    cfg.dynamicSmemBytes = L::kAlloc;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = (env && std::atoi(env) == 0) ? 0 : 1;
    e = cudaLaunchKernelEx(&cfg, kernel, tmQ, tmK, tmV, p, pl);
    if (e != cudaSuccess || p.pieces == 0 || !p.out) return e != cudaSuccess ? e : cudaGetLastError();
    const size_t rows = static_cast<size_t>(p.T) * p.Hq;
    cfg.gridDim = dim3(static_cast<unsigned>((rows + kMergeWarps - 1) / kMergeWarps));
    cfg.blockDim = dim3(kMergeWarps * 32);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, lf_attn_merge_kernel<D>, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

int attention_pieces(int T, int N, int Hq, int Hkv, int S, bool causal, int window, int sinks,
                     int sms) {
    const AttnPlan pl = attn_plan(T, N, Hq, Hkv, S, causal, window, sinks, sms);
    return causal && pl.nsplit == 1 ? 0 : pl.nsplit;
}

cudaError_t launch_attention(int D, const CUtensorMap& tmQ, const CUtensorMap& tmK,
                             const CUtensorMap& tmV, const AttnParams& p, int sms,
                             cudaStream_t stream) {
    const AttnPlan pl = attn_plan(p.T, p.N, p.Hq, p.Hkv, p.S, p.causal, p.window, p.sinks, sms);
    if (p.pieces > kMaxPieces) return cudaErrorInvalidConfiguration;
#define LF_ATTN_CASE(DD, RR, CC) \
    if (D == DD && pl.rows_mode == RR && p.causal == CC) \
        return launch_attention_t<DD, RR, CC>(tmQ, tmK, tmV, p, pl, stream);
    LF_ATTN_CASE(64, true, true) LF_ATTN_CASE(64, false, true)
    LF_ATTN_CASE(64, true, false) LF_ATTN_CASE(64, false, false)
    LF_ATTN_CASE(128, true, true) LF_ATTN_CASE(128, false, true)
    LF_ATTN_CASE(128, true, false) LF_ATTN_CASE(128, false, false)
#undef LF_ATTN_CASE
    return cudaErrorInvalidValue;
}

}  // namespace lf
