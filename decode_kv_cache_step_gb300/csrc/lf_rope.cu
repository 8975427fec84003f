// Norm and position rotation of query and key heads in one pass (sm_103a).
//
// A head x of D values with weight w becomes y = x * w / sqrt(mean(x^2) + eps)
// (no norm without weights); each of the rot / 2 rotated pairs (y_i, y_j)
// turns by the angle a = position * inv_freq_i:
//   (y_i cos a - y_j sin a, y_j cos a + y_i sin a),
// with j = i + rot / 2, or pairs (2i, 2i + 1) when interleaved. Value heads
// are copied. All in fp32, rounded to bf16 once.
//
// Memory bound: each value is read and written once. D / 8 lanes hold a head,
// each lane two chunks of 4 values (8 bytes) that rotate among themselves: the
// halves' chunks at the same offset, or the neighbours of an interleaved
// pair, so only the norm's sum crosses lanes. A CTA takes all heads of one to
// four tokens (one warp a token where there are many), and a lane keeps its 4
// angles and its weights for all of them. The angles are formed once per CTA in
// shared memory while the first heads' loads are in flight, with integers:
// any int32 position times a frequency, less its whole turns, needs some 60
// bits (fp64 would take 1000 cycles of an SM's fp64 unit per CTA).
//
// Measured (32 query, 8 KV heads of 128): 20.3K prompt tokens into their
// caches 81 us, 6.2 TB/s read and written, 91% of the measured copy rate (2 us
// more with loads marked evict-first); one token 2.9 us, 128 tokens 3.5 us, which is
// the latency of a launch and three dependent round trips.
//
// With several position axes (kAxes) pair i turns by its axis' position: one more
// word to load per token and axis, requested before the search for the token's
// sequence. The same 20.3K tokens on three axes 82.4 us (85.4 with the load
// behind the search and a byte per pair read from the parameters by each lane),
// one token 2.9.
#include <stdlib.h>

#include <algorithm>

#include "lf_kernels.h"
#include "lf_tcgen05.cuh"

namespace lf {
namespace {

constexpr int kRopeThreads = 256;  // of a CTA when the call is small
constexpr int kRopeWarps = 32;     // resident per SM, at 64 registers a thread
constexpr int kBatch = 4;          // heads whose loads a lane has in flight
constexpr int kMaxAgeParts = 16;   // CTAs that write one head's ages
constexpr int kAgesPerPart = 2048;
// Mean squares taken as they are: none of a head's squares overflows, and what
// the smallest lose below fp32's normal range does not count.
constexpr float kMeanMax = 0x1p110f;
constexpr float kMeanMin = 0x1p-100f;

// Tokens a CTA may take.
__host__ __device__ constexpr int max_tokens(int threads) { return threads >= 128 ? 4 : 1; }

struct TokenAt {
    int b, slot, pos;  // b < 0: no output for this token
};

// The sequence of packed row t by the whole warp: the last b with
// q_start[b] <= t, 32 probes at a time.
__device__ __forceinline__ int warp_seq_of_row(const int32_t* q_start, int B, int t) {
    const int lane = threadIdx.x & 31;
    int b = 0, len = B;
    while (len > 1) {
        const int step = (len + 31) >> 5;
        const bool le = lane * step < len && q_start[b + lane * step] <= t;
        const unsigned hit = __ballot_sync(0xffffffffu, le);
        const int top = hit ? 31 - __clz(hit) : 0;
        b += top * step;
        len = min(step, len - top * step);
    }
    return b;
}

// Two bf16 values as packed fp32 (exact).
__device__ __forceinline__ uint64_t widen2(uint32_t v) {
    return pack_f32x2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

__device__ __forceinline__ uint32_t narrow2(uint64_t v) {
    float x, y;
    unpack_f32x2(v, x, y);
    return pack_bf16x2(x, y);
}

__device__ __forceinline__ uint64_t swap2(uint64_t v) {
    float x, y;
    unpack_f32x2(v, x, y);
    return pack_f32x2(y, x);
}

// n * f / (2 pi) less its whole turns, to 2^-25 of a turn (the result's last
// bit) for any n and any f below 2^24 (to 2^-23 below 2^32), after Payne and Hanek's reduction: f = M 2^E
// with an integer M of 24 bits, so the fraction of f / (2 pi) is a window of 64
// bits of M times the bits of 1 / (2 pi). n is whole: the product with the
// window, modulo 2^64, is the fraction of a turn.
__device__ __forceinline__ float turns(int n, float f) {
    // 1 / (2 pi), 96 bits behind the point.
    constexpr uint32_t k0 = 0x28be60dbu, k1 = 0x9391054au, k2 = 0x7f09d5f4u;
    const uint32_t bits = __float_as_uint(f);
    const int ex = bits >> 23 & 255;
    if (ex == 255) return NAN;
    const uint64_t m = (bits & 0x7fffffu) | (ex ? 0x800000u : 0u);
    const uint64_t p1 = m * k1 + (m * k2 >> 32);
    const uint64_t p0 = m * k0 + (p1 >> 32);
    const uint64_t lo = p0 << 32 | static_cast<uint32_t>(p1);
    const uint64_t hi = p0 >> 32;
    const int s = 150 - max(ex, 1);
    uint64_t r;
    if (s <= 0)
        r = s > -64 ? lo << -s : 0;
    else if (s < 64)
        r = lo >> s | hi << (64 - s);
    else
        r = s < 128 ? hi >> (s - 64) : 0;
    const uint64_t t = static_cast<uint64_t>(static_cast<int64_t>(n)) * r;
    const float a = static_cast<float>(static_cast<int32_t>(t >> 32)) * 0x1p-32f;
    return bits >> 31 ? -a : a;
}

template <int D, bool kInterleaved, int kThreads, bool kAxes>
__global__ void __launch_bounds__(kThreads, kRopeWarps * 32 / kThreads)
    lf_rope_kernel(const RopeParams p, int tok_per_cta, int tok_ctas, int age_parts) {
    constexpr int kLanes = D / 8;                    // lanes of one head
    constexpr int kGroups = kThreads / kLanes;       // heads a CTA holds at a time
    constexpr int kMaxTokens = max_tokens(kThreads);
    __shared__ TokenAt at[kMaxTokens];
    __shared__ float2 cs[kMaxTokens][D / 2];
    __shared__ int axis_pos[kMaxTokens][kMaxAxes];
    const int tid = threadIdx.x;
    allow_dependent_launch();
    grid_dependency_wait();
    const bool append = p.q_start != nullptr;
    if (static_cast<int>(blockIdx.x) >= tok_ctas) {
        // Ages of the prompt's tokens, age_parts CTAs per (sequence, KV head).
        const int u = (blockIdx.x - tok_ctas) / age_parts;
        const int part = (blockIdx.x - tok_ctas) % age_parts;
        const int b = u / p.Hkv;
        SeqRange r;
        if (!seq_range(p.q_start, p.kv_len, b, p.T, p.S, true, &r)) {
            if (tid == 0) atomicOr(p.dev_err, kErrBadLength);
            return;
        }
        int32_t* m = p.mask + static_cast<size_t>(u) * p.S;
        const int first = part * kThreads + tid;
        const int step = age_parts * kThreads;
        const int fours = reinterpret_cast<uintptr_t>(m) % 16 ? 0 : r.kv / 4;
        for (int i = first; i < fours; i += step) {
            const int a = r.kv - 1 - 4 * i;
            reinterpret_cast<int4*>(m)[i] = make_int4(a, a - 1, a - 2, a - 3);
        }
        for (int j = 4 * fours + first; j < r.kv; j += step) m[j] = r.kv - 1 - j;
        return;
    }
    const int heads = p.Hq + 2 * p.Hkv;
    const int half = p.rot / 2;
    const int tok0 = blockIdx.x * tok_per_cta;
    const int ntok = min(tok_per_cta, p.T - tok0);
    // The lane's token, its first head and the step to its next one.
    const int per_tok = kGroups / tok_per_cta;
    const int group = tid / kLanes;
    const int k = group / per_tok;
    const bool active = k < ntok;
    const int h0 = group - k * per_tok;
    // The lane's chunks: rotated against each other below `half` (in steps of
    // 4 values), the rest in order.
    const int lane = tid % kLanes;
    const bool turned = 8 * lane < p.rot;
    int ea, eb;
    if (kInterleaved || !turned) {
        ea = 8 * lane;
        eb = ea + 4;
    } else {
        ea = 4 * lane;
        eb = ea + half;
    }
    const __nv_bfloat16* row = p.qkv + static_cast<size_t>(tok0 + (active ? k : 0)) * p.stride;
    uint2 ra[kBatch], rb[kBatch];
    auto load = [&](int h) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int hh = h + i * per_tok;
            if (active && hh < heads) {
                const __nv_bfloat16* src = row + static_cast<size_t>(hh) * D;
                ra[i] = __ldcg(reinterpret_cast<const uint2*>(src + ea));
                rb[i] = __ldcg(reinterpret_cast<const uint2*>(src + eb));
            }
        }
    };
    load(h0);
    // Weights of query and key heads (kept packed).
    uint2 wq[2] = {}, wk[2] = {};
    if (p.q_weight) {
        wq[0] = __ldg(reinterpret_cast<const uint2*>(p.q_weight + ea));
        wq[1] = __ldg(reinterpret_cast<const uint2*>(p.q_weight + eb));
        wk[0] = __ldg(reinterpret_cast<const uint2*>(p.k_weight + ea));
        wk[1] = __ldg(reinterpret_cast<const uint2*>(p.k_weight + eb));
    }
    if (tid < ntok * 32) {
        // One warp per token.
        const int i = tid >> 5;
        const int t = tok0 + i;
        TokenAt a{0, 0, 0};
        // (Before the search, so that their round trips overlap.)
        const bool axis = kAxes && (tid & 31) < p.axes;
        const int axis_at = axis ? p.positions[static_cast<size_t>(tid & 31) * p.T + t] : 0;
        if (append) {
            a.b = warp_seq_of_row(p.q_start, p.B, t);
            SeqRange r;
            if (seq_range(p.q_start, p.kv_len, a.b, p.T, p.S, true, &r) && t >= r.q0 &&
                t < r.q0 + r.n) {
                a.slot = r.kv - r.n + (t - r.q0);
                a.pos = a.slot + (p.pos_offset ? p.pos_offset[a.b] : 0);
            } else {
                a.b = -1;
            }
        } else if (!kAxes) {
            a.pos = p.positions[t];
        }
        if (axis) axis_pos[i][tid & 31] = axis_at;
        if ((tid & 31) == 0) at[i] = a;
    }
    __syncthreads();
    for (int i = tid; i < ntok * half; i += kThreads) {
        const int kk = i / half;
        const int pair = i - kk * half;
        int pos = at[kk].pos;
        if constexpr (kAxes) {
            // (Selected, not indexed: lanes that read different words of the
            // parameters do so one after another.)
            const uint32_t lo = pair & 16 ? p.pair_axis[1] : p.pair_axis[0];
            const uint32_t hi = pair & 16 ? p.pair_axis[3] : p.pair_axis[2];
            pos = axis_pos[kk][((pair & 32 ? hi : lo) >> (2 * (pair & 15))) & 3u];
        }
        const float t = turns(pos, __ldg(p.inv_freq + pair));
        float s, c;
        sincospif(2.f * t, &s, &c);
        cs[kk][pair] = make_float2(c, s);
    }
    __syncthreads();
    if (!active) return;
    const TokenAt a = at[k];
    if (a.b < 0) return;
    // y = x cos + other sin, two values at a time: other is the chunk's
    // partner, or (interleaved) its own values swapped, the sign in sin.
    uint64_t ca[2], cb[2], sa[2], sb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 one = make_float2(1.f, 0.f);
        const float2 u = turned ? cs[k][4 * lane + (kInterleaved ? i : 2 * i)] : one;
        const float2 v = turned ? cs[k][4 * lane + (kInterleaved ? i + 2 : 2 * i + 1)] : one;
        if (kInterleaved) {
            ca[i] = pack_f32x2(u.x, u.x);
            sa[i] = pack_f32x2(-u.y, u.y);
            cb[i] = pack_f32x2(v.x, v.x);
            sb[i] = pack_f32x2(-v.y, v.y);
        } else {
            ca[i] = cb[i] = pack_f32x2(u.x, v.x);
            sa[i] = pack_f32x2(-u.y, -v.y);
            sb[i] = pack_f32x2(u.y, v.y);
        }
    }
    const unsigned gmask = ((1u << kLanes) - 1u) << ((tid & 31) / kLanes * kLanes);
    const int t = tok0 + k;
    // Where the token's heads go: queries, keys, values.
    const int64_t kv_step = append ? static_cast<int64_t>(p.S) * D : D;
    const int64_t kv0 = append ? (static_cast<int64_t>(a.b) * p.Hkv * p.S + a.slot) * D
                               : static_cast<int64_t>(t) * p.Hkv * D;
    __nv_bfloat16* const qd = p.q_out + static_cast<int64_t>(t) * p.Hq * D;
    __nv_bfloat16* const kd = p.k_out + kv0 - p.Hq * kv_step;
    __nv_bfloat16* const vd = p.v_out + kv0 - (p.Hq + p.Hkv) * kv_step;
    const bool norm = p.q_weight != nullptr;
    auto sum_squares = [&](const uint64_t* x, const uint64_t* y) {
        float s0, s1;
        unpack_f32x2(fma_f32x2(x[0], x[0], fma_f32x2(x[1], x[1],
                     fma_f32x2(y[0], y[0], mul_f32x2(y[1], y[1])))), s0, s1);
        float ss = s0 + s1;
#pragma unroll
        for (int off = kLanes / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(gmask, ss, off);
        return ss;
    };
    // Head hh from its two chunks: times inv and the weights, turned, stored.
    auto finish = [&](int hh, uint64_t* x, uint64_t* y, float inv) {
        const bool is_q = hh < p.Hq;
        if (norm) {
            const uint64_t inv2 = pack_f32x2(inv, inv);
            const uint2 wa = is_q ? wq[0] : wk[0], wb = is_q ? wq[1] : wk[1];
            // The norm first: a weight times a large value may overflow.
            x[0] = mul_f32x2(mul_f32x2(x[0], inv2), widen2(wa.x));
            x[1] = mul_f32x2(mul_f32x2(x[1], inv2), widen2(wa.y));
            y[0] = mul_f32x2(mul_f32x2(y[0], inv2), widen2(wb.x));
            y[1] = mul_f32x2(mul_f32x2(y[1], inv2), widen2(wb.y));
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint64_t u = kInterleaved ? swap2(x[e]) : y[e];
            const uint64_t v = kInterleaved ? swap2(y[e]) : x[e];
            const uint64_t nx = fma_f32x2(u, sa[e], mul_f32x2(x[e], ca[e]));
            y[e] = fma_f32x2(v, sb[e], mul_f32x2(y[e], cb[e]));
            x[e] = nx;
        }
        __nv_bfloat16* const dst = is_q ? qd + hh * D : kd + hh * kv_step;
        *reinterpret_cast<uint2*>(dst + ea) = make_uint2(narrow2(x[0]), narrow2(x[1]));
        *reinterpret_cast<uint2*>(dst + eb) = make_uint2(narrow2(y[0]), narrow2(y[1]));
    };
    bool odd = false;  // a mean square near the ends of fp32's range, or beyond
    for (int h = h0; h < heads; h += kBatch * per_tok) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int hh = h + i * per_tok;
            if (hh >= heads) break;
            if (hh >= p.Hq + p.Hkv) {
                __nv_bfloat16* const dst = vd + hh * kv_step;
                *reinterpret_cast<uint2*>(dst + ea) = ra[i];
                *reinterpret_cast<uint2*>(dst + eb) = rb[i];
                continue;
            }
            uint64_t x[2] = {widen2(ra[i].x), widen2(ra[i].y)}, y[2] = {widen2(rb[i].x), widen2(rb[i].y)};
            float inv = 1.f;
            if (norm) {
                const float mean = sum_squares(x, y) * (1.f / D) + p.eps;
                odd |= !(mean < kMeanMax && mean > kMeanMin);
                inv = rsqrtf(mean);
            }
            finish(hh, x, y, inv);
        }
        if (h + kBatch * per_tok < heads) load(h + kBatch * per_tok);
    }
    if (!odd) return;
    // Rare: such heads again, scaled by a power of two (eps too).
#pragma unroll 1
    for (int hh = h0; hh < p.Hq + p.Hkv; hh += per_tok) {
        const __nv_bfloat16* src = row + static_cast<size_t>(hh) * D;
        const uint2 a = __ldcg(reinterpret_cast<const uint2*>(src + ea));
        const uint2 b = __ldcg(reinterpret_cast<const uint2*>(src + eb));
        uint64_t x[2] = {widen2(a.x), widen2(a.y)}, y[2] = {widen2(b.x), widen2(b.y)};
        const float mean = sum_squares(x, y) * (1.f / D) + p.eps;
        if (mean < kMeanMax && mean > kMeanMin) continue;  // as its lanes all find
        const float by = mean > 1.f ? 0x1p-100f : 0x1p100f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            x[e] = mul_f32x2(x[e], pack_f32x2(by, by));
            y[e] = mul_f32x2(y[e], pack_f32x2(by, by));
        }
        finish(hh, x, y, rsqrtf(sum_squares(x, y) * (1.f / D) + p.eps * by * by));
    }
}

template <int D, int kThreads>
cudaError_t launch_rope_t(const RopeParams& p, int per, cudaStream_t stream) {
    const int tok_ctas = (p.T + per - 1) / per;
    const int parts = std::max(1, std::min(kMaxAgeParts, p.S / kAgesPerPart));
    const int age_ctas = p.q_start ? p.B * p.Hkv * parts : 0;
    const char* env = std::getenv("LF_PDL");
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(tok_ctas + age_ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = (env && std::atoi(env) == 0) ? 0 : 1;
    const auto kernel = p.axes > 0 ? (p.interleaved ? lf_rope_kernel<D, true, kThreads, true>
                                                    : lf_rope_kernel<D, false, kThreads, true>)
                                   : (p.interleaved ? lf_rope_kernel<D, true, kThreads, false>
                                                    : lf_rope_kernel<D, false, kThreads, false>);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p, per, tok_ctas, parts);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D>
cudaError_t launch_rope_d(const RopeParams& p, int sms, cudaStream_t stream) {
    // Many tokens: a warp takes one, and warps do not wait for one another.
    // Fewer: 256 threads take one, two or four, so that a token's heads are in
    // flight together. Measured, us for 256 threads (best of 1, 2, 4 tokens) /
    // one warp (with evict-first loads, some 3% slower): 32 + 16 heads of 128,
    // 2000 tokens 12.9 / 17.2, 5000 tokens 27.9 / 28.8, 8000 tokens 39.7 / 37.1,
    // 20000 tokens 89.5 / 84.1; 8 + 16 heads of 64, 2000 tokens 5.5 / 6.8, 5000
    // tokens 10.8 / 10.1, 20000 tokens 32.0 / 26.3. And by tokens per CTA 1 / 2 / 4 (the first heads): 128 tokens
    // 3.8 / 5.6 / 7.1, 600 tokens 5.8 / 7.5 / 10.4, 2000 tokens 15.5 / 13.8 / 12.9.
    if (p.T >= 40 * sms) return launch_rope_t<D, 32>(p, 1, stream);
    int per = max_tokens(kRopeThreads);
    while (per > 1 && (p.T + per - 1) / per < 4 * sms) per >>= 1;
    return launch_rope_t<D, kRopeThreads>(p, per, stream);
}

}  // namespace

cudaError_t launch_rope(int D, const RopeParams& p, int sms, cudaStream_t stream) {
    if (D == 64) return launch_rope_d<64>(p, sms, stream);
    if (D == 128) return launch_rope_d<128>(p, sms, stream);
    return cudaErrorInvalidValue;
}

}  // namespace lf
