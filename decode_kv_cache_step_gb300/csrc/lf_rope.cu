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
// four tokens, and a lane keeps its 4 angles and its weights for all of them.
// The angles are formed once per CTA in shared memory (fp64 product and
// reduction to one turn: positions of a million times frequencies near 1 need
// more than 32 bits, and a CTA has only a few hundred of them) while the
// first heads' loads are in flight.
#include <stdlib.h>

#include <algorithm>

#include "lf_kernels.h"
#include "lf_ptx.cuh"

namespace lf {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kBatch = 6;      // heads whose loads a lane has in flight
constexpr int kMaxTokens = 4;  // tokens of a CTA

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

__device__ __forceinline__ void widen4(const uint2& v, float* x) {
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v.y));
    x[0] = a.x;
    x[1] = a.y;
    x[2] = b.x;
    x[3] = b.y;
}

template <int D>
__global__ void __launch_bounds__(kRopeThreads) lf_rope_kernel(const RopeParams p, int tok_per_cta,
                                                               int tok_ctas) {
    constexpr int kLanes = D / 8;                   // lanes of one head
    constexpr int kGroups = kRopeThreads / kLanes;  // heads a CTA holds at a time
    __shared__ TokenAt at[kMaxTokens];
    __shared__ float2 cs[kMaxTokens][D / 2];
    const int tid = threadIdx.x;
    allow_dependent_launch();
    grid_dependency_wait();
    const bool append = p.q_start != nullptr;
    if (static_cast<int>(blockIdx.x) >= tok_ctas) {
        // Ages of the prompt's tokens, one CTA per (sequence, KV head).
        const int u = blockIdx.x - tok_ctas;
        const int b = u / p.Hkv;
        SeqRange r;
        if (!seq_range(p.q_start, p.kv_len, b, p.T, p.S, true, &r)) {
            if (tid == 0) atomicOr(p.dev_err, kErrBadLength);
            return;
        }
        int32_t* m = p.mask + static_cast<size_t>(u) * p.S;
        for (int j = tid; j < r.kv; j += kRopeThreads) m[j] = r.kv - 1 - j;
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
    if (p.interleaved || !turned) {
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
                ra[i] = __ldcs(reinterpret_cast<const uint2*>(src + ea));
                rb[i] = __ldcs(reinterpret_cast<const uint2*>(src + eb));
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
        } else {
            a.pos = p.positions[t];
        }
        if ((tid & 31) == 0) at[i] = a;
    }
    __syncthreads();
    for (int i = tid; i < ntok * half; i += kRopeThreads) {
        const int kk = i / half;
        // Half turns, reduced to [-1, 1]: sin and cos of pi times that.
        double a = static_cast<double>(at[kk].pos) *
                   static_cast<double>(__ldg(p.inv_freq + (i - kk * half))) * 0.31830988618379067154;
        a -= 2.0 * rint(a * 0.5);
        float s, c;
        sincospif(static_cast<float>(a), &s, &c);
        cs[kk][i - kk * half] = make_float2(c, s);
    }
    __syncthreads();
    if (!active) return;
    const TokenAt a = at[k];
    if (a.b < 0) return;
    float c[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = turned ? cs[k][4 * lane + i] : make_float2(1.f, 0.f);
        c[i] = v.x;
        s[i] = v.y;
    }
    const unsigned gmask = ((1u << kLanes) - 1u) << ((tid & 31) / kLanes * kLanes);
    const int t = tok0 + k;
    for (int h = h0; h < heads; h += kBatch * per_tok) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int hh = h + i * per_tok;
            if (hh >= heads) break;
            const bool is_q = hh < p.Hq;
            const bool is_v = hh >= p.Hq + p.Hkv;
            uint2 oa = ra[i], ob = rb[i];
            if (!is_v) {
                float x[4], y[4];
                widen4(ra[i], x);
                widen4(rb[i], y);
                if (p.q_weight) {
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) ss += x[e] * x[e] + y[e] * y[e];
#pragma unroll
                    for (int off = kLanes / 2; off > 0; off >>= 1)
                        ss += __shfl_xor_sync(gmask, ss, off);
                    const float inv = 1.f / sqrtf(ss * (1.f / D) + p.eps);
                    float wa[4], wb[4];
                    widen4(is_q ? wq[0] : wk[0], wa);
                    widen4(is_q ? wq[1] : wk[1], wb);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[e] *= inv * wa[e];
                        y[e] *= inv * wb[e];
                    }
                }
                if (turned) {
                    if (p.interleaved) {
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            const float x0 = x[e], y0 = y[e];
                            x[e] = x0 * c[e / 2] - x[e + 1] * s[e / 2];
                            x[e + 1] = x[e + 1] * c[e / 2] + x0 * s[e / 2];
                            y[e] = y0 * c[2 + e / 2] - y[e + 1] * s[2 + e / 2];
                            y[e + 1] = y[e + 1] * c[2 + e / 2] + y0 * s[2 + e / 2];
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float x0 = x[e];
                            x[e] = x0 * c[e] - y[e] * s[e];
                            y[e] = y[e] * c[e] + x0 * s[e];
                        }
                    }
                }
                oa = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
                ob = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
            }
            __nv_bfloat16* dst;
            if (is_q) {
                dst = p.q_out + (static_cast<size_t>(t) * p.Hq + hh) * D;
            } else {
                const int kvh = is_v ? hh - p.Hq - p.Hkv : hh - p.Hq;
                dst = (is_v ? p.v_out : p.k_out) +
                      (append ? ((static_cast<size_t>(a.b) * p.Hkv + kvh) * p.S + a.slot)
                              : (static_cast<size_t>(t) * p.Hkv + kvh)) * D;
            }
            *reinterpret_cast<uint2*>(dst + ea) = oa;
            *reinterpret_cast<uint2*>(dst + eb) = ob;
        }
        if (h + kBatch * per_tok < heads) load(h + kBatch * per_tok);
    }
}

template <int D>
cudaError_t launch_rope_t(const RopeParams& p, int sms, cudaStream_t stream) {
    // Four tokens per CTA, fewer when the call is too small to fill the GPU.
    int per = kMaxTokens;
    while (per > 1 && (p.T + per - 1) / per < 4 * sms) per >>= 1;
    const int tok_ctas = (p.T + per - 1) / per;
    const int age_ctas = p.q_start ? p.B * p.Hkv : 0;
    const char* env = std::getenv("LF_PDL");
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(tok_ctas + age_ctas);
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = (env && std::atoi(env) == 0) ? 0 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, lf_rope_kernel<D>, p, per, tok_ctas);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(int D, const RopeParams& p, int sms, cudaStream_t stream) {
    if (D == 64) return launch_rope_t<64>(p, sms, stream);
    if (D == 128) return launch_rope_t<128>(p, sms, stream);
    return cudaErrorInvalidValue;
}

}  // namespace lf
