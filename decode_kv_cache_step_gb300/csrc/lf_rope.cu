// Norm and position rotation of query and key heads in one pass (sm_103a).
//
// A head x of D values with weight w becomes y = x * w / sqrt(mean(x^2) + eps)
// (no norm without weights); each of the rot / 2 rotated pairs (y_i, y_j)
// turns by the angle a = position * inv_freq_i:
//   (y_i cos a - y_j sin a, y_j cos a + y_i sin a),
// with j = i + rot / 2, or pairs (2i, 2i + 1) when interleaved. Value heads
// are copied. All in fp32, rounded to bf16 once.
//
// Memory bound: each value is read and written once. D / 8 lanes hold a head
// (16 bytes per lane), so the norm is a few shuffles and a half-split partner
// one shuffle away. The angles of a token are shared by all its heads: a CTA
// takes whole rows of a few tokens and computes their cos and sin once, in
// shared memory (fp64 product and reduction to one turn: positions of a
// million times frequencies near 1 need more than 32 bits, and a CTA has
// only a few hundred of them).
#include <algorithm>

#include "lf_kernels.h"
#include "lf_ptx.cuh"

namespace lf {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kBatch = 4;  // head rows a lane group loads before it computes

struct TokenAt {
    int b, slot, pos;  // b < 0: no output for this token
};

template <int D>
__global__ void __launch_bounds__(kRopeThreads) lf_rope_kernel(const RopeParams p, int rows_per_cta,
                                                               int row_ctas, int tok_max) {
    constexpr int kLanes = D / 8;                      // lanes of one head
    constexpr int kGroups = kRopeThreads / kLanes;     // heads a CTA holds at a time
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x;
    const bool append = p.q_start != nullptr;
    if (static_cast<int>(blockIdx.x) >= row_ctas) {
        // Ages of the prompt's tokens, one CTA per (sequence, KV head).
        const int u = blockIdx.x - row_ctas;
        const int b = u / p.Hkv;
        SeqRange r;
        if (!seq_range(p.q_start, p.kv_len, b, p.T, p.S, true, p.dev_err, &r)) return;
        int32_t* m = p.mask + static_cast<size_t>(u) * p.S;
        for (int j = tid; j < r.kv; j += kRopeThreads) m[j] = r.kv - 1 - j;
        return;
    }
    const int heads = p.Hq + 2 * p.Hkv;
    const int half = p.rot / 2;
    TokenAt* at = reinterpret_cast<TokenAt*>(smem);                       // [tok_max]
    float2* cs = reinterpret_cast<float2*>(smem + ((tok_max * sizeof(TokenAt) + 15) & ~size_t(15)));
    const int row0 = blockIdx.x * rows_per_cta;
    const int row_end = min(row0 + rows_per_cta, p.T * heads);
    const int tok0 = row0 / heads;
    const int ntok = (row_end - 1) / heads - tok0 + 1;
    for (int i = tid; i < ntok; i += kRopeThreads) {
        const int t = tok0 + i;
        TokenAt a;
        if (append) {
            a.b = seq_of_row(p.q_start, p.B, t);
            SeqRange r;
            if (seq_range(p.q_start, p.kv_len, a.b, p.T, p.S, true, p.dev_err, &r) && t >= r.q0 &&
                t < r.q0 + r.n) {
                a.slot = r.kv - r.n + (t - r.q0);
                a.pos = a.slot + (p.pos_offset ? p.pos_offset[a.b] : 0);
            } else {
                a.b = -1;
                a.slot = a.pos = 0;
            }
        } else {
            a.b = 0;
            a.slot = 0;
            a.pos = p.positions[t];
        }
        at[i] = a;
    }
    __syncthreads();
    for (int i = tid; i < ntok * half; i += kRopeThreads) {
        const int k = i / half;
        // Half turns, reduced to [-1, 1]: sin and cos of pi times that.
        double a = static_cast<double>(at[k].pos) * static_cast<double>(p.inv_freq[i - k * half]) *
                   0.31830988618379067154;
        a -= 2.0 * rint(a * 0.5);
        float s, c;
        sincospif(static_cast<float>(a), &s, &c);
        cs[i] = make_float2(c, s);
    }
    __syncthreads();

    const int lane = tid % kLanes;
    const int e0 = lane * 8;
    const unsigned gmask = kLanes == 32 ? 0xffffffffu
                                        : ((1u << kLanes) - 1u) << ((tid & 31) / kLanes * kLanes);
    for (int base = row0 + tid / kLanes; base < row_end; base += kBatch * kGroups) {
        uint4 raw[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int row = base + k * kGroups;
            if (row < row_end) {
                const int t = row / heads;
                raw[k] = __ldg(reinterpret_cast<const uint4*>(
                    p.qkv + static_cast<size_t>(t) * p.stride +
                    static_cast<size_t>(row - t * heads) * D + e0));
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int row = base + k * kGroups;
            if (row >= row_end) break;
            const int t = row / heads;
            const int h = row - t * heads;
            const TokenAt a = at[t - tok0];
            if (a.b < 0) continue;
            const bool is_q = h < p.Hq;
            const bool is_v = h >= p.Hq + p.Hkv;
            uint4 res = raw[k];
            if (!is_v) {
                float x[8];
                const __nv_bfloat162* xb = reinterpret_cast<const __nv_bfloat162*>(&raw[k]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = __bfloat1622float2(xb[i]);
                    x[2 * i] = f.x;
                    x[2 * i + 1] = f.y;
                }
                const __nv_bfloat16* w = is_q ? p.q_weight : p.k_weight;
                if (w) {
                    float ss = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
#pragma unroll
                    for (int off = kLanes / 2; off > 0; off >>= 1)
                        ss += __shfl_xor_sync(gmask, ss, off);
                    const float inv = 1.f / sqrtf(ss * (1.f / D) + p.eps);
                    const uint4 wr = __ldg(reinterpret_cast<const uint4*>(w + e0));
                    const __nv_bfloat162* wb = reinterpret_cast<const __nv_bfloat162*>(&wr);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = __bfloat1622float2(wb[i]);
                        x[2 * i] *= inv * f.x;
                        x[2 * i + 1] *= inv * f.y;
                    }
                }
                const float2* c = cs + (t - tok0) * half;
                if (p.interleaved) {
                    if (e0 < p.rot) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 r = c[e0 / 2 + i];
                            const float y0 = x[2 * i], y1 = x[2 * i + 1];
                            x[2 * i] = y0 * r.x - y1 * r.y;
                            x[2 * i + 1] = y1 * r.x + y0 * r.y;
                        }
                    }
                } else {
                    const int dist = half / 8;  // lanes between the two halves
                    const bool low = e0 < half;
                    const bool turned = e0 < p.rot;
                    const int src = turned ? (low ? lane + dist : lane - dist) : lane;
                    const int i0 = low ? e0 : e0 - half;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float o = __shfl_sync(gmask, x[i], src, kLanes);
                        if (turned) {
                            const float2 r = c[i0 + i];
                            x[i] = low ? x[i] * r.x - o * r.y : x[i] * r.x + o * r.y;
                        }
                    }
                }
                res.x = pack_bf16x2(x[0], x[1]);
                res.y = pack_bf16x2(x[2], x[3]);
                res.z = pack_bf16x2(x[4], x[5]);
                res.w = pack_bf16x2(x[6], x[7]);
            }
            __nv_bfloat16* dst;
            if (is_q) {
                dst = p.q_out + (static_cast<size_t>(t) * p.Hq + h) * D;
            } else {
                const int kvh = is_v ? h - p.Hq - p.Hkv : h - p.Hq;
                dst = (is_v ? p.v_out : p.k_out) +
                      (append ? ((static_cast<size_t>(a.b) * p.Hkv + kvh) * p.S + a.slot)
                              : (static_cast<size_t>(t) * p.Hkv + kvh)) * D;
            }
            *reinterpret_cast<uint4*>(dst + e0) = res;
        }
    }
}

template <int D>
cudaError_t launch_rope_t(const RopeParams& p, int sms, cudaStream_t stream) {
    constexpr int kGroups = kRopeThreads / (D / 8);
    const int heads = p.Hq + 2 * p.Hkv;
    const long long rows = static_cast<long long>(p.T) * heads;
    // A few tokens per CTA, fewer rows when the call is too small to fill the
    // GPU that way.
    long long per = std::min<long long>(4LL * heads, (rows + 4LL * sms - 1) / (4LL * sms));
    per = std::max<long long>(1, (per + kGroups - 1) / kGroups) * kGroups;
    const int row_ctas = static_cast<int>((rows + per - 1) / per);
    const int tok_max = static_cast<int>(per / heads) + 2;
    const size_t smem = ((tok_max * sizeof(TokenAt) + 15) & ~size_t(15)) +
                        static_cast<size_t>(tok_max) * (p.rot / 2) * sizeof(float2);
    const int age_ctas = p.q_start ? p.B * p.Hkv : 0;
    lf_rope_kernel<D><<<row_ctas + age_ctas, kRopeThreads, smem, stream>>>(
        p, static_cast<int>(per), row_ctas, tok_max);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(int D, const RopeParams& p, int sms, cudaStream_t stream) {
    if (D == 64) return launch_rope_t<64>(p, sms, stream);
    if (D == 128) return launch_rope_t<128>(p, sms, stream);
    return cudaErrorInvalidValue;
}

}  // namespace lf
