// Attention of packed query rows over in-order caches (sm_103a): the sliding
// window with visible first tokens, and the shared prefix of a decode batch.
//
// One pass over a row's visible keys with the running maximum m and sum l of
// its softmax (log2 domain): s = scale * q.k, p = 2^(s - m), O += p v. The
// row's output is O / l; with pieces, (m, l) and the unnormalised O are
// written instead and a later kernel joins them.
#include <math.h>

#include "lf_kernels.h"
#include "lf_ptx.cuh"

namespace lf {
namespace {

// One warp, one query row, keys visible by select: lane i scores key j0 + i of
// each 32, then the lanes share the values' columns. (m, l) and the lane's
// columns lane * D / 32 ... of O.
template <int D>
__device__ void attn_row(const __nv_bfloat16* q, const __nv_bfloat16* k, const __nv_bfloat16* v,
                         int j_lo, int j_hi, int lo, int hi, int sinks, float scale_log2, float& m,
                         float& l, float (&o)[D / 32]) {
    const int lane = threadIdx.x & 31;
    constexpr int kC = D / 32;
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
#pragma unroll
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
        for (unsigned left = any; left; left &= left - 1) {
            const int i = __ffs(left) - 1;
            const float pj = __shfl_sync(0xffffffffu, p, i);
            const __nv_bfloat16* vr = v + static_cast<size_t>(j0 + i) * D + lane * kC;
#pragma unroll
            for (int c = 0; c < kC; ++c) o[c] += pj * __bfloat162float(vr[c]);
        }
    }
}

constexpr int kRowWarps = 8;

// The simplest form: one warp per query row, every key of the row in one piece.
template <int D>
__global__ void __launch_bounds__(kRowWarps * 32) lf_attn_rows_kernel(const AttnParams p) {
    const int lane = threadIdx.x & 31;
    const size_t row = static_cast<size_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
    if (row >= static_cast<size_t>(p.T) * p.Hq) return;
    const int t = static_cast<int>(row / p.Hq);
    const int h = static_cast<int>(row - static_cast<size_t>(t) * p.Hq);
    const int n = seq_of_row(p.q_start, p.N, t);
    SeqRange r;
    if (!seq_range(p.q_start, p.kv_len, n, p.T, p.S, p.causal, p.dev_err, &r)) return;
    if (t < r.q0 || t >= r.q0 + r.n) return;
    int lo = 0, hi = r.kv, sinks = 0;
    if (p.causal) {
        hi = r.kv - r.n + (t - r.q0) + 1;
        if (p.window > 0) lo = max(0, hi - p.window);
        sinks = p.sinks;
    }
    const size_t base = (static_cast<size_t>(n) * p.Hkv + h / (p.Hq / p.Hkv)) * p.S * D;
    const __nv_bfloat16* q = p.q + row * D;
    float m = -INFINITY, l = 0.f, o[D / 32];
#pragma unroll
    for (int c = 0; c < D / 32; ++c) o[c] = 0.f;
    const int first = min(sinks, lo);
    attn_row<D>(q, p.k + base, p.v + base, 0, first, lo, hi, sinks, p.scale_log2, m, l, o);
    attn_row<D>(q, p.k + base, p.v + base, lo, hi, lo, hi, sinks, p.scale_log2, m, l, o);
    if (p.pieces == 0) {
        const float il = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
            p.out[row * D + lane * (D / 32) + c] = __float2bfloat16_rn(l == 0.f ? 0.f : o[c] * il);
    } else {
        if (lane == 0) p.part_ml[row] = make_float2(m, l);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) p.part_o[row * D + lane * (D / 32) + c] = o[c];
    }
}

}  // namespace

int attention_pieces(int, int, int, int, int, bool causal, int, int, int) { return causal ? 0 : 1; }

cudaError_t launch_attention(int D, int G, const AttnParams& p, cudaStream_t stream) {
    const size_t rows = static_cast<size_t>(p.T) * p.Hq;
    const unsigned grid = static_cast<unsigned>((rows + kRowWarps - 1) / kRowWarps);
    if (D == 64)
        lf_attn_rows_kernel<64><<<grid, kRowWarps * 32, 0, stream>>>(p);
    else if (D == 128)
        lf_attn_rows_kernel<128><<<grid, kRowWarps * 32, 0, stream>>>(p);
    else
        return cudaErrorInvalidValue;
    return cudaGetLastError();
}

}  // namespace lf
