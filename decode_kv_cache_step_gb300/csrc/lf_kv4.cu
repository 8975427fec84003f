// A cache held in 4 bits: a prompt's rows into it and back, and decode
// attention over it (sm_103a).
//
// A row of d values has d / 32 groups of 32. A group's scale is s = max|x| / 7
// rounded to bf16, a value's code round(x / s) in [-7, 7] (ties to even), and
// the value it stands for code * s. A row takes d / 2 bytes of codes (plus 8, in
// nibbles) and d / 32 scales: 4.5 bits a value, 3.56 times fewer bytes than
// bf16. (A power of two as the scale would save 8 bits in 136 and double the
// error of half the groups.)
//
// Order of a row's codes: value c of group g lies in nibble
// ((r / e) * (d / 32) + g) * e + r % e, r = c % 32, low nibble of a byte first,
// with pieces of e = 8 in keys and e = 4 in values. The pieces of the groups
// take turns so that what one lane of a matrix product needs of a row, some
// codes of each group, lies together (see lf_kv4_attn_kernel).
//
// Measured (8 KV heads of 128): 20.3K tokens packed in 48 us, 5.6 TB/s read and
// written, and unpacked in 36; 64 caches of 4096 to 16384 slots attended with 32
// query heads in 175 us, 4.6 TB/s, one of 16384 in 12.8.
#include <cuda_fp16.h>
#include <math.h>
#include <stdlib.h>

#include <algorithm>
#include <type_traits>

#include "../../include/lf_decode.h"
#include "lf_kernels.h"
#include "lf_ptx.cuh"

namespace lf {
namespace {

constexpr int kPackThreads = 256;
constexpr int kPackSlots = 64;  // slots of one (sequence, KV head) a CTA packs or unpacks

// ------------------------------------------------------------ quantisation --

// Codes of 8 values (4 lanes hold a group): nibble i of the result is value i's
// code plus 8. *scale gets the group's scale.
//
// The codes are those of the exact quotients. x = X 2^a and s = Y 2^b have
// 8-bit integers X, Y, so where x / s is not halfway between two integers it is
// at least 2^-10 away from that: a product with the rounded reciprocal (off by
// 2^-20 at most), rounded to multiples of 2^-12, is on the right side, and a tie
// is a tie again. Both roundings are sums with a constant, the second of which
// leaves the code plus 8 in the low bits, and a sum of those times powers of 16
// is the word: packing is bound by memory, and a conversion per value is not.
__device__ __forceinline__ float bf16_at(const uint32_t (&w)[4], int i) {
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
}

__device__ __forceinline__ uint32_t quantise8(const uint4 v, unsigned mask, __nv_bfloat16* scale) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t two = 0;  // the largest magnitudes of the halves
#pragma unroll
    for (int i = 0; i < 4; ++i) two = __vimax3_u16x2(two, w[i] & 0x7fff7fffu, 0u);
    uint32_t top = max(two & 0xffffu, two >> 16);
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) top = max(top, __shfl_xor_sync(mask, top, off));
    // A group with a value that is not finite stands for NaN.
    const float amax = __uint_as_float(top << 16);
    // (The product with the rounded 1 / 7 rounds like the quotient: that is at
    // least 2^-12 of itself away from halfway between two bf16, as 8 bits over 7.)
    const __nv_bfloat16 s =
        top < 0x7f80u ? __float2bfloat16_rn(__fmul_rn(amax, 1.f / 7.f)) : __ushort_as_bfloat16(0x7fffu);
    *scale = s;
    constexpr float kSnap = 0x1.8p11f;              // sums are multiples of 2^-12
    constexpr float kWhole = 0x1.8p23f + 8 - kSnap;  // and then integers
    uint32_t codes = 0;
    if (amax >= 0x1p-60f && top < 0x7f80u) {
        const float inv = __frcp_rn(__bfloat162float(s));
#pragma unroll
        for (int i = 7; i >= 0; --i) {
            const float t = __fadd_rn(__fmaf_rn(bf16_at(w, i), inv, kSnap), kWhole);
            codes = codes * 16u + __float_as_uint(t);
        }
        // Less what else the eight sums hold.
        codes -= 0x4b400000u * 0x11111111u;
    } else {
        // Small groups times 2^64, so that the reciprocal is finite.
        const float sf = __bfloat162float(s) * 0x1p64f;
        const bool some = sf > 0.f;  // neither 0 nor NaN
        const float inv = some ? 1.f / sf : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float t = some ? bf16_at(w, i) * 0x1p64f * inv : 0.f;
            t = __fadd_rn(__fadd_rn(t, kSnap), -kSnap);
            const int c = min(7, max(-7, __float2int_rn(t)));
            codes |= static_cast<uint32_t>(c + 8) << (4 * i);
        }
    }
    return codes;
}

// Where the 8 codes of values 8 i .. 8 i + 7 of a row lie: one piece of 8, or
// two of 4 that lie `kPair` bytes apart.
template <int D>
__device__ __forceinline__ void store_k8(uint8_t* row, int i, uint32_t codes) {
    const int g = i >> 2, r8 = i & 3;
    *reinterpret_cast<uint32_t*>(row + (r8 * (D / 32) + g) * 4) = codes;
}
template <int D>
__device__ __forceinline__ void store_v8(uint8_t* row, int i, uint32_t codes) {
    const int g = i >> 2, r4 = (i & 3) * 2;
    *reinterpret_cast<uint16_t*>(row + (r4 * (D / 32) + g) * 2) = static_cast<uint16_t>(codes);
    *reinterpret_cast<uint16_t*>(row + ((r4 + 1) * (D / 32) + g) * 2) = static_cast<uint16_t>(codes >> 16);
}
template <int D>
__device__ __forceinline__ uint32_t load_k8(const uint8_t* row, int i) {
    return __ldg(reinterpret_cast<const uint32_t*>(row + ((i & 3) * (D / 32) + (i >> 2)) * 4));
}
template <int D>
__device__ __forceinline__ uint32_t load_v8(const uint8_t* row, int i) {
    const int g = i >> 2, r4 = (i & 3) * 2;
    const uint32_t lo = __ldg(reinterpret_cast<const uint16_t*>(row + (r4 * (D / 32) + g) * 2));
    const uint32_t hi = __ldg(reinterpret_cast<const uint16_t*>(row + ((r4 + 1) * (D / 32) + g) * 2));
    return lo | hi << 16;
}

// The range of slots of sequence b, and whether it fits both buffers.
struct SlotRange {
    int first, end;
};
__device__ __forceinline__ bool slot_range(const Kv4PackParams& p, int b, SlotRange* r) {
    r->first = p.kv_from ? p.kv_from[b] : 0;
    r->end = p.kv_len[b];
    return r->first >= 0 && r->first <= r->end && r->end <= min(p.P, p.S);
}

// Slots of bf16 caches [B][Hkv][P][D] into the 4-bit cache [B][Hkv][S], and the
// ages of an in-order cache. Memory bound: a thread takes 16 bytes of a row, and
// the loads of its four rows (d = 128) are in flight at once. (20.3K tokens of 8
// heads packed and unpacked 79.3 us, 89% of the copy rate; with 128 slots a CTA
// 98, with 32 82; read without the streaming hint 85.)
template <int D>
__global__ void __launch_bounds__(kPackThreads) lf_kv4_pack_kernel(const Kv4PackParams p) {
    allow_dependent_launch();
    grid_dependency_wait();
    const int u = blockIdx.y;
    const int b = u / p.Hkv;
    const int j0 = blockIdx.x * kPackSlots;
    const int tid = threadIdx.x;
    SlotRange r;
    if (!slot_range(p, b, &r)) {
        if (tid == 0 && blockIdx.x == 0) atomicOr(p.dev_err, kErrBadLength);
        return;
    }
    if (tid < kPackSlots && j0 + tid < r.end)
        p.mask[static_cast<size_t>(u) * p.S + j0 + tid] = r.end - 1 - (j0 + tid);
    constexpr int kLanes = D / 8;
    constexpr int kRows = kPackThreads / kLanes;
    constexpr int kBatch = kPackSlots / kRows;  // rows of a thread, all in flight
    const int i = tid % kLanes;
    const unsigned mask = 0xfu << (tid & 28);
    // The thread's first row; the others follow kRows apart.
    const int jt = j0 + tid / kLanes;
    const size_t src = (static_cast<size_t>(u) * p.P + jt) * D + 8 * i;
    const size_t dst = static_cast<size_t>(u) * p.S + jt;
    const auto inside = [&](int n) { return jt + n * kRows >= r.first && jt + n * kRows < r.end; };
    uint4 k[kBatch], v[kBatch];
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
        if (!inside(n)) continue;
        k[n] = __ldcs(reinterpret_cast<const uint4*>(p.k + src + n * kRows * D));
        v[n] = __ldcs(reinterpret_cast<const uint4*>(p.v + src + n * kRows * D));
    }
    uint8_t* const k4 = p.k4 + dst * (D / 2);
    uint8_t* const v4 = p.v4 + dst * (D / 2);
    __nv_bfloat16* const k_scale = p.k_scale + dst * (D / 32) + (i >> 2);
    __nv_bfloat16* const v_scale = p.v_scale + dst * (D / 32) + (i >> 2);
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
        if (!inside(n)) continue;
        __nv_bfloat16 s;
        store_k8<D>(k4 + n * kRows * (D / 2), i, quantise8(k[n], mask, &s));
        if ((i & 3) == 0) k_scale[n * kRows * (D / 32)] = s;
        store_v8<D>(v4 + n * kRows * (D / 2), i, quantise8(v[n], mask, &s));
        if ((i & 3) == 0) v_scale[n * kRows * (D / 32)] = s;
    }
}

// The values of 8 codes (plus 8), two at a time: 0x4300 | c is the bf16 128 + c, so
// a difference gives the code, exactly, and the product with the scale is rounded
// once. Codes i and i + 4 share a register.
__device__ __forceinline__ uint4 values8(uint32_t codes, __nv_bfloat16 scale) {
    const __nv_bfloat162 bias = __halves2bfloat162(__ushort_as_bfloat16(0x4308u), __ushort_as_bfloat16(0x4308u));
    const __nv_bfloat162 s2 = __halves2bfloat162(scale, scale);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t c = ((codes >> (4 * i)) & 0x000f000fu) | 0x43004300u;
        const __nv_bfloat162 v = __hmul2(__hsub2(*reinterpret_cast<const __nv_bfloat162*>(&c), bias), s2);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    return make_uint4(__byte_perm(w[0], w[1], 0x5410u), __byte_perm(w[2], w[3], 0x5410u),
                      __byte_perm(w[0], w[1], 0x7632u), __byte_perm(w[2], w[3], 0x7632u));
}

template <int D>
__global__ void __launch_bounds__(kPackThreads) lf_kv4_unpack_kernel(const Kv4PackParams p) {
    allow_dependent_launch();
    grid_dependency_wait();
    const int u = blockIdx.y;
    const int b = u / p.Hkv;
    const int j0 = blockIdx.x * kPackSlots;
    const int tid = threadIdx.x;
    SlotRange r;
    if (!slot_range(p, b, &r)) {
        if (tid == 0 && blockIdx.x == 0) atomicOr(p.dev_err, kErrBadLength);
        return;
    }
    constexpr int kLanes = D / 8;
    constexpr int kRows = kPackThreads / kLanes;
    const int i = tid % kLanes;
    constexpr int kBatch = kPackSlots / kRows;
    const int jt = j0 + tid / kLanes;
    const size_t src = static_cast<size_t>(u) * p.S + jt;
    const size_t dst = (static_cast<size_t>(u) * p.P + jt) * D + 8 * i;
    const auto inside = [&](int n) { return jt + n * kRows >= r.first && jt + n * kRows < r.end; };
    const uint8_t* const k4 = p.k4 + src * (D / 2);
    const uint8_t* const v4 = p.v4 + src * (D / 2);
    const __nv_bfloat16* const k_scale = p.k_scale + src * (D / 32) + (i >> 2);
    const __nv_bfloat16* const v_scale = p.v_scale + src * (D / 32) + (i >> 2);
    uint32_t k[kBatch], v[kBatch];
    __nv_bfloat16 ks[kBatch], vs[kBatch];
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
        if (!inside(n)) continue;
        k[n] = load_k8<D>(k4 + n * kRows * (D / 2), i);
        v[n] = load_v8<D>(v4 + n * kRows * (D / 2), i);
        ks[n] = k_scale[n * kRows * (D / 32)];
        vs[n] = v_scale[n * kRows * (D / 32)];
    }
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
        if (!inside(n)) continue;
        __stcs(reinterpret_cast<uint4*>(p.k_out + dst + n * kRows * D), values8(k[n], ks[n]));
        __stcs(reinterpret_cast<uint4*>(p.v_out + dst + n * kRows * D), values8(v[n], vs[n]));
    }
}

// -------------------------------------------------------- decode attention --

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxChunkSlots = 2048;
constexpr int kTileSlots = 32;
constexpr int kMaxWarpTiles = kMaxChunkSlots / kTileSlots / kWarps;
// A warp's ring of tiles of 32 slots in shared memory.
template <int D>
struct Ring {
    static constexpr int kKRow = D / 2;
    // Rows of values 16 bytes apart: four lanes that read rows 2 c at once then
    // touch different banks.
    static constexpr int kVRow = D / 2 + 16;
    static constexpr int kScaleRow = D / 16;
    static constexpr int kVOff = kTileSlots * kKRow;
    static constexpr int kKScaleOff = kVOff + kTileSlots * kVRow;
    static constexpr int kVScaleOff = kKScaleOff + kTileSlots * kScaleRow;
    static constexpr int kStage = kVScaleOff + kTileSlots * kScaleRow;
    static constexpr int kStages = D == 128 ? 3 : 6;
    // Behind the tiles: the scales of one tile's keys, and of one tile's values, in
    // fp32 (rows of d / 32).
    static constexpr int kKWideOff = kStages * kStage;
    static constexpr int kVWideOff = kKWideOff + kTileSlots * (D / 8);
    static constexpr int kWarp = kVWideOff + kTileSlots * (D / 8);
    static constexpr int kAlloc = kWarps * kWarp;
};
constexpr float kCode = 0x1p-24f;  // what the integer 1 in a half's low bits is worth

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1, const float (&c)[4]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]),
          "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Asynchronous copies of N bytes into shared memory (nothing is read and zeros are
// stored with there = false), in groups that complete in order.
template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool there) {
    const int bytes = there ? N : 0;
    if constexpr (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(bytes)
                     : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int N>
__device__ __forceinline__ void shared_words(const uint8_t* a, uint32_t (&w)[N]) {
    static_assert(N == 1 || N == 2 || N == 4, "words of a load");
    if constexpr (N == 1) {
        w[0] = *reinterpret_cast<const uint32_t*>(a);
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(a);
        w[0] = v.x;
        w[1] = v.y;
    } else {
        const uint4 v = *reinterpret_cast<const uint4*>(a);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    }
}

__device__ __forceinline__ float scale_of(uint32_t word, int odd) {
    return __uint_as_float(odd ? word & 0xffff0000u : word << 16);
}

// One CTA: chunk blockIdx.x of unit blockIdx.y. Each warp takes 32 slots at a
// time, where one of them is live, through a ring of its own in shared memory
// (asynchronous copies; no other warp is waited for):
//   S^T[16 x 8] = K[16 x d] Q^T[d x 8]          per group, times the key's scale
//   O^T[d x 8] += V^T[d x 16] (P s)^T[16 x 8]   per group, P s the weights times
//                                               the values' scales
// A code needs no conversion: an integer n in the low bits of a half is the half
// n 2^-24 (a subnormal; linear up to n = 2047, and the tensor cores take it), so
// the codes at bits 0 and 16 of a word are an operand after one AND, those at
// bits 4 and 20, as 16 n, after another. The 16 is taken out of q, or of the row
// of O. Codes are stored plus 8: the logits start at -8 sum q s (one product of
// the scales with q's sums over the groups, in three bf16 parts), and 8 sum P s,
// a product per group with constant codes, is taken off O at the end.
//
// Tensor cores by registers (mma.sync): G rows of queries leave a 128-row
// accumulator empty, and the codes would have to be widened through shared memory.
// What bounds it: long caches, instructions: 616 a warp for 32 slots, half of
// them on the integer units (AND, shift, byte permutation), which are busy 49% of
// the cycles, issue 55%, DRAM 66%; 12 warps an SM, as many as 168 registers
// leave. One cache of 16384 slots: latency, 344 CTAs of three tiles a warp, each
// with a prologue (q, its sums) and an epilogue as long as two more.
// 64 caches of 4096 to 16384 slots, us: 175. Steps on the way, each against the
// one before it: the ring and a rare reference 211 (275), the next tile's logits
// beside this one's values 202, tiles of 32 slots 186 (of 16), scales widened once
// a tile 178 (182, by each lane that uses them). Two stages at 4 CTAs an SM took
// 197 against 186, tiles read straight into registers 254, chunks of 1024 slots
// 212, of 4096 183 (and 16 caches took longer).
template <int D, int G>
__global__ void __launch_bounds__(kThreads, 3) lf_kv4_attn_kernel(const Kv4Params p) {
    using R = Ring<D>;
    constexpr int NG = D / 32;
    extern __shared__ __align__(16) uint8_t s_ring[];
    __shared__ uint2 s_tiles[kWarps][kMaxWarpTiles];  // live slots, index in the chunk
    __shared__ float s_m[kWarps][G], s_l[kWarps][G];
    __shared__ __align__(16) uint8_t s_new[2][D / 2];  // the token's row in 4 bits
    __shared__ __nv_bfloat16 s_new_scale[2][NG];
    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const int lane = tid & 31;
    const int r = lane >> 2;
    const int c = lane & 3;
    const int u = blockIdx.y;
    const int b = u / p.Hkv;
    const int kvh = u - b * p.Hkv;
    const int S = p.S;
    const int slot0 = blockIdx.x * p.chunk_slots;
    const int slots = min(p.chunk_slots, S - slot0);
    // (The join is not let in early: its CTAs, waiting, took the places of this
    // kernel's next ones, 152 units of 2400 slots, d = 64, 18.9 us against 14.0.)
    grid_dependency_wait();

    int ws = p.write_slot[u];
    // The warp's slots: 32 of every 128. Their ages first, all in flight.
    constexpr int kBlocks = kMaxChunkSlots / 32 / kWarps;
    int32_t* const ages = p.mask + static_cast<size_t>(u) * S + slot0;
    int age[kBlocks];
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
        const int i = (k * kWarps + warp) * 32 + lane;
        age[k] = i < slots ? ages[i] : -1;
    }
    // q of head r: the lane's values 8 c .. 8 c + 7 of each group.
    const size_t row0 = static_cast<size_t>(b) * p.Hq + static_cast<size_t>(kvh) * G;
    uint4 qv[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g)
        qv[g] = r < G ? *reinterpret_cast<const uint4*>(p.q + (row0 + r) * D + 32 * g + 8 * c)
                      : make_uint4(0, 0, 0, 0);
    if (ws < -1 || ws >= S) {
        if (tid == 0 && blockIdx.x == 0) atomicOr(p.dev_err, LF_DEVERR_BAD_WRITE_SLOT);
        ws = -1;
    }
    const int wi = ws - slot0;
    const bool mine = ws >= 0 && wi >= 0 && wi < slots && ((wi >> 5) & (kWarps - 1)) == warp;
    // The warp's tiles with a live slot.
    int tiles = 0;
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
        const int block = k * kWarps + warp;
        bool live = age[k] >= 0;
        if (mine && block * 32 + lane == wi && !live) {
            ages[wi] = 0;
            live = true;
        }
        const uint32_t bits = __ballot_sync(0xffffffffu, live);
        if (lane == 0 && bits) s_tiles[warp][tiles] = make_uint2(bits, block);
        tiles += bits ? 1 : 0;
    }
    __syncwarp();

    // Copies of a tile: 16 bytes of codes a lane at a time, a row's scales.
    const size_t unit0 = static_cast<size_t>(u) * S + slot0;
    constexpr int kRowChunks = D / 32;             // 16-byte chunks of a row's codes
    constexpr int kCopies = kRowChunks;            // of a lane, per tile and operand
    constexpr int kStep = 32 / kRowChunks;         // rows between them
    const int crow = lane / kRowChunks;
    const uint8_t* const pk = p.k4 + unit0 * (D / 2) + lane * 16;
    const uint8_t* const pv = p.v4 + unit0 * (D / 2) + lane * 16;
    const uint8_t* const pks = reinterpret_cast<const uint8_t*>(p.k_scale) + (unit0 + lane) * R::kScaleRow;
    const uint8_t* const pvs = reinterpret_cast<const uint8_t*>(p.v_scale) + (unit0 + lane) * R::kScaleRow;
    uint8_t* const ring = s_ring + warp * R::kWarp;
    const uint32_t dk = smem_u32(ring) + lane * 16;
    const uint32_t dv = smem_u32(ring) + R::kVOff + crow * R::kVRow + (lane % kRowChunks) * 16;
    const uint32_t ds = smem_u32(ring) + R::kKScaleOff + lane * R::kScaleRow;
    auto copy_tile = [&](int tile, int stage) {
        const int at = stage * R::kStage;
        const uint8_t* const k = pk + tile * (kTileSlots * D / 2);
        const uint8_t* const v = pv + tile * (kTileSlots * D / 2);
        const uint8_t* const k_scales = pks + tile * (kTileSlots * R::kScaleRow);
        const uint8_t* const v_scales = pvs + tile * (kTileSlots * R::kScaleRow);
        const auto rows = [&](int most) {  // copies of the rows that are there
#pragma unroll
            for (int i = 0; i < kCopies; ++i) {
                copy_async<16>(dk + at + i * 512, k + i * 512, crow + i * kStep < most);
                copy_async<16>(dv + at + i * kStep * R::kVRow, v + i * 512, crow + i * kStep < most);
            }
            copy_async<R::kScaleRow>(ds + at, k_scales, lane < most);
            copy_async<R::kScaleRow>(ds + at + kTileSlots * R::kScaleRow, v_scales, lane < most);
        };
        const int most = slots - tile * kTileSlots;
        if (most >= kTileSlots)
            rows(kTileSlots);
        else
            rows(most);
    };
#pragma unroll
    for (int i = 0; i < R::kStages; ++i) {
        if (i < tiles) copy_tile(s_tiles[warp][i].y, i);
        copy_commit();
    }

    // The token's row into its slot, by the warp that holds it: lanes below D / 8
    // the key, the next D / 8 the value. What the copies bring of the row may be
    // old or new: the warp puts s_new in its place.
    if (mine) {
        const int i = lane % (D / 8);
        const bool is_v = lane / (D / 8) == 1;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (lane < D / 4)
            x = *reinterpret_cast<const uint4*>((is_v ? p.new_v : p.new_k) + static_cast<size_t>(u) * D + 8 * i);
        __nv_bfloat16 s;
        const uint32_t codes = quantise8(x, 0xfu << (lane & 28), &s);
        const size_t at = static_cast<size_t>(u) * S + ws;
        if (lane < D / 4) {
            if (is_v) {
                store_v8<D>(p.v4 + at * (D / 2), i, codes);
                store_v8<D>(s_new[1], i, codes);
            } else {
                store_k8<D>(p.k4 + at * (D / 2), i, codes);
                store_k8<D>(s_new[0], i, codes);
            }
            if ((i & 3) == 0) {
                (is_v ? p.v_scale : p.k_scale)[at * NG + (i >> 2)] = s;
                s_new_scale[is_v][i >> 2] = s;
            }
        }
        __syncwarp();
    }

    // q as halves of 2^13 to 2^14 for the largest, a sixteenth of that where odd nibbles
    // meet it: within 2^-34 of the head's largest value (2^-38 at even places), exact for
    // values of at least 2^-26 of it.
    uint32_t qf[NG][4];      // k steps of a group: codes at even, then odd nibbles
    uint32_t start[2];       // -8 sum q of the groups: an operand with the scales
    float qs[2];             // what a logit's sum is worth (log2 domain)
    {
        uint32_t top = 0;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const uint32_t w[4] = {qv[g].x, qv[g].y, qv[g].z, qv[g].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
                if (lo < 0x7f80u) top = max(top, lo);
                if (hi < 0x7f80u) top = max(top, hi);
            }
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = min(126, 13 + 127 - static_cast<int>(top >> 7));  // >= -114
        const float f = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);     // 2^e
        const float unit = p.unit * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // times 2^-e
        float sum[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const uint32_t w[4] = {qv[g].x, qv[g].y, qv[g].z, qv[g].w};
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = scale_of(w[i >> 1], i & 1) * f;
            // Nibbles n and n + 4 of a word share a register.
            qf[g][0] = pack_f16x2(x[0], x[4]);
            qf[g][1] = pack_f16x2(x[2], x[6]);
            qf[g][2] = pack_f16x2(x[1] * 0.0625f, x[5] * 0.0625f);
            qf[g][3] = pack_f16x2(x[3] * 0.0625f, x[7] * 0.0625f);
            float2 a[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = __half22float2(*reinterpret_cast<const __half2*>(&qf[g][i]));
            float t = (a[0].x + a[0].y) + (a[1].x + a[1].y) + 16.f * ((a[2].x + a[2].y) + (a[3].x + a[3].y));
            t += __shfl_xor_sync(0xffffffffu, t, 1);
            t += __shfl_xor_sync(0xffffffffu, t, 2);
            sum[g] = -8.f * kCode * t;
        }
        // Row k = NG part + g of that operand: part 0, 1 or 2 of group g's sum. A
        // lane holds rows 2 c, 2 c + 1 and 2 c + 8, 2 c + 9 of head r.
        float part[3][NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            part[0][g] = __bfloat162float(__float2bfloat16_rn(sum[g]));
            part[1][g] = __bfloat162float(__float2bfloat16_rn(sum[g] - part[0][g]));
            part[2][g] = sum[g] - part[0][g] - part[1][g];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            // (As words: selected one by one, d = 64 kept them in local memory, in the same time.)
            uint32_t v = 0;
#pragma unroll
            for (int k = 0; k < 3 * NG; k += 2) {
                const uint32_t two = pack_bf16x2(part[k / NG][k % NG], part[(k + 1) / NG][(k + 1) % NG]);
                v = k / 2 == c + 4 * i ? two : v;
            }
            start[i] = v;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) qs[h] = __shfl_sync(0xffffffffu, unit, 4 * (2 * c + h));
    }

    const float NEG = -INFINITY;
    float acc[2 * NG][4];  // [group][values 4 r + 0, 1 | 2, 3], of heads 2 c and 2 c + 1
    float off[NG][4];      // 8 sum P s
#pragma unroll
    for (int i = 0; i < 2 * NG; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
#pragma unroll
    for (int g = 0; g < NG; ++g) off[g][0] = off[g][1] = off[g][2] = off[g][3] = 0.f;
    auto rescale = [&](float f0, float f1) {
#pragma unroll
        for (int k = 0; k < 2 * NG; ++k) {
            acc[k][0] *= f0;
            acc[k][1] *= f1;
            acc[k][2] *= f0;
            acc[k][3] *= f1;
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            off[g][0] *= f0;
            off[g][1] *= f1;
            off[g][2] *= f0;
            off[g][3] *= f1;
        }
    };
    // The reference of the softmax follows a head's largest logit only once one
    // is more than kGrowth above it: weights up to 2^kGrowth serve as well, and
    // most tiles need no maximum across the lanes.
    constexpr float kGrowth = 8.f;
    float m0 = NEG, m1 = NEG, base0 = 0.f, base1 = 0.f, l0 = 0.f, l1 = 0.f;
    // P s is held as halves of p s 2^(6 - E), 2^E the power of two of the largest
    // scale so far: below 2^15, 11 bits down to 2^-20 of the largest possible
    // value, and nothing below 2^-31 of it.
    constexpr int kHalfExp = 6;
    uint32_t E = 20;
    float fE = __uint_as_float((kHalfExp + 254 - 20) << 23);

    float* const k_wide = reinterpret_cast<float*>(ring + R::kKWideOff);
    float* const v_wide = reinterpret_cast<float*>(ring + R::kVWideOff);
    // A lane widens the scales of its row of the tile once for all that read them.
    auto widen = [&](const uint32_t (&w)[NG / 2], float f, float* to) {
        float v[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) v[g] = scale_of(w[g >> 1], g & 1) * f;
        if constexpr (NG == 4)
            reinterpret_cast<float4*>(to)[lane] = make_float4(v[0], v[1], v[2], v[3]);
        else
            reinterpret_cast<float2*>(to)[lane] = make_float2(v[0], v[1]);
    };
    auto wide = [&](const float* from, int row, float (&v)[NG]) {
        if constexpr (NG == 4) {
            const float4 x = reinterpret_cast<const float4*>(from)[row];
            v[0] = x.x;
            v[1] = x.y;
            v[2] = x.z;
            v[3] = x.w;
        } else {
            const float2 x = reinterpret_cast<const float2*>(from)[row];
            v[0] = x.x;
            v[1] = x.y;
        }
    };
    // Waits for tile i of the list, puts the token's row in its place there and
    // widens the keys' scales.
    auto arrive = [&](int i, uint8_t* tile) {
        copy_wait<R::kStages - 2>();
        __syncwarp();
        if (mine && static_cast<int>(s_tiles[warp][i].y) == wi / kTileSlots) {
            const int row = wi % kTileSlots;
            if (lane < D / 32)
                reinterpret_cast<uint4*>(tile + row * R::kKRow)[lane] = reinterpret_cast<const uint4*>(s_new[0])[lane];
            else if (lane < D / 16)
                reinterpret_cast<uint4*>(tile + R::kVOff + row * R::kVRow)[lane - D / 32] =
                    reinterpret_cast<const uint4*>(s_new[1])[lane - D / 32];
            else if (lane < D / 16 + 2 * NG) {
                const int g = (lane - D / 16) % NG, is_v = (lane - D / 16) / NG;
                reinterpret_cast<__nv_bfloat16*>(tile + (is_v ? R::kVScaleOff : R::kKScaleOff) +
                                                 row * R::kScaleRow)[g] = s_new_scale[is_v][g];
            }
            __syncwarp();
        }
        uint32_t ks[NG / 2];
        shared_words<NG / 2>(tile + R::kKScaleOff + lane * R::kScaleRow, ks);
        widen(ks, 1.f, k_wide);
        __syncwarp();
    };
    // Logits of the tile's slots r + 8 h: x[2 h] and x[2 h + 1], heads 2 c and 2 c + 1.
    float x[8];
    auto logits = [&](const uint8_t* tile) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t kw[2][NG], kz[2];
            float ks[2][NG];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = r + 8 * h + 16 * half;
                shared_words<NG>(tile + row * R::kKRow + c * (D / 8), kw[h]);
                wide(k_wide, row, ks[h]);
                kz[h] = *reinterpret_cast<const uint32_t*>(tile + R::kKScaleOff + row * R::kScaleRow +
                                                           c % (NG / 2) * 4);
            }
            const float zero[4] = {0.f, 0.f, 0.f, 0.f};
            float y[4] = {0.f, 0.f, 0.f, 0.f};
            const uint32_t z[4] = {kz[0], kz[1], kz[0], kz[1]};
            mma_bf16_16816(y, z, start[0], start[1]);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                float sc[4];
                const uint32_t a[4] = {kw[0][g] & 0x000f000fu, kw[1][g] & 0x000f000fu,
                                       (kw[0][g] >> 8) & 0x000f000fu, (kw[1][g] >> 8) & 0x000f000fu};
                mma_f16_16816(sc, a, qf[g][0], qf[g][1], zero);
                const uint32_t o[4] = {kw[0][g] & 0x00f000f0u, kw[1][g] & 0x00f000f0u,
                                       (kw[0][g] >> 8) & 0x00f000f0u, (kw[1][g] >> 8) & 0x00f000f0u};
                mma_f16_16816(sc, o, qf[g][2], qf[g][3], sc);
                y[0] += sc[0] * ks[0][g];
                y[1] += sc[1] * ks[0][g];
                y[2] += sc[2] * ks[1][g];
                y[3] += sc[3] * ks[1][g];
            }
            x[4 * half] = y[0] * qs[0];
            x[4 * half + 1] = y[1] * qs[1];
            x[4 * half + 2] = y[2] * qs[0];
            x[4 * half + 3] = y[3] * qs[1];
        }
    };

    uint8_t* tile = ring;
    int stage = 0;
    if (tiles > 0) {
        arrive(0, tile);
        logits(tile);
    }
    // The weights and values of tile i, the next tile's logits beside them.
    const auto step = [&](int i, auto last) {
        const uint32_t live = s_tiles[warp][i].x;
        uint32_t vs[NG / 2];  // of the lane's row
        shared_words<NG / 2>(tile + R::kVScaleOff + lane * R::kScaleRow, vs);
        if (live != 0xffffffffu) {
            // Masked slots: weight 0, and 0 for the scales of whatever lies there.
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const bool is = (live >> (r + 8 * h)) & 1u;
                x[2 * h] = is ? x[2 * h] : NEG;
                x[2 * h + 1] = is ? x[2 * h + 1] : NEG;
            }
#pragma unroll
            for (int k = 0; k < NG / 2; ++k) vs[k] = (live >> lane) & 1u ? vs[k] : 0u;
        }
        float mx0 = fmaxf(fmaxf(x[0], x[2]), fmaxf(x[4], x[6]));
        float mx1 = fmaxf(fmaxf(x[1], x[3]), fmaxf(x[5], x[7]));
        if (__any_sync(0xffffffffu, mx0 > m0 + kGrowth || mx1 > m1 + kGrowth)) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
                mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
            }
            mx0 = fmaxf(mx0, m0);
            mx1 = fmaxf(mx1, m1);
            base0 = mx0 == NEG ? 0.f : mx0;
            base1 = mx1 == NEG ? 0.f : mx1;
            const float f0 = ex2_approx(m0 - base0), f1 = ex2_approx(m1 - base1);
            l0 *= f0;
            l1 *= f1;
            m0 = mx0;
            m1 = mx1;
            rescale(f0, f1);
        }
        // The largest scale, as the bits of two bf16 side by side.
        const uint32_t two = __vimax3_u16x2(vs[0], vs[NG / 2 - 1], 0u);
        if (__any_sync(0xffffffffu, max(two & 0xffffu, two >> 16) >= (E + 1) << 7)) {
            // Rare: a new power of two, of the finite ones.
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < NG / 2; ++k) {
                const uint32_t lo = vs[k] & 0x7f80u, hi = (vs[k] >> 16) & 0x7f80u;
                if (lo != 0x7f80u) top = max(top, lo);
                if (hi != 0x7f80u) top = max(top, hi);
            }
            top = __reduce_max_sync(0xffffffffu, top) >> 7;
            if (top > E) {
                const float down = __uint_as_float(static_cast<uint32_t>(max(0, 127 - static_cast<int>(top - E))) << 23);
                rescale(down, down);
                E = top;
                fE = __uint_as_float((kHalfExp + 254 - E) << 23);
            }
        }
        widen(vs, fE, v_wide);
        // The weights; the sums take them unrounded.
        float f[8];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            f[2 * h] = ex2_approx(x[2 * h] - base0);
            f[2 * h + 1] = ex2_approx(x[2 * h + 1] - base1);
        }
        l0 += (f[0] + f[2]) + (f[4] + f[6]);
        l1 += (f[1] + f[3]) + (f[5] + f[7]);
        // Two chains of products to keep the pipes busy.
        const int next_stage = stage + 1 == R::kStages ? 0 : stage + 1;
        uint8_t* const next = ring + next_stage * R::kStage;
        if constexpr (!last.value) {
            arrive(i + 1, next);
            logits(next);
        } else {
            __syncwarp();
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t vw[4][NG / 2];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                shared_words<NG / 2>(tile + R::kVOff + (16 * half + 2 * c + (k & 1) + 8 * (k >> 1)) * R::kVRow +
                                         r * (D / 16),
                                     vw[k]);
            const float* const fh = f + 4 * half;
            float sa[NG], sb[NG];
            wide(v_wide, 16 * half + r, sa);
            wide(v_wide, 16 * half + r + 8, sb);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const uint32_t b0 = movmatrix_trans(pack_f16x2(fh[0] * sa[g], fh[1] * sa[g]));
                const uint32_t b1 = movmatrix_trans(pack_f16x2(fh[2] * sb[g], fh[3] * sb[g]));
                // Slots 2 c and 2 c + 1 side by side: the lane's four codes of group g.
                const uint32_t pick = g & 1 ? 0x7632u : 0x5410u;
                const uint32_t ya = __byte_perm(vw[0][g >> 1], vw[1][g >> 1], pick);
                const uint32_t yb = __byte_perm(vw[2][g >> 1], vw[3][g >> 1], pick);
                const uint32_t lo[4] = {ya & 0x000f000fu, ya & 0x00f000f0u, yb & 0x000f000fu, yb & 0x00f000f0u};
                mma_f16_16816(acc[2 * g], lo, b0, b1, acc[2 * g]);
                const uint32_t za = ya >> 8, zb = yb >> 8;
                const uint32_t hi[4] = {za & 0x000f000fu, za & 0x00f000f0u, zb & 0x000f000fu, zb & 0x00f000f0u};
                mma_f16_16816(acc[2 * g + 1], hi, b0, b1, acc[2 * g + 1]);
                const uint32_t eight[4] = {0x00080008u, 0x00800080u, 0x00080008u, 0x00800080u};
                mma_f16_16816(off[g], eight, b0, b1, off[g]);
            }
        }
        if constexpr (!last.value) {
            __syncwarp();
            if (i + R::kStages < tiles) copy_tile(s_tiles[warp][i + R::kStages].y, stage);
            copy_commit();
            stage = next_stage;
            tile = next;
        }
    };
#pragma unroll 1
    for (int i = 0; i + 1 < tiles; ++i) step(i, std::false_type());
    if (tiles > 0) step(tiles - 1, std::true_type());

    // The four warps' states, joined (each warp's part of O over its ring).
    copy_wait<0>();
    __syncwarp();
    constexpr int kORow = D + 4;
    static_assert(G * kORow * 4 <= R::kWarp, "a warp's part of O exceeds its ring");
    float* const my_o = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, o);
        l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
    const int h0 = 2 * c;
    if (r == 0) {
        if (h0 < G) { s_m[warp][h0] = m0; s_l[warp][h0] = l0; }
        if (h0 + 1 < G) { s_m[warp][h0 + 1] = m1; s_l[warp][h0 + 1] = l1; }
    }
    {
        const float back = __uint_as_float((E - kHalfExp) << 23);  // 2^(E - 127 - kHalfExp)
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int dd = 32 * g + 4 * r + 2 * k;
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = (acc[2 * g + k][e] - off[g][e]) * (e < 2 ? 0x1p24f : 0x1p20f) * back;
                if (h0 < G) { my_o[h0 * kORow + dd] = v[0]; my_o[h0 * kORow + dd + 1] = v[2]; }
                if (h0 + 1 < G) { my_o[(h0 + 1) * kORow + dd] = v[1]; my_o[(h0 + 1) * kORow + dd + 1] = v[3]; }
            }
    }
    __syncthreads();
    const size_t part = static_cast<size_t>(u) * gridDim.x + blockIdx.x;
    for (int e = tid; e < G * D; e += kThreads) {
        const int h = e / D, dd = e % D;
        float mh = NEG;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mh = fmaxf(mh, s_m[w][h]);
        float o = 0.f, l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            // A warp without a live slot has l = 0 (with one, l is NaN or > 0).
            if (s_l[w][h] == 0.f) continue;
            const float f = exp2f(s_m[w][h] - (mh == NEG ? 0.f : mh));
            o += reinterpret_cast<const float*>(s_ring + w * R::kWarp)[h * kORow + dd] * f;
            l += s_l[w][h] * f;
        }
        if (gridDim.x == 1) {
            p.out[(row0 + h) * D + dd] = __float2bfloat16_rn(l == 0.f ? 0.f : o / l);
        } else {
            p.part_o[part * G * D + e] = o;
            if (dd == 0) p.part_ml[part * G + h] = make_float2(mh, l);
        }
    }
}

// The chunks of a query row joined by one CTA: its warps share the chunks, whose
// loads are in flight eight at a time. (43 chunks of 32 rows: some 2 us of 13.)
template <int D>
__global__ void __launch_bounds__(kThreads) lf_kv4_join_kernel(const Kv4Params p, int G, int nchunk) {
    __shared__ float s_o[kWarps][D];
    __shared__ float s_l[kWarps];
    allow_dependent_launch();
    grid_dependency_wait();
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x;
    const int u = row / G, h = row % G;
    const float2* ml = p.part_ml + static_cast<size_t>(u) * nchunk * G + h;
    const float* po = p.part_o + (static_cast<size_t>(u) * nchunk * G + h) * D;
    constexpr int kE = D / 32;  // values of a lane
    constexpr int kAhead = 8;
    float2 v[kAhead];
    float x[kAhead][kE];
    const auto load = [&](int k0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int k = k0 + i * kWarps;
            v[i] = k < nchunk ? __ldcg(ml + static_cast<size_t>(k) * G) : make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < kE; ++e)
                x[i][e] = k < nchunk ? __ldcg(po + static_cast<size_t>(k) * G * D + e * 32 + lane) : 0.f;
        }
    };
    load(warp);  // in flight with the maximum's loads
    float m = -INFINITY;
    for (int k = lane; k < nchunk; k += 32) m = fmaxf(m, __ldcg(&ml[static_cast<size_t>(k) * G].x));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m == -INFINITY) m = 0.f;
    float o[kE], l = 0.f;
#pragma unroll
    for (int e = 0; e < kE; ++e) o[e] = 0.f;
    for (int k0 = warp;;) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            // A chunk without a live slot has l = 0, its output is not there.
            if (v[i].y == 0.f) continue;
            const float f = exp2f(v[i].x - m);
            l += v[i].y * f;
#pragma unroll
            for (int e = 0; e < kE; ++e) o[e] += x[i][e] * f;
        }
        k0 += kWarps * kAhead;
        if (k0 >= nchunk) break;
        load(k0);
    }
#pragma unroll
    for (int e = 0; e < kE; ++e) s_o[warp][e * 32 + lane] = o[e];
    if (lane == 0) s_l[warp] = l;
    __syncthreads();
    const int dd = threadIdx.x;
    if (dd < D) {
        float sum = 0.f, all = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            sum += s_o[w][dd];
            all += s_l[w];
        }
        p.out[static_cast<size_t>(row) * D + dd] = __float2bfloat16_rn(all == 0.f ? 0.f : sum / all);
    }
}

// Launch configuration with programmatic dependent launch (LF_PDL=0: without).
struct Config {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    Config(dim3 grid, int threads, cudaStream_t stream) {
        const char* env = std::getenv("LF_PDL");
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = grid;
        cfg.blockDim = dim3(threads);
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = (env && std::atoi(env) == 0) ? 0 : 1;
    }
};

template <int D, int G>
cudaError_t launch_kv4_dg(const Kv4Params& p, int units, int nchunk, cudaStream_t stream) {
    constexpr auto kernel = lf_kv4_attn_kernel<D, G>;
    const cudaError_t e = allow_shared<kernel>(Ring<D>::kAlloc);
    if (e != cudaSuccess) return e;
    Config c(dim3(nchunk, units), kThreads, stream);
    c.cfg.dynamicSmemBytes = Ring<D>::kAlloc;
    return cudaLaunchKernelEx(&c.cfg, kernel, p);
}

template <int D>
cudaError_t launch_kv4_d(int G, const Kv4Params& p, int units, int nchunk, cudaStream_t stream) {
    cudaError_t e = cudaErrorInvalidValue;
    if (G == 1) e = launch_kv4_dg<D, 1>(p, units, nchunk, stream);
    if (G == 2) e = launch_kv4_dg<D, 2>(p, units, nchunk, stream);
    if (G == 4) e = launch_kv4_dg<D, 4>(p, units, nchunk, stream);
    if (G == 8) e = launch_kv4_dg<D, 8>(p, units, nchunk, stream);
    if (e != cudaSuccess || nchunk == 1) return e;
    Config j(dim3(units * G), kThreads, stream);
    return cudaLaunchKernelEx(&j.cfg, lf_kv4_join_kernel<D>, p, G, nchunk);
}

}  // namespace

Kv4Plan kv4_plan(int units, int S, int sms) {
    // Three CTAs are resident per SM; chunks of whole 128 slots (32 a warp).
    // Up to 512 slots: one chunk, which needs no join (8 units, us in one chunk: 128
    // slots 5.2, 256 6.0, 512 7.8; in chunks of 128 and joined, 640 slots 7.1).
    const int steps = (S + 127) / 128;
    const int longest = kMaxChunkSlots / 128;
    const int fill = steps <= 4 ? 1 : std::max(1, 3 * sms / units);
    const int n = std::max((steps + longest - 1) / longest, std::min(steps, fill));
    const int per = (steps + n - 1) / n;
    // One chunk too where an SM's three CTAs would do no less of a unit between them
    // (152 units, d = 64, us: 1024 slots 7.8 in one chunk, 9.4 in three; 640 slots 6.2
    // and 8.1 in three; 104 units of 1500 slots 9.7 in one and 9.2 in four).
    if (steps <= longest && (units + sms - 1) / sms * steps <= 3 * per) return Kv4Plan{steps * 128, 1};
    return Kv4Plan{per * 128, (steps + per - 1) / per};
}

cudaError_t launch_kv4_attention(int D, int G, const Kv4Params& p, int units, int nchunk,
                                 cudaStream_t stream) {
    if (D == 64) return launch_kv4_d<64>(G, p, units, nchunk, stream);
    if (D == 128) return launch_kv4_d<128>(G, p, units, nchunk, stream);
    return cudaErrorInvalidValue;
}

cudaError_t launch_kv4_pack(int D, bool unpack, const Kv4PackParams& p, int units, cudaStream_t stream) {
    Config c(dim3((p.P + kPackSlots - 1) / kPackSlots, units), kPackThreads, stream);
    if (D == 64)
        return unpack ? cudaLaunchKernelEx(&c.cfg, lf_kv4_unpack_kernel<64>, p)
                      : cudaLaunchKernelEx(&c.cfg, lf_kv4_pack_kernel<64>, p);
    if (D == 128)
        return unpack ? cudaLaunchKernelEx(&c.cfg, lf_kv4_unpack_kernel<128>, p)
                      : cudaLaunchKernelEx(&c.cfg, lf_kv4_pack_kernel<128>, p);
    return cudaErrorInvalidValue;
}

}  // namespace lf
