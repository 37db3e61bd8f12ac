// mma_tile.cuh -- pieces of the warp-MMA kernels: the m16n8k16 instruction, and
// the loads and the rebuild of one lane's weights of a 16-row tile in fragment
// order (plain BF16 or compressed planes).
#pragma once
#include "device_common.cuh"
#include "uw_format.h"

namespace uw {
namespace dev {

// One lane's 16*Q weights of one chunk (64*Q weights along K) of one row, as
// loaded.  Plain: the weights, 16*Q BF16 in a[] then b[].  Fused: sign/mantissa
// bytes in a[]; the palette words (2*Q of them) in b[0], or the raw
// exponents (16*Q bytes) in b[].
template <int Q>
struct Half {
    uint4 a[Q];
    uint4 b[Q];
};

__device__ __forceinline__ void prefetch_l1(const void *p) {
    asm volatile("prefetch.global.L1 [%0];" ::"l"(p));
}

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// raw bits of the 64 groups starting at global group `gfirst` (bit i = group
// gfirst + i) from the staged bitmap (word index relative to `wbase`); words
// past the staged ones read as 0, and bits beyond the caller's chunks are
// never used
__device__ __forceinline__ uint64_t raw_window(const uint32_t *sflags, int nwords, int64_t wbase, int64_t gfirst) {
    const int64_t w = (gfirst >> 5) - wbase;
    const uint32_t sh = uint32_t(gfirst) & 31u;
    uint32_t v[3];
#pragma unroll
    for (int q = 0; q < 3; q++) v[q] = (w + q < nwords) ? sflags[w + q] : 0u;
    const uint64_t lo = (uint64_t(v[1]) << 32 | v[0]) >> sh;
    const uint64_t hi = uint64_t(v[2]) << (64 - sh);   // sh = 0: shift by 64 is avoided below
    return sh ? (lo | hi) : (uint64_t(v[1]) << 32 | v[0]);
}

// loads of one lane's weights of one chunk of one row; `g` is the lane's
// group, `goff` the lane's byte offset inside that group's 64 raw exponents
template <bool PAL, int Q>
__device__ __forceinline__ Half<Q> load_half(const uint8_t *rawexp, const uint8_t *smp, const uint32_t *palp,
                                             const uint16_t *wp, bool raw, int64_t g, int goff,
                                             const uint32_t *sflags, const uint32_t *srb, int64_t wbase) {
    Half<Q> h;
    if (!PAL) {
        const uint4 *u = reinterpret_cast<const uint4 *>(wp);
#pragma unroll
        for (int i = 0; i < Q; i++) {
            h.a[i] = __ldcs(u + i);
            h.b[i] = __ldcs(u + Q + i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < Q; i++) h.a[i] = __ldcs(reinterpret_cast<const uint4 *>(smp) + i);
        if (raw) {
            const int wi = int((g >> 5) - wbase);
            const uint32_t rank = srb[wi] + __popc(sflags[wi] & ((1u << (uint32_t(g) & 31u)) - 1u));
            const uint4 *e = reinterpret_cast<const uint4 *>(rawexp + uint64_t(rank) * kGroup + goff);
#pragma unroll
            for (int i = 0; i < Q; i++) h.b[i] = __ldcs(e + i);
        } else if (Q == 1) {
            const uint2 p = __ldcs(reinterpret_cast<const uint2 *>(palp));
            h.b[0] = make_uint4(p.x, p.y, 0u, 0u);
        } else {
            h.b[0] = __ldcs(reinterpret_cast<const uint4 *>(palp));
#pragma unroll
            for (int i = 1; i < Q; i++) h.b[i] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    return h;
}

__device__ __forceinline__ uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Half -> 8*Q BF16 pairs (weights 2i, 2i+1 in pair i)
template <bool PAL, int Q>
__device__ __forceinline__ void rebuild(const Half<Q> &h, bool raw, const Palette16 &P, uint32_t (&w)[8 * Q]) {
    if (!PAL) {
#pragma unroll
        for (int i = 0; i < 4 * Q; i++) w[i] = word(h.a[i / 4], i % 4);
#pragma unroll
        for (int i = 0; i < 4 * Q; i++) w[4 * Q + i] = word(h.b[i / 4], i % 4);
    } else {
        uint32_t r[4 * Q];   // rotated exponent bytes, 4 weights per word
        if (raw) {
#pragma unroll
            for (int i = 0; i < 4 * Q; i++) r[i] = rot4(word(h.b[i / 4], i % 4));
        } else {
#pragma unroll
            for (int i = 0; i < 2 * Q; i++) pal_rot(word(h.b[0], i), P, r[2 * i], r[2 * i + 1]);
        }
#pragma unroll
        for (int i = 0; i < 4 * Q; i++) join4(r[i], word(h.a[i / 4], i % 4), w[2 * i], w[2 * i + 1]);
    }
}

}  // namespace dev
}  // namespace uw
