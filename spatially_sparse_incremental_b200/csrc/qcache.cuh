// Shared by the quantised cache and the operators that read it: the formats'
// code arithmetic, the list of pixels a call covers, and the host's checks.
#pragma once

#include <cuda_fp8.h>

#include "sige_internal.cuh"

namespace sige {

// ------------------------------------------------------------------ pixels

// The pixels of a call: those under the listed tiles (clipped to the map), or
// every pixel when idx is NULL.  Slot i of the listed form is pixel
// (i mod b^2) of tile (i / b^2) / N for batch item (i / b^2) mod N.
struct PixelList {
    const int32_t *idx, *count;
    int32_t cap, b, N, H, W;
    UDiv dbb, db, dN;
};

__device__ __forceinline__ int64_t pixel_slots(const PixelList &p)
{
    if (!p.idx)
        return (int64_t)p.N * p.H * p.W;
    return (int64_t)max(0, min(__ldg(p.count), p.cap)) * p.N * p.b * p.b;
}

// The flat pixel (n H + y) W + x of slot i, -1 for a clipped one.  Slots stay
// below 2^31 (checked on the host for the list's capacity).
__device__ __forceinline__ int64_t pixel_of(const PixelList &p, uint32_t i)
{
    if (!p.idx)
        return i;
    const uint32_t tn = udiv(i, p.dbb), w = i - tn * (uint32_t)(p.b * p.b);
    const uint32_t t = udiv(tn, p.dN), n = tn - t * (uint32_t)p.N;
    const uint32_t dy = udiv(w, p.db), dx = w - dy * (uint32_t)p.b;
    const int2 org = __ldg(reinterpret_cast<const int2 *>(p.idx) + t);
    if (org.x < 0 || org.y < 0 || org.x >= p.H || org.y >= p.W)
        return -1;
    if ((int)dy >= p.H - org.x || (int)dx >= p.W - org.y)   // (a sum may leave 32 bits)
        return -1;
    return ((int64_t)n * p.H + org.x + (int)dy) * p.W + org.y + (int)dx;
}

// Fills `p`; a sige_status.  *slots = the most pixels the call can cover.
int pixel_list_make(PixelList *p, int32_t N, int32_t H, int32_t W, int32_t block, const int32_t *idx,
                    const int32_t *count, int32_t capacity, int64_t *slots);

// ------------------------------------------------------------------ formats

constexpr float kMinScale = 1.1754943508222875e-38f;   // 2^-126: below it a group is stored as zeros

// The scale of a group whose largest magnitude has the bits `amax` (float32
// without the sign; an infinity or a NaN of the group is the largest of all).
// Integer formats: the float32 quotient amax / qmax.  e4m3 keeps three
// mantissa bits wherever a value lies, so a power of two loses nothing and
// makes every quotient exact: 2^ceil(log2(amax / 448)), 448 = 1.75 * 2^8.
template <int kFmt>
__device__ __forceinline__ float group_scale(uint32_t amax)
{
    if (amax >= 0x7F800000u)
        return __uint_as_float(0x7FC00000u);
    if constexpr (kFmt == SIGE_Q_E4M3) {
        const int e = (int)(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u);
        return e < 1 ? 0.0f : __uint_as_float((uint32_t)e << 23);
    } else {
        const float s = __fdiv_rn(__uint_as_float(amax), kFmt == SIGE_Q_S8 ? 127.0f : 7.0f);
        return s < kMinScale ? 0.0f : s;
    }
}

// What the quotient is formed with: the scale's reciprocal, 0 where the group
// stores zeros (scale 0 or NaN).  Exact for e4m3 (a power of two); for the
// integers within 2^-23 (an approximate reciprocal: the scale and its reciprocal
// are normal numbers).
template <int kFmt>
__device__ __forceinline__ float scale_reciprocal(float s)
{
    if constexpr (kFmt == SIGE_Q_E4M3) {
        return s > 0.0f ? __uint_as_float(0x7F000000u - __float_as_uint(s)) : 0.0f;
    } else {
        float r;
        asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(s));
        return s > 0.0f ? r : 0.0f;
    }
}

// round(v / s) to the nearest integer, ties to even, of the exact quotient.
// v * (1 / s) is off by at most 127.5 (2^-23 + 2^-24) < 2^-15 for |v / s| <=
// 127.5, so its nearest integer k is the right one or, next to a tie, its
// neighbour.  The remainder e = v - k s tells: it is exact in float32 (a
// multiple of half the scale's last bit, below 2^24 of them; above the smallest
// subnormal), and k stands unless 2 |e| > s, or 2 |e| = s with k odd.
constexpr float kRoundBase = 12582912.0f;   // 1.5 * 2^23: a sum's low bits are the rounded integer's
__device__ __forceinline__ float quotient_rest(float v, float s, float k) { return fmaf(-k, s, v); }
__device__ __forceinline__ int quotient_code(float v, float s, float r)
{
    const float k = rintf(v * r), e = quotient_rest(v, s, k), e2 = 2.0f * fabsf(e);
    int c = (int)k;
    if (e2 > s || (e2 == s && (c & 1)))
        c += e > 0.0f ? 1 : -1;
    return c;
}

// Four codes of an integer format from a 32-bit word (s8) or half a word (s4).
__device__ __forceinline__ float s8_value(uint32_t w, int k) { return (float)(int8_t)(w >> (8 * k)); }
__device__ __forceinline__ float s4_value(uint32_t w, int k) { return (float)((int)(w << (28 - 4 * k)) >> 28); }

__device__ __forceinline__ float e4m3_value(uint32_t byte)
{
    __nv_fp8_e4m3 v;
    v.__x = (__nv_fp8_storage_t)byte;
    return (float)v;
}

// The value of one code of any format; `i` is the element's index.
__device__ __forceinline__ float code_at(const uint8_t *codes, int64_t i, int fmt)
{
    if (fmt == SIGE_Q_S4)
        return s4_value(codes[i >> 1], (int)(i & 1));
    return fmt == SIGE_Q_S8 ? (float)(int8_t)codes[i] : e4m3_value(codes[i]);
}

// ------------------------------------------------------------------ host

// SIGE_OK when `d` describes a cache: positive sizes, a known format, a group
// that divides the channels (whole bytes of 4-bit codes), pixels in 32 bits.
int qcache_check(const sige_qcache_desc *d);
inline int64_t qcache_bytes(const sige_qcache_desc *d)
{
    const int64_t e = (int64_t)d->n * d->h * d->w * d->c;
    return d->format == SIGE_Q_S4 ? e / 2 : e;
}
inline int64_t qcache_scale_count(const sige_qcache_desc *d)
{
    return (int64_t)d->n * d->h * d->w * (d->c / d->group);
}
inline bool ranges_overlap(const void *a, int64_t na, const void *b, int64_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}
// Whether the tile list or its count lies in memory that the call writes.
inline bool list_overlaps(const void *a, int64_t na, const int32_t *idx, const int32_t *count, int32_t capacity)
{
    return idx && (ranges_overlap(a, na, idx, 8ll * capacity) || ranges_overlap(a, na, count, 4));
}
inline bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

} // namespace sige
