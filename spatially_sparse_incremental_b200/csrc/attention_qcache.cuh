// Parameters of the attention step over a quantised key / value cache, shared
// by its kernels.
#pragma once

#include "qcache.cuh"

namespace sige {

// Sums of weighted values are kept before they are divided by the sum of the
// weights, so they are larger than the result: by the weights' sum (up to the
// number of keys) and by how far a weight's exponent base lies below the row's
// maximum.  Value scales below kBigScale leave room for both: 2^49 (448 times the
// scale) x 2^40 (the tensor-core kernel's base) x 2^31 keys < 2^128.  A chunk of
// keys with a larger one has its base 2^kRoom above the maximum, so that weights
// are at most 2^-kRoom and any finite value summed over any number of keys stays
// finite.
constexpr float kBigScale = 1099511627776.0f;   // 2^40
constexpr float kRoom = 32.0f;

struct AttnQParams {
    const __nv_bfloat16 *q;      // [N][H][W][D]
    __nv_bfloat16 *o;            // [N][H][W][Dv]
    const uint8_t *kc, *vc;      // codes [N][keys][D], [N][keys][Dv]
    const float *ks, *vs;        // scales [N][keys][D / group], [N][keys][Dv / group]
    const int32_t *key_counts;   // [N] or NULL: every key
    const int32_t *idx, *count;  // tile list, or idx == NULL: every pixel
    int32_t cap, b;
    int32_t N, H, W, D, Dv, keys, heads, dh, dvh;
    int32_t kfmt, vfmt;
    int32_t kng, vng;            // scales of a key, of a value
    int32_t kgroup, vgroup;
    int64_t slots;               // most query slots of a batch item
    float scale;                 // 1 / sqrt(dh)
    UDiv dbb, db;
    WsHeader *hdr;
};

// Query slots of one batch item on the device.
__device__ __forceinline__ int query_slots(const AttnQParams &p)
{
    return p.idx ? max(0, min(__ldg(p.count), p.cap)) * p.b * p.b : p.H * p.W;
}

// The flat pixel (n H + y) W + x of query slot s (below query_slots) of item
// n, -1 for a pixel outside the map.
__device__ __forceinline__ int64_t query_pixel(const AttnQParams &p, int n, int s)
{
    if (!p.idx)
        return (int64_t)n * p.H * p.W + s;
    const uint32_t t = udiv((uint32_t)s, p.dbb), w = (uint32_t)s - t * (uint32_t)(p.b * p.b);
    const uint32_t dy = udiv(w, p.db), dx = w - dy * (uint32_t)p.b;
    const int2 org = __ldg(reinterpret_cast<const int2 *>(p.idx) + t);
    if (org.x < 0 || org.y < 0 || org.x >= p.H || org.y >= p.W)
        return -1;
    if ((int)dy >= p.H - org.x || (int)dx >= p.W - org.y)   // (a sum may leave 32 bits)
        return -1;
    return ((int64_t)n * p.H + org.x + (int)dy) * p.W + org.y + (int)dx;
}

__device__ __forceinline__ int key_count(const AttnQParams &p, int n)
{
    return p.key_counts ? max(0, min(__ldg(p.key_counts + n), p.keys)) : p.keys;
}

// The tensor-core kernel: a sige_status, or 1 when the call is outside its
// scope.
int launch_attention_qcache_tc(const AttnQParams &p, cudaStream_t stream);
bool attention_qcache_tc_scope(int dh, int dvh);

} // namespace sige
