// Parameters of the product of 8-bit integers, shared by its kernels.
#pragma once

#include "qcache.cuh"

namespace sige {

struct QLinearParams {
    PixelList px;            // the tokens
    const uint8_t *a;        // [tokens][C] signed codes
    const float *sa;         // [tokens]
    const uint8_t *w;        // [Co][C] signed codes
    const float *sw;         // [Co]
    const float *bias;       // [Co] or NULL
    const uint8_t *residual; // [tokens][Co] in y's dtype, or NULL
    uint8_t *y;              // [tokens][Co]
    int32_t C, Co, dtype;
    int64_t rows;            // tokens of the whole map
    int64_t slots;           // most token slots the call can cover
    WsHeader *hdr;
};

// One output before its residual and rounding: the exact integer sum (rounded to
// float32, 2^-24), the token's scale, the channel's scale, then the bias.  The two
// scales are applied one after the other: their product alone may leave float32's
// range where the value does not.  So may the sum (below 2^31) times a token scale
// above 2^96 (is_big): 2^64 of such a scale come last.
struct TokenScale {
    float first, last;
};
__device__ __forceinline__ bool is_big(float sa) { return fabsf(sa) > 0x1p96f; }
__device__ __forceinline__ TokenScale token_scale(float sa)
{
    const bool big = is_big(sa);
    return TokenScale{big ? sa * 0x1p-64f : sa, big ? 0x1p64f : 1.0f};
}
__device__ __forceinline__ float qlinear_value(int acc, TokenScale sa, float sw, float bias)
{
    return fmaf(__int2float_rn(acc) * sa.first * sw, sa.last, bias);
}

// The kernels (qlinear_tc.cu): a sige_status.
int launch_qlinear(const QLinearParams &p, cudaStream_t stream);
// Channels whose operands TMA copies (from 16-byte aligned codes).
bool qlinear_tma_scope(int c);

} // namespace sige
