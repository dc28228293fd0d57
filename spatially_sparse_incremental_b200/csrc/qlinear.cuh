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

// One output before its rounding: the exact integer sum (rounded to float32,
// 2^-24), the token's scale, the channel's scale, then bias and residual.  The
// two scales are applied one after the other: their product alone may leave
// float32's range where the value does not.
__device__ __forceinline__ float qlinear_value(int acc, float sa, float sw) { return __int2float_rn(acc) * sa * sw; }

// The kernels (qlinear_tc.cu): a sige_status.
int launch_qlinear(const QLinearParams &p, cudaStream_t stream);
// Channels whose operands TMA copies (from 16-byte aligned codes).
bool qlinear_tma_scope(int c);

} // namespace sige
