// Product of 8-bit integers with a scale for each token and each output
// channel: y[t][o] = round(sa[t] * sw[o] * sum_c a[t][c] w[o][c] + bias[o] +
// residual[t][o]) at the tokens under the listed tiles or at every token.  It
// is the 1x1 layer F_l of the sparse engine (SIGE project page, "Overview") on
// a quantised cache.
//
// This file holds the call and the kernel for shapes the tensor-core kernel
// does not take (channels that are not a multiple of 16, unaligned buffers):
// 64 tokens x 64 channels a CTA, operands staged 64 bytes of K at a time, four
// products an instruction (dp4a), 4 x 4 outputs a thread.
#include <algorithm>

#include "qlinear.cuh"

namespace sige {
namespace ql {

constexpr int kThreads = 256;
constexpr int kTile = 64;       // tokens, and channels, of a CTA's tile
constexpr int kWords = 16;      // 32-bit words of K staged at a time

// Four codes of a row from element k on, zero past the end.
__device__ __forceinline__ int load4(const uint8_t *row, int k, int C, bool words)
{
    if (words && k + 4 <= C)
        return *reinterpret_cast<const int *>(row + k);
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (k + j < C)
            w |= (uint32_t)row[k + j] << (8 * j);
    return (int)w;
}

__global__ void __launch_bounds__(kThreads) k_qlinear_any(const __grid_constant__ QLinearParams p, int words)
{
    __shared__ int As[kWords][kTile + 1], Ws[kWords][kTile + 1];
    __shared__ int64_t tok[kTile];
    pdl_wait();
    const int64_t slots = pixel_slots(p.px);
    const int nb = (p.Co + kTile - 1) / kTile;
    const int64_t units = (slots + kTile - 1) / kTile * nb;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll 1
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t s0 = u / nb * kTile;
        const int o0 = (int)(u % nb) * kTile;
        __syncthreads();   // the previous unit has finished with tok
        if (threadIdx.x < kTile)
            tok[threadIdx.x] = s0 + threadIdx.x < slots ? pixel_of(p.px, (uint32_t)(s0 + threadIdx.x)) : -1;
        int acc[4][4] = {};
#pragma unroll 1
        for (int k0 = 0; k0 < p.C; k0 += 4 * kWords) {
            __syncthreads();
#pragma unroll
            for (int e = threadIdx.x; e < kTile * kWords; e += kThreads) {
                const int r = e / kWords, j = e % kWords, k = k0 + 4 * j;
                As[j][r] = tok[r] >= 0 && k < p.C ? load4(p.a + tok[r] * p.C, k, p.C, words) : 0;
                Ws[j][r] = o0 + r < p.Co && k < p.C ? load4(p.w + (int64_t)(o0 + r) * p.C, k, p.C, words) : 0;
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kWords; ++j) {
                int a[4], w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[i] = As[j][ty + 16 * i];
                    w[i] = Ws[j][tx + 16 * i];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int o = 0; o < 4; ++o)
                        acc[i][o] = __dp4a(a[i], w[o], acc[i][o]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t t = tok[ty + 16 * i];
            if (t < 0)
                continue;
            const float sa = __ldg(p.sa + t);
#pragma unroll
            for (int o = 0; o < 4; ++o) {
                const int c = o0 + tx + 16 * o;
                if (c >= p.Co)
                    continue;
                const int64_t e = t * p.Co + c;
                float v = qlinear_value(acc[i][o], sa, __ldg(p.sw + c));
                if (p.bias)
                    v += __ldg(p.bias + c);
                if (p.dtype == SIGE_BF16) {
                    if (p.residual)
                        v += __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p.residual)[e]);
                    reinterpret_cast<__nv_bfloat16 *>(p.y)[e] = __float2bfloat16_rn(v);
                } else {
                    if (p.residual)
                        v += reinterpret_cast<const float *>(p.residual)[e];
                    reinterpret_cast<float *>(p.y)[e] = v;
                }
            }
        }
    }
}

static int launch_any(const QLinearParams &p, cudaStream_t stream)
{
    prefer_max_shared(k_qlinear_any);
    const int64_t units = (p.slots + kTile - 1) / kTile * ((p.Co + kTile - 1) / kTile);
    const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(units, (int64_t)device_sm_count() * 8));
    const int words = p.C % 4 == 0 && aligned_to(p.a, 4) && aligned_to(p.w, 4);
    if (launch_pdl(k_qlinear_any, dim3(grid), dim3(kThreads), 0, stream, p, words) != cudaSuccess) {
        cudaGetLastError();
        return SIGE_ERR_CUDA;
    }
    count_launch();
    return launch_check();
}

} // namespace ql
} // namespace sige

using namespace sige;

extern "C" int sige_qlinear(const void *a_codes, const float *a_scales, const sige_qcache_desc *ad,
                            const void *w_codes, const float *w_scales, const sige_qcache_desc *wd, const float *bias,
                            int32_t block, const int32_t *idx, const int32_t *count, int32_t capacity,
                            const void *residual, void *y, const sige_tensor_desc *yd, void *workspace,
                            size_t workspace_bytes, sige_stream_t stream)
{
    if (!a_codes || !a_scales || !w_codes || !w_scales || !y || !yd)
        return SIGE_ERR_INVALID_ARG;
    int st = qcache_check(ad);
    if (st == SIGE_OK)
        st = qcache_check(wd);
    if (st != SIGE_OK)
        return st;
    if (wd->h != 1 || wd->w != 1 || wd->c != ad->c || yd->n != ad->n || yd->h != ad->h || yd->w != ad->w ||
        yd->c != wd->n)
        return SIGE_ERR_INVALID_ARG;
    if (ad->format != SIGE_Q_S8 || wd->format != SIGE_Q_S8 || ad->group != ad->c || wd->group != wd->c)
        return SIGE_ERR_UNSUPPORTED;
    if ((yd->dtype != SIGE_BF16 && yd->dtype != SIGE_F32) || yd->layout != SIGE_NHWC)
        return SIGE_ERR_UNSUPPORTED;
    // a sum of 131071 products of magnitude 2^14 (codes of -128 included) stays in 32 bits
    if (ad->c > 131071)
        return SIGE_ERR_UNSUPPORTED;
    const int esz = yd->dtype == SIGE_BF16 ? 2 : 4;
    if (!aligned_to(a_scales, 4) || !aligned_to(w_scales, 4) || !aligned_to(bias, 4) || !aligned_to(y, esz) ||
        !aligned_to(residual, esz))
        return SIGE_ERR_INVALID_ARG;
    const int64_t rows = (int64_t)ad->n * ad->h * ad->w, ybytes = rows * yd->c * esz;
    // y is written while the operands are read
    if (ranges_overlap(y, ybytes, a_codes, qcache_bytes(ad)) || ranges_overlap(y, ybytes, a_scales, 4 * rows) ||
        ranges_overlap(y, ybytes, w_codes, qcache_bytes(wd)) || ranges_overlap(y, ybytes, w_scales, 4ll * wd->n) ||
        ranges_overlap(y, ybytes, bias, 4ll * wd->n) || ranges_overlap(y, ybytes, residual, ybytes))
        return SIGE_ERR_INVALID_ARG;
    QLinearParams p{};
    st = pixel_list_make(&p.px, ad->n, ad->h, ad->w, block, idx, count, capacity, &p.slots);
    if (st != SIGE_OK)
        return st;
    if (!workspace || workspace_bytes < kWsHeader || !aligned_to(workspace, 16))
        return SIGE_ERR_WORKSPACE;
    if (p.slots == 0)
        return SIGE_OK;
    p.a = static_cast<const uint8_t *>(a_codes);
    p.sa = a_scales;
    p.w = static_cast<const uint8_t *>(w_codes);
    p.sw = w_scales;
    p.bias = bias;
    p.residual = static_cast<const uint8_t *>(residual);
    p.y = static_cast<uint8_t *>(y);
    p.C = ad->c;
    p.Co = wd->n;
    p.dtype = yd->dtype;
    p.rows = rows;
    p.hdr = static_cast<WsHeader *>(workspace);
    const int tc = launch_qlinear_tc(p, (cudaStream_t)stream);
    return tc != 1 ? tc : ql::launch_any(p, (cudaStream_t)stream);
}

extern "C" int sige_qlinear_path(int32_t c) { return c > 0 && qlinear_tc_scope(c) ? 1 : 0; }
