// Product of 8-bit integers with a scale for each token and each output
// channel: y[t][o] = round(sa[t] * sw[o] * sum_c a[t][c] w[o][c] + bias[o] +
// residual[t][o]) at the tokens under the listed tiles or at every token.  It
// is the 1x1 layer F_l of the sparse engine (SIGE project page, "Overview") on
// a quantised cache.
//
// This file holds the call and its checks; the kernels are in qlinear_tc.cu.
#include "qlinear.cuh"

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
    // (and channels are counted in 32 bits, up to a tile past the last)
    if (ad->c > 131071 || wd->n > INT32_MAX - 1024)
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
    if (list_overlaps(y, ybytes, idx, count, capacity) || ranges_overlap(y, ybytes, workspace, kWsHeader))
        return SIGE_ERR_INVALID_ARG;
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
    return launch_qlinear(p, (cudaStream_t)stream);
}

extern "C" int sige_qlinear_path(int32_t c) { return c > 0 && qlinear_tma_scope(c) ? 1 : 0; }
