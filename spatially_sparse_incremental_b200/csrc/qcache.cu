// The quantised activation cache: a map is written as 8- or 4-bit codes with
// one float32 scale per group of channels of a pixel, and read back, at the
// listed tiles or whole.  (mer.dev notes on SIGE, section 3 "Method" and
// section 4.2: the activations of the original are kept, for a diffusion model
// those of every step, which costs memory; the formats are this library's.)
//
// Both kernels are one pass over the data and bound by memory: a group's
// elements are loaded once into registers (16 bytes a lane), the largest
// magnitude is found among the lanes that share the group, and the codes leave
// from the same registers.
#include <algorithm>

#include "qcache.cuh"
#include "transform.cuh"

namespace sige {

int pixel_list_make(PixelList *p, int32_t N, int32_t H, int32_t W, int32_t block, const int32_t *idx,
                    const int32_t *count, int32_t capacity, int64_t *slots)
{
    p->idx = idx;
    p->count = count;
    p->N = N; p->H = H; p->W = W;
    p->cap = capacity;
    p->b = block;
    *slots = (int64_t)N * H * W;
    if (!idx) {
        p->b = 1;
    } else {
        if (!count || capacity < 0 || block < 1 || !aligned_to(idx, 8) || !aligned_to(count, 4))
            return SIGE_ERR_INVALID_ARG;
        if (block > 64)
            return SIGE_ERR_UNSUPPORTED;
        *slots = (int64_t)capacity * block * block;
        if (*slots > INT32_MAX || *slots * N > INT32_MAX)
            return SIGE_ERR_UNSUPPORTED;
        *slots *= N;
    }
    p->dbb = udiv_make((uint32_t)(p->b * p->b));
    p->db = udiv_make((uint32_t)p->b);
    p->dN = udiv_make((uint32_t)N);
    return SIGE_OK;
}

int qcache_check(const sige_qcache_desc *d)
{
    if (!d || d->n < 1 || d->h < 1 || d->w < 1 || d->c < 1 || d->group < 1 || d->c % d->group)
        return SIGE_ERR_INVALID_ARG;
    if (d->format != SIGE_Q_S8 && d->format != SIGE_Q_E4M3 && d->format != SIGE_Q_S4)
        return SIGE_ERR_INVALID_ARG;
    if (d->format == SIGE_Q_S4 && (d->group & 1))
        return SIGE_ERR_UNSUPPORTED;
    if ((int64_t)d->n * d->h > INT32_MAX || (int64_t)d->n * d->h * d->w > INT32_MAX)
        return SIGE_ERR_UNSUPPORTED;
    return SIGE_OK;
}

namespace qc {

constexpr int kThreads = 256;

struct Args {
    PixelList px;
    const uint8_t *x;      // map read (write call)
    uint8_t *y;            // map written (read call)
    uint8_t *codes;
    float *scales;
    const float *gsc, *gsh;
    int32_t silu;
    int32_t dtype, C, group, ng;
    int32_t lanes;         // lanes that share a group (write, vector form)
    int32_t vecs;          // 8-element vectors: of a group (write), of a pixel (read)
    UDiv dng, dvecs, dgv;  // groups of a pixel, vectors of a pixel, vectors of a group
    int32_t fast;          // every item index fits 32 bits
};

// item -> (slot, part) with `n` parts to a slot
__device__ __forceinline__ void split_item(int64_t item, int n, UDiv d, int fast, uint32_t *slot, int *part)
{
    if (fast) {
        const uint32_t q = udiv((uint32_t)item, d);
        *slot = q;
        *part = (int)((uint32_t)item - q * (uint32_t)n);
    } else {
        const int64_t q = item / n;
        *slot = (uint32_t)q;
        *part = (int)(item - q * n);
    }
}

__device__ __forceinline__ void load8(const Args &p, int64_t e, float (&v)[8])
{
    if (p.dtype == SIGE_BF16) {
        const uint4 r = ld_nc16(p.x + e * 2);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[2 * k] = bf16_lo(w[k]);
            v[2 * k + 1] = bf16_hi(w[k]);
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 r = ld_nc16(p.x + e * 4 + 16 * h);
            v[4 * h] = __uint_as_float(r.x);
            v[4 * h + 1] = __uint_as_float(r.y);
            v[4 * h + 2] = __uint_as_float(r.z);
            v[4 * h + 3] = __uint_as_float(r.w);
        }
    }
}

template <int kFmt>
__device__ __forceinline__ void store8(uint8_t *codes, int64_t e, const float (&v)[8], float s, float r)
{
    if constexpr (kFmt == SIGE_Q_E4M3) {
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * h] * r, v[4 * h + 1] * r), __NV_SATFINITE,
                                                         __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * h + 2] * r, v[4 * h + 3] * r),
                                                         __NV_SATFINITE, __NV_E4M3);
            w[h] = lo | (hi << 16);
        }
        *reinterpret_cast<uint2 *>(codes + e) = r > 0.0f ? make_uint2(w[0], w[1]) : make_uint2(0, 0);
    } else {
        uint32_t w[2] = {0, 0};
        if (r > 0.0f) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t c = (uint32_t)quotient_code(v[k], s, r);
                if constexpr (kFmt == SIGE_Q_S8)
                    w[k >> 2] |= (c & 255u) << (8 * (k & 3));
                else
                    w[0] |= (c & 15u) << (4 * k);
            }
        }
        if constexpr (kFmt == SIGE_Q_S8)
            *reinterpret_cast<uint2 *>(codes + e) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint32_t *>(codes + (e >> 1)) = w[0];
    }
}

// Write, vector form: `lanes` neighbouring lanes share one group, each with up
// to V vectors of 8 channels in registers.
template <int kFmt, int V>
__global__ void __launch_bounds__(kThreads) k_qcache_write(const __grid_constant__ Args p)
{
    pdl_wait();
    const int64_t items = pixel_slots(p.px) * p.ng;
    const int sub = threadIdx.x & (p.lanes - 1);
    const int per_block = kThreads / p.lanes;
    const int64_t step = (int64_t)gridDim.x * per_block;
    // whole warps leave the loop together: the shuffles below need every lane
    const int64_t first = (int64_t)blockIdx.x * per_block + (threadIdx.x & ~31) / p.lanes;
    const int mine = (threadIdx.x & 31) / p.lanes;
#pragma unroll 1
    for (int64_t base = first; base < items; base += step) {
        const int64_t item = base + mine;
        int64_t pix = -1;
        int g = 0;
        if (item < items) {
            uint32_t slot;
            split_item(item, p.ng, p.dng, p.fast, &slot, &g);
            pix = pixel_of(p.px, slot);
        }
        const int64_t e0 = pix * p.C + (int64_t)g * p.group;
        float v[V][8];
        uint32_t amax = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int vec = sub + j * p.lanes;
            if (pix >= 0 && vec < p.vecs)
                load8(p, e0 + 8 * vec, v[j]);
        }
        if (p.gsc || p.silu) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int vec = sub + j * p.lanes;
                if (pix >= 0 && vec < p.vecs) {
                    const int64_t n = pix / ((int64_t)p.px.H * p.px.W);
                    const int64_t c = n * p.C + g * p.group + 8 * vec;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        v[j][k] = transform1(v[j][k], p.gsc ? p.gsc + c : nullptr, p.gsc ? p.gsh + c : nullptr, k,
                                             p.silu);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int vec = sub + j * p.lanes;
            if (pix >= 0 && vec < p.vecs) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    amax = max(amax, __float_as_uint(v[j][k]) & 0x7FFFFFFFu);
            }
        }
        for (int o = p.lanes >> 1; o > 0; o >>= 1)
            amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
        if (pix < 0)
            continue;
        const float s = group_scale<kFmt>(amax), r = scale_reciprocal(s);
        if (sub == 0)
            p.scales[pix * p.ng + g] = s;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int vec = sub + j * p.lanes;
            if (vec < p.vecs)
                store8<kFmt>(p.codes, e0 + 8 * vec, v[j], s, r);
        }
    }
}

__device__ __forceinline__ float load1(const Args &p, int64_t e)
{
    if (p.dtype == SIGE_BF16)
        return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p.x)[e]);
    return reinterpret_cast<const float *>(p.x)[e];
}

// Write, any alignment and any group: a warp per group, the elements read
// twice (the second time from the caches).
template <int kFmt>
__global__ void __launch_bounds__(kThreads) k_qcache_write_any(const __grid_constant__ Args p)
{
    pdl_wait();
    const int64_t items = pixel_slots(p.px) * p.ng;
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
#pragma unroll 1
    for (int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); item < items; item += step) {
        uint32_t slot;
        int g;
        split_item(item, p.ng, p.dng, p.fast, &slot, &g);
        const int64_t pix = pixel_of(p.px, slot);
        if (pix < 0)
            continue;
        const int64_t e0 = pix * p.C + (int64_t)g * p.group;
        const int64_t c0 = pix / ((int64_t)p.px.H * p.px.W) * p.C + (int64_t)g * p.group;
        const float *sc = p.gsc ? p.gsc + c0 : nullptr, *sh = p.gsc ? p.gsh + c0 : nullptr;
        uint32_t amax = 0;
        for (int k = lane; k < p.group; k += 32)
            amax = max(amax, __float_as_uint(transform1(load1(p, e0 + k), sc, sh, k, p.silu)) & 0x7FFFFFFFu);
        amax = __reduce_max_sync(0xFFFFFFFFu, amax);
        const float s = group_scale<kFmt>(amax), r = scale_reciprocal(s);
        if (lane == 0)
            p.scales[pix * p.ng + g] = s;
        constexpr int kPer = kFmt == SIGE_Q_S4 ? 2 : 1;   // elements of a byte
        for (int k = kPer * lane; k < p.group; k += kPer * 32) {
            uint32_t byte = 0;
            if (r > 0.0f) {
                const float a = transform1(load1(p, e0 + k), sc, sh, k, p.silu);
                if constexpr (kFmt == SIGE_Q_E4M3)
                    byte = __nv_cvt_float_to_fp8(a * r, __NV_SATFINITE, __NV_E4M3);
                else
                    byte = (uint32_t)quotient_code(a, s, r) & (kFmt == SIGE_Q_S8 ? 255u : 15u);
                if constexpr (kFmt == SIGE_Q_S4)
                    byte |= ((uint32_t)quotient_code(transform1(load1(p, e0 + k + 1), sc, sh, k + 1, p.silu), s, r) &
                             15u) << 4;
            }
            p.codes[(e0 + k) / kPer] = (uint8_t)byte;
        }
    }
}

// Read, vector form: 8 codes of one group a thread.
template <int kFmt>
__global__ void __launch_bounds__(kThreads) k_qcache_read(const __grid_constant__ Args p)
{
    pdl_wait();
    const int64_t items = pixel_slots(p.px) * p.vecs;
    const int64_t step = (int64_t)gridDim.x * kThreads;
#pragma unroll 1
    for (int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x; item < items; item += step) {
        uint32_t slot;
        int vec;
        split_item(item, p.vecs, p.dvecs, p.fast, &slot, &vec);
        const int64_t pix = pixel_of(p.px, slot);
        if (pix < 0)
            continue;
        const int64_t e = pix * p.C + 8 * vec;
        const float s = __ldg(p.scales + pix * p.ng + udiv((uint32_t)vec, p.dgv));
        float v[8];
        if constexpr (kFmt == SIGE_Q_S4) {
            const uint32_t w = __ldg(reinterpret_cast<const uint32_t *>(p.codes + (e >> 1)));
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] = s4_value(w, k);
        } else {
            const uint2 w = __ldg(reinterpret_cast<const uint2 *>(p.codes + e));
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t u = k < 4 ? w.x : w.y;
                v[k] = kFmt == SIGE_Q_S8 ? s8_value(u, k & 3) : e4m3_value((u >> (8 * (k & 3))) & 255u);
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] *= s;
        if (p.dtype == SIGE_BF16) {
            *reinterpret_cast<uint4 *>(p.y + e * 2) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                                 pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
        } else {
            float4 *o = reinterpret_cast<float4 *>(p.y + e * 4);
            o[0] = make_float4(v[0], v[1], v[2], v[3]);
            o[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    }
}

// Read, any alignment and any group: one element a thread.
__global__ void __launch_bounds__(kThreads) k_qcache_read_any(const __grid_constant__ Args p, int fmt)
{
    pdl_wait();
    const int64_t items = pixel_slots(p.px) * p.C;
    const int64_t step = (int64_t)gridDim.x * kThreads;
#pragma unroll 1
    for (int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x; item < items; item += step) {
        uint32_t slot;
        int c;
        split_item(item, p.C, p.dvecs, p.fast, &slot, &c);
        const int64_t pix = pixel_of(p.px, slot);
        if (pix < 0)
            continue;
        const int64_t e = pix * p.C + c;
        const float v = code_at(p.codes, e, fmt) * __ldg(p.scales + pix * p.ng + c / p.group);
        if (p.dtype == SIGE_BF16)
            reinterpret_cast<__nv_bfloat16 *>(p.y)[e] = __float2bfloat16_rn(v);
        else
            reinterpret_cast<float *>(p.y)[e] = v;
    }
}

template <typename K, typename... A>
static int run(K kernel, int64_t items, int per_block, cudaStream_t stream, const A &...args)
{
    prefer_max_shared(kernel);
    const int64_t most = (int64_t)device_sm_count() * 32;
    const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>((items + per_block - 1) / per_block, most));
    if (launch_pdl(kernel, dim3(grid), dim3(kThreads), 0, stream, args...) != cudaSuccess) {
        cudaGetLastError();
        return SIGE_ERR_CUDA;
    }
    count_launch();
    return launch_check();
}

template <int kFmt>
static int run_write(Args &a, int64_t slots, bool vec, cudaStream_t stream)
{
    const int64_t items = slots * a.ng;
    a.fast = items <= INT32_MAX;
    if (!vec)
        return run(k_qcache_write_any<kFmt>, items, kThreads / 32, stream, a);
    a.vecs = a.group / 8;
    // as many lanes to a group as it has vectors (a power of two), a second
    // vector a lane before a ninth lane
    int V = 1;
    a.lanes = 1;
    while (a.lanes * V < a.vecs) {
        if (V == 1 && a.lanes == 8)
            V = 2;
        else if (a.lanes < 32)
            a.lanes *= 2;
        else
            V *= 2;
    }
    const int per_block = kThreads / a.lanes;
    switch (V) {
    case 1: return run(k_qcache_write<kFmt, 1>, items, per_block, stream, a);
    case 2: return run(k_qcache_write<kFmt, 2>, items, per_block, stream, a);
    case 4: return run(k_qcache_write<kFmt, 4>, items, per_block, stream, a);
    default: return run(k_qcache_write<kFmt, 8>, items, per_block, stream, a);
    }
}

// What the two calls check alike, and the arguments they share.
static int common(Args *a, const void *map, const sige_tensor_desc *md, const void *codes, const float *scales,
                  const sige_qcache_desc *cd, int32_t block, const int32_t *idx, const int32_t *count,
                  int32_t capacity, int64_t *slots, bool *vec)
{
    if (!map || !md || !codes || !scales)
        return SIGE_ERR_INVALID_ARG;
    int st = qcache_check(cd);
    if (st != SIGE_OK)
        return st;
    if (md->n != cd->n || md->h != cd->h || md->w != cd->w || md->c != cd->c)
        return SIGE_ERR_INVALID_ARG;
    if ((md->dtype != SIGE_BF16 && md->dtype != SIGE_F32) || md->layout != SIGE_NHWC)
        return SIGE_ERR_UNSUPPORTED;
    const int esz = md->dtype == SIGE_BF16 ? 2 : 4;
    if (!aligned_to(map, esz) || !aligned_to(scales, 4))
        return SIGE_ERR_INVALID_ARG;
    const int64_t elems = (int64_t)cd->n * cd->h * cd->w * cd->c;
    if (ranges_overlap(map, elems * esz, codes, qcache_bytes(cd)) ||
        ranges_overlap(map, elems * esz, scales, 4 * qcache_scale_count(cd)) ||
        ranges_overlap(codes, qcache_bytes(cd), scales, 4 * qcache_scale_count(cd)))
        return SIGE_ERR_INVALID_ARG;
    st = pixel_list_make(&a->px, cd->n, cd->h, cd->w, block, idx, count, capacity, slots);
    if (st != SIGE_OK)
        return st;
    a->codes = const_cast<uint8_t *>(static_cast<const uint8_t *>(codes));
    a->scales = const_cast<float *>(scales);
    a->dtype = md->dtype;
    a->C = cd->c;
    a->group = cd->group;
    a->ng = cd->c / cd->group;
    a->dng = udiv_make((uint32_t)a->ng);
    // 8 elements of a group from aligned addresses, a group in the registers of a warp
    *vec = cd->group % 8 == 0 && aligned_to(map, 16) && aligned_to(codes, cd->format == SIGE_Q_S4 ? 4 : 8);
    return SIGE_OK;
}

} // namespace qc
} // namespace sige

using namespace sige;

extern "C" size_t sige_qcache_code_bytes(const sige_qcache_desc *cd)
{
    return qcache_check(cd) == SIGE_OK ? (size_t)qcache_bytes(cd) : 0;
}

extern "C" size_t sige_qcache_scales(const sige_qcache_desc *cd)
{
    return qcache_check(cd) == SIGE_OK ? (size_t)qcache_scale_count(cd) : 0;
}

extern "C" int sige_qcache_write(const void *x, const sige_tensor_desc *xd, const float *gn_scale,
                                 const float *gn_shift, int32_t silu, int32_t block, const int32_t *idx,
                                 const int32_t *count, int32_t capacity, void *codes, float *scales,
                                 const sige_qcache_desc *cd, sige_stream_t stream)
{
    qc::Args a{};
    int64_t slots;
    bool vec;
    const int st = qc::common(&a, x, xd, codes, scales, cd, block, idx, count, capacity, &slots, &vec);
    if (st != SIGE_OK)
        return st;
    if ((gn_scale == nullptr) != (gn_shift == nullptr) || !aligned_to(gn_scale, 4) || !aligned_to(gn_shift, 4))
        return SIGE_ERR_INVALID_ARG;
    if (slots == 0)
        return SIGE_OK;
    a.x = static_cast<const uint8_t *>(x);
    a.gsc = gn_scale;
    a.gsh = gn_shift;
    a.silu = silu ? 1 : 0;
    vec = vec && cd->group <= 2048;
    switch (cd->format) {
    case SIGE_Q_S8: return qc::run_write<SIGE_Q_S8>(a, slots, vec, (cudaStream_t)stream);
    case SIGE_Q_E4M3: return qc::run_write<SIGE_Q_E4M3>(a, slots, vec, (cudaStream_t)stream);
    default: return qc::run_write<SIGE_Q_S4>(a, slots, vec, (cudaStream_t)stream);
    }
}

extern "C" int sige_qcache_read(const void *codes, const float *scales, const sige_qcache_desc *cd, int32_t block,
                                const int32_t *idx, const int32_t *count, int32_t capacity, void *y,
                                const sige_tensor_desc *yd, sige_stream_t stream)
{
    qc::Args a{};
    int64_t slots;
    bool vec;
    const int st = qc::common(&a, y, yd, codes, scales, cd, block, idx, count, capacity, &slots, &vec);
    if (st != SIGE_OK)
        return st;
    if (slots == 0)
        return SIGE_OK;
    a.y = static_cast<uint8_t *>(y);
    a.vecs = vec ? cd->c / 8 : cd->c;
    a.dvecs = udiv_make((uint32_t)a.vecs);
    a.dgv = udiv_make((uint32_t)std::max(1, cd->group / 8));
    const int64_t items = slots * a.vecs;
    a.fast = items <= INT32_MAX;
    if (!vec)
        return qc::run(qc::k_qcache_read_any, items, qc::kThreads, (cudaStream_t)stream, a, (int)cd->format);
    switch (cd->format) {
    case SIGE_Q_S8: return qc::run(qc::k_qcache_read<SIGE_Q_S8>, items, qc::kThreads, (cudaStream_t)stream, a);
    case SIGE_Q_E4M3: return qc::run(qc::k_qcache_read<SIGE_Q_E4M3>, items, qc::kThreads, (cudaStream_t)stream, a);
    default: return qc::run(qc::k_qcache_read<SIGE_Q_S4>, items, qc::kThreads, (cudaStream_t)stream, a);
    }
}
