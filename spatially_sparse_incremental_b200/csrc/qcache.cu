// The quantised activation cache: a map is written as 8- or 4-bit codes with
// one float32 scale per group of channels of a pixel, and read back, at the
// listed tiles or whole.  (mer.dev notes on SIGE, section 3 "Method" and
// section 4.2: the activations of the original are kept, for a diffusion model
// those of every step, which costs memory; the formats are this library's.)
//
// Both kernels are one pass over the data and bound by memory: a group's
// elements are loaded once into registers (16 bytes a load), the largest
// magnitude is found among the lanes that share the group, and the codes leave
// from the same registers.  Accesses are of 8, 4 or 2 elements.  4 x 256 x 256 x 128 bf16, 105 MB each way: write
// 19.5 us in e4m3 with a scale per 32 channels (5.4 TB/s), 28.0 us in s8 with a
// scale per pixel (the tie tests; 24 us on data without ties), read 18.5 us
// (5.7 TB/s).  The forms for any alignment and any group take 249, 135 and 106
// to 127 us there; groups of more than 2048 channels are written by that form
// too (16 x 32 x 32 x 2560 in s8, a scale per pixel, 170 us).  With the affine and
// SiLU the e4m3 write takes 44 us: its parameters are read a float at a time.
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
    int32_t gv;            // vectors of a group
    UDiv dng, dvecs, dgv;  // groups of a pixel, vectors of a pixel, vectors of a group
    UDiv dhw;              // pixels of an item
    int32_t fast;          // every item index fits 32 bits
    int32_t wide;          // the map's groups (write) or vectors (read) do not
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

// kN (8, 4 or 2) elements of kE bytes, as loaded.
template <int kE, int kN>
struct Raw {
    static constexpr int kWords = kN * kE / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int k = 0; k < kWords; ++k)
            w[k] = 0;
    }
    __device__ __forceinline__ void load(const uint8_t *x, int64_t e)
    {
        const uint8_t *p = x + e * kE;
        if constexpr (kWords >= 4) {
#pragma unroll
            for (int h = 0; h < kWords / 4; ++h) {
                const uint4 r = ld_nc16(p + 16 * h);
                w[4 * h] = r.x; w[4 * h + 1] = r.y; w[4 * h + 2] = r.z; w[4 * h + 3] = r.w;
            }
        } else if constexpr (kWords == 2) {
            const uint2 r = __ldg(reinterpret_cast<const uint2 *>(p));
            w[0] = r.x; w[1] = r.y;
        } else {
            w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
        }
    }
    __device__ __forceinline__ void values(float (&v)[kN]) const
    {
#pragma unroll
        for (int k = 0; k < kN; ++k)
            v[k] = kE == 4 ? __uint_as_float(w[k]) : k & 1 ? bf16_hi(w[k >> 1]) : bf16_lo(w[k >> 1]);
    }
};

// Larger magnitude of two, a NaN if either is one.
__device__ __forceinline__ float amax2(float m, float v)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
    return r;
}

template <int kFmt, int kN>
__device__ __forceinline__ void store_codes(uint8_t *codes, int64_t e, const float (&v)[kN], float s, float r)
{
    uint32_t w[2] = {0, 0};
    if constexpr (kFmt == SIGE_Q_E4M3) {
        if (r > 0.0f) {
#pragma unroll
            for (int k = 0; k < kN; k += 2)
                w[k >> 2] |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[k] * r, v[k + 1] * r), __NV_SATFINITE, __NV_E4M3)
                             << (8 * (k & 3));
        }
    } else if (r > 0.0f) {
        // round(v r) by way of 1.5 * 2^23, where float32 has a spacing of one:
        // the sum's low bits are the code.  One test for all of them: bf16
        // elements make near ties common (half the largest magnitude is one), and
        // most of them are rounded right.
        uint32_t c[kN];
        float off = 0.0f;
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            const float t = __fadd_rn(v[k] * r, kRoundBase);
            c[k] = __float_as_uint(t);
            off = fmaxf(off, fabsf(quotient_rest(v[k], s, __fsub_rn(t, kRoundBase))));
        }
        if (2.0f * off >= s) {
#pragma unroll
            for (int k = 0; k < kN; ++k)
                c[k] = (uint32_t)quotient_code(v[k], s, r);
        }
        if constexpr (kFmt == SIGE_Q_S4) {
#pragma unroll
            for (int k = 0; k < kN; ++k)
                w[0] |= (c[k] & 15u) << (4 * k);
        } else if constexpr (kN == 2) {
            w[0] = __byte_perm(c[0], c[1], 0x0040) & 0xFFFFu;
        } else {
#pragma unroll
            for (int h = 0; h < kN / 4; ++h)
                w[h] = __byte_perm(__byte_perm(c[4 * h], c[4 * h + 1], 0x0040),
                                   __byte_perm(c[4 * h + 2], c[4 * h + 3], 0x0040), 0x5410);
        }
    }
    constexpr int kBytes = kFmt == SIGE_Q_S4 ? kN / 2 : kN;
    uint8_t *dst = codes + (kFmt == SIGE_Q_S4 ? e >> 1 : e);
    if constexpr (kBytes == 8)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
    else if constexpr (kBytes == 4)
        *reinterpret_cast<uint32_t *>(dst) = w[0];
    else if constexpr (kBytes == 2)
        *reinterpret_cast<uint16_t *>(dst) = (uint16_t)w[0];
    else
        *dst = (uint8_t)w[0];
}

// Write, vector form: `lanes` neighbouring lanes share one group, each with up
// to V vectors of kN (8, 4 or 2) channels in registers.  Over a whole map group i's elements
// start at i * group: no division.
template <int kFmt, int kE, int kN, int V>
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
        int64_t at = base + mine;   // the group's number in the map, -1: none
        if (at >= items)
            at = -1;
        if (p.px.idx && at >= 0) {
            uint32_t slot;
            int g;
            split_item(at, p.ng, p.dng, p.fast, &slot, &g);
            const int64_t pix = pixel_of(p.px, slot);
            at = pix < 0 ? -1 : pix * p.ng + g;
        }
        Raw<kE, kN> raw[V];
        float v[V][kN], m = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int vec = sub + j * p.lanes;
            raw[j].zero();
            if (at >= 0 && vec < p.vecs)
                raw[j].load(p.x, at * p.group + kN * vec);
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
            raw[j].values(v[j]);
        if ((p.gsc || p.silu) && at >= 0) {
            uint32_t pix;
            int g;
            split_item(at, p.ng, p.dng, !p.wide, &pix, &g);
            const int64_t c0 = (int64_t)udiv(pix, p.dhw) * p.C + (int64_t)g * p.group;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int vec = sub + j * p.lanes;
                if (vec < p.vecs) {
                    const int64_t c = c0 + kN * vec;
#pragma unroll
                    for (int k = 0; k < kN; ++k)
                        v[j][k] = transform1(v[j][k], p.gsc ? p.gsc + c : nullptr, p.gsc ? p.gsh + c : nullptr, k, p.silu);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int k = 0; k < kN; ++k)
                m = amax2(m, v[j][k]);
        uint32_t amax = __float_as_uint(m);
        for (int o = p.lanes >> 1; o > 0; o >>= 1)
            amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
        if (at < 0)
            continue;
        const float s = group_scale<kFmt>(amax), r = scale_reciprocal<kFmt>(s);
        if (sub == 0)
            p.scales[at] = s;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int vec = sub + j * p.lanes;
            if (vec < p.vecs)
                store_codes<kFmt, kN>(p.codes, at * p.group + kN * vec, v[j], s, r);
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
        const float s = group_scale<kFmt>(amax), r = scale_reciprocal<kFmt>(s);
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

// What kN codes stand for, before the scale.
template <int kFmt, int kN>
__device__ __forceinline__ void code_values(uint2 w, float (&v)[kN])
{
    if constexpr (kFmt == SIGE_Q_S4) {
#pragma unroll
        for (int k = 0; k < kN; ++k)
            v[k] = s4_value(w.x, k);
    } else if constexpr (kFmt == SIGE_Q_S8) {
        // byte b of 128 + code is the float32 2^23 + b, less 2^23 + 128
        const uint32_t u[2] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u};
#pragma unroll
        for (int k = 0; k < kN; ++k)
            v[k] = __uint_as_float(__byte_perm(u[k >> 2], 0x4B000000u, 0x7440 + (k & 3))) - 8388736.0f;
    } else {
#pragma unroll
        for (int k = 0; k < kN / 2; ++k) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                (__nv_fp8x2_storage_t)((k < 2 ? w.x : w.y) >> (16 * (k & 1))), __NV_E4M3);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            v[2 * k] = f.x;
            v[2 * k + 1] = f.y;
        }
    }
}

// Read, vector form: kN (8, 4 or 2) codes of one group a thread.  Over a whole map
// vector i's elements start at kN i.
template <int kFmt, int kE, int kN>
__global__ void __launch_bounds__(kThreads) k_qcache_read(const __grid_constant__ Args p)
{
    pdl_wait();
    const int64_t items = pixel_slots(p.px) * p.vecs;
    const int64_t step = (int64_t)gridDim.x * kThreads;
#pragma unroll 1
    for (int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x; item < items; item += step) {
        int64_t at = item;   // the vector's number in the map
        if (p.px.idx) {
            uint32_t slot;
            int vec;
            split_item(item, p.vecs, p.dvecs, p.fast, &slot, &vec);
            const int64_t pix = pixel_of(p.px, slot);
            if (pix < 0)
                continue;
            at = pix * p.vecs + vec;
        }
        const float s = __ldg(p.scales + (p.wide ? at / p.gv : (int64_t)udiv((uint32_t)at, p.dgv)));
        constexpr int kBytes = kFmt == SIGE_Q_S4 ? kN / 2 : kN;
        uint2 w = make_uint2(0, 0);
        if constexpr (kBytes == 8)
            w = __ldg(reinterpret_cast<const uint2 *>(p.codes) + at);
        else if constexpr (kBytes == 4)
            w.x = __ldg(reinterpret_cast<const uint32_t *>(p.codes) + at);
        else if constexpr (kBytes == 2)
            w.x = __ldg(reinterpret_cast<const uint16_t *>(p.codes) + at);
        else
            w.x = __ldg(p.codes + at);
        float v[kN];
        code_values<kFmt, kN>(w, v);
#pragma unroll
        for (int k = 0; k < kN; ++k)
            v[k] *= s;
        if constexpr (kE == 4 && kN >= 4) {
            float4 *o = reinterpret_cast<float4 *>(p.y) + kN / 4 * at;
#pragma unroll
            for (int h = 0; h < kN / 4; ++h)
                o[h] = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
        } else if constexpr (kE == 4) {
            reinterpret_cast<float2 *>(p.y)[at] = make_float2(v[0], v[1]);
        } else if constexpr (kN == 8) {
            reinterpret_cast<uint4 *>(p.y)[at] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
        } else if constexpr (kN == 4) {
            reinterpret_cast<uint2 *>(p.y)[at] = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        } else {
            reinterpret_cast<uint32_t *>(p.y)[at] = pack_bf16x2(v[0], v[1]);
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

template <auto kKernel, typename... A>
static int run(int64_t items, int per_block, cudaStream_t stream, const A &...args)
{
    prefer_max_shared_of<kKernel>();
    const int64_t most = (int64_t)device_sm_count() * 32;
    const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>((items + per_block - 1) / per_block, most));
    if (launch_pdl(kKernel, dim3(grid), dim3(kThreads), 0, stream, args...) != cudaSuccess) {
        cudaGetLastError();
        return SIGE_ERR_CUDA;
    }
    count_launch();
    return launch_check();
}

template <int kFmt, int kE, int kN>
static int run_write_as(Args &a, int64_t items, cudaStream_t stream)
{
    a.vecs = a.group / kN;
    // (lanes, V) with the fewest places left empty; two vectors a lane before
    // one, then the fewest.  Powers of two only left 24 of 64 places empty for 40
    // vectors: 16 x 64 x 64 x 320 in s8 29.1 us, 16.5 us with 8 lanes of 5.
    const int choice[] = {2, 1, 3, 4, 5, 8};
    int V = 0, best = INT32_MAX;
    for (int c : choice) {
        int lanes = a.vecs > 1 ? 2 : 1;
        while (lanes < 32 && lanes * c < a.vecs)
            lanes *= 2;
        if (lanes * c >= a.vecs && lanes * c < best) {
            best = lanes * c;
            V = c;
            a.lanes = lanes;
        }
    }
    const int per_block = kThreads / a.lanes;
    switch (V) {
    case 1: return run<k_qcache_write<kFmt, kE, kN, 1>>(items, per_block, stream, a);
    case 2: return run<k_qcache_write<kFmt, kE, kN, 2>>(items, per_block, stream, a);
    case 3: return run<k_qcache_write<kFmt, kE, kN, 3>>(items, per_block, stream, a);
    case 4: return run<k_qcache_write<kFmt, kE, kN, 4>>(items, per_block, stream, a);
    case 5: return run<k_qcache_write<kFmt, kE, kN, 5>>(items, per_block, stream, a);
    default: return run<k_qcache_write<kFmt, kE, kN, 8>>(items, per_block, stream, a);
    }
}

// kN elements of kE bytes at once, or (0) any group at any address.
template <int kFmt, int kE>
static int run_write(Args &a, int64_t slots, int n, cudaStream_t stream)
{
    const int64_t items = slots * a.ng;
    a.fast = items <= INT32_MAX;
    switch (a.group <= 256 * n ? n : 0) {   // (a group in a warp's registers: 32 lanes, 8 vectors)
    case 8: return run_write_as<kFmt, kE, 8>(a, items, stream);
    case 4: return run_write_as<kFmt, kE, 4>(a, items, stream);
    case 2: return run_write_as<kFmt, kE, 2>(a, items, stream);
    default: return run<k_qcache_write_any<kFmt>>(items, kThreads / 32, stream, a);
    }
}

template <int kFmt, int kE>
static int run_read(const Args &a, int64_t items, int n, cudaStream_t stream)
{
    switch (n) {
    case 8: return run<k_qcache_read<kFmt, kE, 8>>(items, kThreads, stream, a);
    case 4: return run<k_qcache_read<kFmt, kE, 4>>(items, kThreads, stream, a);
    case 2: return run<k_qcache_read<kFmt, kE, 2>>(items, kThreads, stream, a);
    default: return run<k_qcache_read_any>(items, kThreads, stream, a, kFmt);
    }
}

// What the two calls check alike, and the arguments they share.
static int common(Args *a, const void *map, const sige_tensor_desc *md, const void *codes, const float *scales,
                  const sige_qcache_desc *cd, int32_t block, const int32_t *idx, const int32_t *count,
                  int32_t capacity, int64_t *slots, int *n)
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
    a->dhw = udiv_make((uint32_t)((int64_t)cd->h * cd->w));
    // the most elements of a group that one aligned access takes: 4 x 256 x 256 x
    // 120 bf16 in e4m3, a scale per 40, written 19.4 us by 8, 22.2 by 4, 29.4 by 2,
    // 221 by one; read 16.5, 21.9, 31.0, 115
    for (*n = 8; *n; *n = *n > 2 ? *n / 2 : 0)
        if (cd->group % *n == 0 && aligned_to(map, (uintptr_t)std::min(16, *n * esz)) &&
            aligned_to(codes, (uintptr_t)std::max(1, cd->format == SIGE_Q_S4 ? *n / 2 : *n)))
            break;
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
    int n;
    const int st = qc::common(&a, x, xd, codes, scales, cd, block, idx, count, capacity, &slots, &n);
    if (st != SIGE_OK)
        return st;
    if ((gn_scale == nullptr) != (gn_shift == nullptr) || !aligned_to(gn_scale, 4) || !aligned_to(gn_shift, 4))
        return SIGE_ERR_INVALID_ARG;
    // the cache is written while the other operands are read
    const int64_t cb = qcache_bytes(cd), sb = 4 * qcache_scale_count(cd), gb = 4ll * cd->n * cd->c;
    if (ranges_overlap(codes, cb, gn_scale, gb) || ranges_overlap(codes, cb, gn_shift, gb) ||
        ranges_overlap(scales, sb, gn_scale, gb) || ranges_overlap(scales, sb, gn_shift, gb) ||
        list_overlaps(codes, cb, idx, count, capacity) || list_overlaps(scales, sb, idx, count, capacity))
        return SIGE_ERR_INVALID_ARG;
    if (slots == 0)
        return SIGE_OK;
    a.x = static_cast<const uint8_t *>(x);
    a.gsc = gn_scale;
    a.gsh = gn_shift;
    a.silu = silu ? 1 : 0;
    a.wide = (int64_t)cd->n * cd->h * cd->w * a.ng > INT32_MAX;
    const cudaStream_t st_ = (cudaStream_t)stream;
    const bool bf16 = xd->dtype == SIGE_BF16;
    switch (cd->format) {
    case SIGE_Q_S8: return bf16 ? qc::run_write<SIGE_Q_S8, 2>(a, slots, n, st_) : qc::run_write<SIGE_Q_S8, 4>(a, slots, n, st_);
    case SIGE_Q_E4M3: return bf16 ? qc::run_write<SIGE_Q_E4M3, 2>(a, slots, n, st_) : qc::run_write<SIGE_Q_E4M3, 4>(a, slots, n, st_);
    default: return bf16 ? qc::run_write<SIGE_Q_S4, 2>(a, slots, n, st_) : qc::run_write<SIGE_Q_S4, 4>(a, slots, n, st_);
    }
}

extern "C" int sige_qcache_read(const void *codes, const float *scales, const sige_qcache_desc *cd, int32_t block,
                                const int32_t *idx, const int32_t *count, int32_t capacity, void *y,
                                const sige_tensor_desc *yd, sige_stream_t stream)
{
    qc::Args a{};
    int64_t slots;
    int n;
    const int st = qc::common(&a, y, yd, codes, scales, cd, block, idx, count, capacity, &slots, &n);
    if (st != SIGE_OK)
        return st;
    if (list_overlaps(y, (int64_t)cd->n * cd->h * cd->w * cd->c * (yd->dtype == SIGE_BF16 ? 2 : 4), idx, count, capacity))
        return SIGE_ERR_INVALID_ARG;
    if (slots == 0)
        return SIGE_OK;
    a.y = static_cast<uint8_t *>(y);
    a.vecs = n ? cd->c / n : cd->c;
    a.dvecs = udiv_make((uint32_t)a.vecs);
    a.gv = n ? cd->group / n : 1;
    a.dgv = udiv_make((uint32_t)a.gv);
    const int64_t items = slots * a.vecs;
    a.fast = items <= INT32_MAX;
    a.wide = (int64_t)cd->n * cd->h * cd->w * a.vecs > INT32_MAX;
    const cudaStream_t st_ = (cudaStream_t)stream;
    const bool bf16 = yd->dtype == SIGE_BF16;
    switch (cd->format) {
    case SIGE_Q_S8: return bf16 ? qc::run_read<SIGE_Q_S8, 2>(a, items, n, st_) : qc::run_read<SIGE_Q_S8, 4>(a, items, n, st_);
    case SIGE_Q_E4M3: return bf16 ? qc::run_read<SIGE_Q_E4M3, 2>(a, items, n, st_) : qc::run_read<SIGE_Q_E4M3, 4>(a, items, n, st_);
    default: return bf16 ? qc::run_read<SIGE_Q_S4, 2>(a, items, n, st_) : qc::run_read<SIGE_Q_S4, 4>(a, items, n, st_);
    }
}
