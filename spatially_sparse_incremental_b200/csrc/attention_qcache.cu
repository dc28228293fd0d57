// Attention step with pruned query tokens over a quantised key / value cache:
// for every token under the tile list (or every token), per head,
//   o = softmax(q K^T / sqrt(dh)) V,   K = key codes * scales, V = value codes * scales,
// over the item's first key_counts[n] keys; a token without keys gets 0.  (The
// nubint.ai review of the SIGE paper, "Proposed method": attention layers by
// pruning the query tokens of unedited regions; the cache's formats are this
// library's.)
//
// This file holds the call and the CUDA-core kernel, for head widths the
// tensor-core kernel has no room for (193 .. 256): a CTA owns 64 query slots of one (batch item, head) and
// walks the keys in chunks of 32 decoded into shared memory; a warp owns 8
// queries, lane j scores key j, and a running maximum and sum per query
// (float32) rescale the lanes' accumulators of the columns lane + 32 c.
#include <algorithm>
#include <atomic>
#include <math.h>

#include "attention_qcache.cuh"

namespace sige {
namespace aq {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kKeys = 32;
constexpr int kQueries = 64;
constexpr int kPerWarp = kQueries / kWarps;
constexpr int kMaxHead = 256;
constexpr int kCols = kMaxHead / 32;

static size_t smem_bytes(int dh, int dvh)
{
    return sizeof(float) * ((size_t)kQueries * dh + (size_t)kKeys * (dh + 1) + (size_t)kKeys * dvh + kWarps * kKeys);
}

__device__ __forceinline__ float wmax(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

__device__ __forceinline__ float wsum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__global__ void __launch_bounds__(kThreads) k_attention_qcache(const __grid_constant__ AttnQParams p)
{
    extern __shared__ float aq_smem[];
    const int dh = p.dh, dvh = p.dvh, dhp = dh + 1;
    float *Qs = aq_smem;                  // [64][dh]
    float *Ks = Qs + kQueries * dh;       // [32][dh + 1]: 32 lanes read a column from 32 banks
    float *Vs = Ks + kKeys * dhp;         // [32][dvh]
    float *Ps = Vs + kKeys * dvh;         // [8][32]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slots = query_slots(p);
    const int qblocks = (slots + kQueries - 1) / kQueries;
    const int64_t units = (int64_t)qblocks * p.N * p.heads;

#pragma unroll 1
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int qb = (int)(u % qblocks);
        const int rest = (int)(u / qblocks), head = rest % p.heads, n = rest / p.heads;
        const int nq = min(kQueries, slots - qb * kQueries);
        const int keys = key_count(p, n);
        const int kg = head * dh / p.kgroup, vg = head * dvh / p.vgroup;
        __syncthreads();   // the previous unit has finished with the staged queries
#pragma unroll 1
        for (int e = threadIdx.x; e < nq * dh; e += kThreads) {
            const int qi = e / dh, d = e - qi * dh;
            const int64_t pix = query_pixel(p, n, qb * kQueries + qi);
            Qs[e] = pix >= 0 ? __bfloat162float(p.q[pix * p.D + head * dh + d]) : 0.0f;
        }
        float m[kPerWarp], l[kPerWarp], acc[kPerWarp][kCols];
#pragma unroll
        for (int s = 0; s < kPerWarp; ++s) {
            m[s] = -INFINITY;
            l[s] = 0.0f;
#pragma unroll
            for (int c = 0; c < kCols; ++c)
                acc[s][c] = 0.0f;
        }
        const int64_t kbase = (int64_t)n * p.keys;
#pragma unroll 1
        for (int k0 = 0; k0 < keys; k0 += kKeys) {
            const int nk = min(kKeys, keys - k0);
            __syncthreads();   // queries staged; the previous chunk consumed
#pragma unroll 1
            for (int e = threadIdx.x; e < kKeys * dh; e += kThreads) {
                const int j = e / dh, d = e - j * dh;
                const int64_t row = kbase + k0 + j;
                Ks[j * dhp + d] = j < nk ? code_at(p.kc, row * p.D + head * dh + d, p.kfmt) * __ldg(p.ks + row * p.kng + kg)
                                         : 0.0f;
            }
            int big = 0;   // (kBigScale)
#pragma unroll 1
            for (int e = threadIdx.x; e < kKeys * dvh; e += kThreads) {
                const int j = e / dvh, d = e - j * dvh;
                const int64_t row = kbase + k0 + j;
                const float s = j < nk ? __ldg(p.vs + row * p.vng + vg) : 0.0f;
                Vs[e] = j < nk ? code_at(p.vc, row * p.Dv + head * dvh + d, p.vfmt) * s : 0.0f;
                big |= fabsf(s) >= kBigScale;
            }
            const float room = __syncthreads_or(big) ? kRoom * 0.6931472f : 0.0f;
#pragma unroll
            for (int s = 0; s < kPerWarp; ++s) {
                const int qi = warp + kWarps * s;
                if (qi >= nq)   // the same for the whole warp
                    break;
                float sc = 0.0f;
                const float *qr = Qs + qi * dh, *kr = Ks + lane * dhp;
#pragma unroll 4
                for (int d = 0; d < dh; ++d)
                    sc = fmaf(qr[d], kr[d], sc);
                sc = lane < nk ? sc * p.scale : -INFINITY;
                const float mn = fmaxf(m[s], wmax(sc) + room);
                const float pj = lane < nk ? expf(sc - mn) : 0.0f;
                const float corr = expf(m[s] - mn);   // 0 on the first chunk (m = -inf)
                l[s] = l[s] * corr + wsum(pj);
                Ps[warp * kKeys + lane] = pj;
                __syncwarp();
#pragma unroll
                for (int c = 0; c < kCols; ++c) {
                    const int d = c * 32 + lane;
                    if (c * 32 < dvh) {
                        float a = acc[s][c] * corr;
                        if (d < dvh) {
#pragma unroll 4
                            for (int j = 0; j < nk; ++j)
                                a = fmaf(Ps[warp * kKeys + j], Vs[j * dvh + d], a);
                        }
                        acc[s][c] = a;
                    }
                }
                __syncwarp();
                m[s] = mn;
            }
        }
#pragma unroll
        for (int s = 0; s < kPerWarp; ++s) {
            const int qi = warp + kWarps * s;
            if (qi >= nq)
                break;
            const int64_t pix = query_pixel(p, n, qb * kQueries + qi);
            if (pix < 0)
                continue;
            const float inv = keys > 0 ? 1.0f / l[s] : 0.0f;   // no keys: 0
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
                const int d = c * 32 + lane;
                if (d < dvh)
                    p.o[pix * p.Dv + head * dvh + d] = __float2bfloat16_rn(acc[s][c] * inv);
            }
        }
    }
}

static int launch(const AttnQParams &p, cudaStream_t stream)
{
    const size_t smem = smem_bytes(p.dh, p.dvh);
    static std::atomic<int> smem_set[64];   // per device: the opt-in of the largest request
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return SIGE_ERR_CUDA;
    if (!smem_set[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(k_attention_qcache, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)smem_bytes(kMaxHead, kMaxHead)) != cudaSuccess) {
            cudaGetLastError();
            return SIGE_ERR_CUDA;
        }
        smem_set[dev].store(1, std::memory_order_release);
    }
    prefer_max_shared(k_attention_qcache);
    const int64_t units = (p.slots + kQueries - 1) / kQueries * p.N * p.heads;
    const int grid = (int)std::min<int64_t>(units, (int64_t)device_sm_count() * 4);
    k_attention_qcache<<<grid, kThreads, smem, stream>>>(p);
    count_launch();
    return launch_check();
}

static int check(const sige_tensor_desc *qd, const sige_qcache_desc *kd, const sige_qcache_desc *vd, int32_t heads)
{
    if (!qd || heads < 1 || qd->n < 1 || qd->h < 1 || qd->w < 1 || qd->c < 1)
        return SIGE_ERR_INVALID_ARG;
    int st = qcache_check(kd);
    if (st == SIGE_OK)
        st = qcache_check(vd);
    if (st != SIGE_OK)
        return st;
    if (kd->n != qd->n || vd->n != qd->n || (int64_t)kd->h * kd->w != (int64_t)vd->h * vd->w || kd->c != qd->c ||
        qd->c % heads || vd->c % heads)
        return SIGE_ERR_INVALID_ARG;
    const int dh = qd->c / heads, dvh = vd->c / heads;
    // one scale for a head's whole slice of a key or a value
    if (qd->dtype != SIGE_BF16 || qd->layout != SIGE_NHWC || dh > kMaxHead || dvh > kMaxHead || kd->group % dh ||
        vd->group % dvh)
        return SIGE_ERR_UNSUPPORTED;
    // (keys are counted in 32 bits, up to a chunk past the last)
    if ((int64_t)qd->n * qd->h > INT32_MAX || (int64_t)qd->n * qd->h * qd->w > INT32_MAX ||
        (int64_t)kd->h * kd->w > INT32_MAX - 1024)
        return SIGE_ERR_UNSUPPORTED;
    return SIGE_OK;
}

} // namespace aq
} // namespace sige

using namespace sige;

extern "C" int sige_attention_qcache(const void *q, const sige_tensor_desc *qd, const void *k_codes,
                                     const float *k_scales, const sige_qcache_desc *kd, const void *v_codes,
                                     const float *v_scales, const sige_qcache_desc *vd, const int32_t *key_counts,
                                     int32_t heads, int32_t block, const int32_t *idx, const int32_t *count,
                                     int32_t capacity, void *o, void *workspace, size_t workspace_bytes,
                                     sige_stream_t stream)
{
    if (!q || !k_codes || !k_scales || !v_codes || !v_scales || !o)
        return SIGE_ERR_INVALID_ARG;
    int st = aq::check(qd, kd, vd, heads);
    if (st != SIGE_OK)
        return st;
    if (!aligned_to(q, 2) || !aligned_to(o, 2) || !aligned_to(k_scales, 4) || !aligned_to(v_scales, 4) ||
        !aligned_to(key_counts, 4))
        return SIGE_ERR_INVALID_ARG;
    const int64_t pixels = (int64_t)qd->n * qd->h * qd->w, obytes = pixels * vd->c * 2;
    if (ranges_overlap(o, obytes, q, pixels * qd->c * 2) || ranges_overlap(o, obytes, k_codes, qcache_bytes(kd)) ||
        ranges_overlap(o, obytes, v_codes, qcache_bytes(vd)) ||
        ranges_overlap(o, obytes, k_scales, 4 * qcache_scale_count(kd)) ||
        ranges_overlap(o, obytes, v_scales, 4 * qcache_scale_count(vd)) || ranges_overlap(o, obytes, key_counts, 4ll * qd->n))
        return SIGE_ERR_INVALID_ARG;
    PixelList px;
    AttnQParams p{};
    st = pixel_list_make(&px, qd->n, qd->h, qd->w, block, idx, count, capacity, &p.slots);
    if (st != SIGE_OK)
        return st;
    if (!workspace || workspace_bytes < kWsHeader || !aligned_to(workspace, 16))
        return SIGE_ERR_WORKSPACE;
    if (list_overlaps(o, obytes, idx, count, capacity) || ranges_overlap(o, obytes, workspace, kWsHeader))
        return SIGE_ERR_INVALID_ARG;
    if (p.slots == 0)
        return SIGE_OK;
    p.slots /= qd->n;
    // the device indexes a unit's slots, items and heads in 32 bits
    if (p.slots > INT32_MAX - 1024 || (int64_t)qd->n * heads > INT32_MAX)
        return SIGE_ERR_UNSUPPORTED;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.kc = static_cast<const uint8_t *>(k_codes);
    p.vc = static_cast<const uint8_t *>(v_codes);
    p.ks = k_scales;
    p.vs = v_scales;
    p.key_counts = key_counts;
    p.idx = idx; p.count = count; p.cap = capacity; p.b = px.b;
    p.N = qd->n; p.H = qd->h; p.W = qd->w; p.D = qd->c; p.Dv = vd->c;
    p.keys = kd->h * kd->w;
    p.heads = heads; p.dh = qd->c / heads; p.dvh = vd->c / heads;
    p.kfmt = kd->format; p.vfmt = vd->format;
    p.kgroup = kd->group; p.vgroup = vd->group;
    p.kng = kd->c / kd->group; p.vng = vd->c / vd->group;
    p.scale = (float)(1.0 / std::sqrt((double)p.dh));
    p.dbb = px.dbb; p.db = px.db;
    p.hdr = static_cast<WsHeader *>(workspace);
    const int tc = launch_attention_qcache_tc(p, (cudaStream_t)stream);
    return tc != 1 ? tc : aq::launch(p, (cudaStream_t)stream);
}

extern "C" int sige_attention_qcache_path(int32_t dh, int32_t dvh)
{
    if (dh < 1 || dvh < 1)
        return SIGE_ERR_INVALID_ARG;
    if (dh > aq::kMaxHead || dvh > aq::kMaxHead)
        return SIGE_ERR_UNSUPPORTED;
    return attention_qcache_tc_scope(dh, dvh) ? 1 : 0;
}
