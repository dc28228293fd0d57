// Tensor-core form of the attention step over a quantised key / value cache
// (sige_attention_qcache): o = softmax(q K^T / sqrt(dh)) V with K and V in
// codes.  A code is an integer of at most 8 bits or an e4m3 value: exact in
// bf16.  So both products run on the codes as bf16 operands, and the scales,
// one per key and head, are applied in float32 where a score meets its key: to
// the score before the softmax (key scale), to the weight after it (value
// scale); the only rounding of an operand is that of weight * scale to bf16.
//
// Work unit: one or two blocks of 128 query slots of one (batch item, head), the
// keys in chunks of 128 (heads up to 64 channels) or 64 (wider).  A job is one
// chunk against one block.  Roles of a CTA's 16 warps:
//   * warp 0 issues S = Q K^T (M 128, N a chunk), warp 1 O += P V (M 128, K a
//     chunk), each from one elected lane.  One warp for both took about 1300
//     cycles a job.  Warps 0 and 1 because the schedulers serve the lowest numbers
//     first: 1 us of 80 on one map;
//   * six warps stage the operands: the unit's queries once, and for each chunk
//     the codes (global loads of 8 codes a thread, a chunk ahead in registers),
//     turned into bf16 rows of 128 bytes with the 128-byte swizzle (K-major for
//     the first product, MN-major for the second), and the chunk's scales;
//   * two groups of four warps do the softmax of a job each, in one pass over the
//     scores: read in the fragment layout, scaled, weighted against a standing
//     exponent base, P = 2^(s - base) * value scale stored as bf16.  The base
//     moves only when a score lies kSlack above it, so an ordinary job reads its
//     scores once and leaves O alone.  Four groups at 80 registers were slower.
// With more units than CTAs a unit is two blocks, one for each group, so that a
// chunk is staged once for 256 queries (64x64, 8 heads of 40, one map: 79 us, 111
// in units of one block), where that saves enough rounds of units; otherwise the
// groups take the chunks of one block in turn and their rows (O, base, sum) are
// merged through shared memory at the end of the unit.  Where units are few, the CTAs of a cluster also split the keys and
// push their rows to the row's owner through distributed shared memory (25 tiles
// of 4x4 against 4096 keys, 32 units: 24.5 us, 57 without the split; one 32x32 map,
// 8 heads of 80: 22 and 30 us).  A launch is at most as many clusters of four as fit
// the device at once, 33 here: 132 CTAs, 16 of the 148 SMs take no part.
//
// Head widths up to 192 in three layouts (64, 128, 192 channels staged a row), each
// in two forms: vectors of 8 codes and 16-byte query and output vectors, or (kAny:
// widths that are not multiples of 8, unaligned tensors) codes out of aligned words
// and the rest element by element: 44 us for the 25 tiles, 142 for the map (the
// CUDA-core kernel: 2575 and 5680).
//
// Bound: the softmax groups.  One map (4096 queries and keys, 8 heads of 40) is
// 134M exponentials, 30 us at 16 a cycle and SM, and 21.5 GFLOP (26 with heads of
// 40 run as 48), 16 us at the bf16 rate.  A job of 128 queries x 128 keys takes
// about 4700 cycles of a group, two groups at once: the scores' way out of tensor
// memory, scaling, exponentials and packing of its 128 values a lane, with the two
// groups' four schedulers shared with staging (codes to bf16) and issue; about 1900
// of them are the wait for the next scores.
#include <algorithm>
#include <atomic>
#include <math.h>
#include <type_traits>

#include "attention_qcache.cuh"
#include "attn_ptx.cuh"

namespace sige {
namespace at {

using namespace attn;

constexpr int kRows = 128;
constexpr int kGroup = 128;         // threads of a softmax group
constexpr int kStage = 192;         // staging threads
constexpr int kCluster = 4;
// A weight's rounding to bf16 is as large as an output's, whatever the number of
// keys: results of 33 to 4096 keys are 1.2 to 1.5 times as far from the exact ones as
// those of float32 weights (both rounded to bf16 at the end; 1.6 for some sets of
// four queries).  Items of at most kShort keys, where it does not average out (with
// one or two keys it is all that a row's values share), have their weights in two
// bf16 terms, and 1.0.  kShort: the second terms lie where the weights of the next
// kShort keys would, and meet the same values, so that the narrowest chunk (64
// keys) holds both and they cost no product.
constexpr int kShort = 32;
constexpr float kSlack = 40.0f;     // how far (base 2) a score may lie above the exponent base (kBigScale)

// Shared and tensor memory for heads of up to KD (64, 128 or 192) channels.
template <int KD>
struct Lay {
    static constexpr int kKeys = KD == 64 ? 128 : 64;                 // keys of a chunk
    static constexpr int kSoft = 2 * kGroup, kThreads = kSoft + 64 + kStage;
    static constexpr int kAtoms = KD / 64;                            // 64-channel blocks of 128-byte rows
    static constexpr int kStages = KD == 192 ? 2 : 3;                 // chunk ring
    static constexpr uint32_t kQAtom = kRows * 128, kKvAtom = kKeys * 128;
    static constexpr uint32_t kOffQ = 0;                              // queries, a second block's at kOffQ2
    static constexpr uint32_t kOffQ2 = kAtoms * kQAtom;
    // rows exchanged by the groups of a block, 32 floats a softmax thread at a
    // time (over the second block's queries: units of one block only)
    static constexpr uint32_t kOffX = kOffQ2;
    static constexpr uint32_t kX = kSoft * 32 * 4 > kAtoms * kQAtom ? kSoft * 32 * 4 : kAtoms * kQAtom;
    static constexpr uint32_t kOffK = kOffX + kX;                     // [stage][K atoms, V atoms]
    static constexpr uint32_t kKvStage = 2 * kAtoms * kKvAtom;
    static constexpr uint32_t kScStage = 2 * kKeys * 4;
    static constexpr uint32_t kOffSc = kOffK + kStages * kKvStage;    // [stage][key scales, value scales]
    static constexpr uint32_t kOffMl = kOffSc + kStages * kScStage;   // (max, sum) of a softmax thread's row
    static constexpr uint32_t kOffBar = kOffMl + kSoft * 8;
    static constexpr uint32_t kBytes = kOffBar + 256 + 1024;          // + alignment slack
    // rows pushed by the CTAs of a split unit, over the queries and the ring
    // (both idle by then): kSoft rows of KD floats
    static constexpr uint32_t kOffPush = 0;
    static_assert(232 + 8 * kStages <= 256, "flags behind the barriers (kBig)");
    static_assert(kOffPush + kSoft * KD * 4 <= kOffSc, "pushed rows");
    static_assert(kOffK % 1024 == 0, "swizzled rows");
    static_assert(kBytes <= 227 * 1024, "shared memory");
    // Tensor memory, 512 columns.  Heads up to 64: a group's S (128 columns), its
    // P apart (64), so that the next S comes while the weights are still being
    // made; O (64).  Up to 128: two buffers of 64 columns a group, P over S; O
    // (128).  Up to 192: one such buffer; O (192).
    static constexpr bool kApart = KD == 64;
    static constexpr int kBufs = KD == 128 ? 2 : 1;
    static constexpr uint32_t kOCol = KD == 64 ? 384 : KD == 128 ? 256 : 128;
    static __device__ __forceinline__ uint32_t tmem_s(uint32_t g, uint32_t b) { return kApart ? 128u * g : 64u * (kBufs * g + b); }
    static __device__ __forceinline__ uint32_t tmem_p(uint32_t g, uint32_t b) { return kApart ? 256u + 64u * g : tmem_s(g, b); }
    static __device__ __forceinline__ uint32_t tmem_o(uint32_t g) { return kOCol + (uint32_t)KD * g; }
    static_assert(kOCol + 2 * KD == 512, "tensor memory");
};

constexpr uint32_t kBarKvFull = 0;      // + 8 stage
constexpr uint32_t kBarKvEmpty = 32;    // + 8 stage
constexpr uint32_t kBarSFull = 64;      // + 8 buffer (group by group)
constexpr uint32_t kBarSFree = 96;      // + 8 group: its S has been read (P apart)
constexpr uint32_t kBarPFull = 112;     // + 8 buffer
constexpr uint32_t kBarPvDone = 144;    // + 8 buffer: the P V of its last job has landed
constexpr uint32_t kBarQFull = 176;
constexpr uint32_t kBarQEmpty = 184;
constexpr uint32_t kBarReady = 192;     // every CTA of a split unit has finished its products
constexpr uint32_t kBarPush = 200;      // the rows this CTA owns have been pushed
constexpr uint32_t kBarDrain = 208;     // + 8 for the P V warp
constexpr uint32_t kTmemSlot = 224;
constexpr uint32_t kAbort = 228;
constexpr uint32_t kBig = 232;          // + 8 stage, a byte of each staging warp: value scales of kBigScale in the chunk
constexpr uint32_t kTmemCols = 512;

// wait sites (the detail of a recorded SIGE_ERR_TIMEOUT)
constexpr int kSiteKvEmpty = 401, kSiteKvFull = 402, kSiteQEmpty = 403, kSitePFull = 404, kSiteQFull = 405,
              kSiteSFull = 406, kSitePvDone = 407, kSiteReady = 408, kSitePush = 409, kSiteFree = 410;

struct Args {
    AttnQParams a;
    int32_t dhp, dvp;         // head widths padded to 16
    int32_t nk, nv;           // 8-channel vectors of a query or key row, of a value row
    float sc;                 // log2(e) / sqrt(dh): scores in base-2 exponent units
    UDiv dkv, dvv;            // dhp / 8, nv
};

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b)
{
    __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
    return *reinterpret_cast<uint32_t *>(&r);
}

// Two codes to a pair of bf16, exactly.  Integers by way of the bf16 numbers
// 128 + n (0x4300 | n, n < 128, unit spacing): a signed code is its low bits
// less the weight of its sign bit, so (128 + low) - (128 + sign weight) is one
// exact subtraction (256 = 0x4380).
__device__ __forceinline__ uint32_t s8_pair(uint32_t t)   // codes in the low bytes of the halves
{
    return sub_bf16x2((t & 0x007F007Fu) | 0x43004300u, (t & 0x00800080u) | 0x43004300u);
}
__device__ __forceinline__ uint32_t s4_pair(uint32_t t)   // codes in the low nibbles of the halves
{
    return sub_bf16x2((t & 0x00070007u) | 0x43004300u, (t & 0x00080008u) | 0x43004300u);
}
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t t)  // codes in the two low bytes
{
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)t, __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    return pack_bf16x2(f.x, f.y);
}

// 8 codes (two words; one for s4) to 8 bf16.
template <int kFmt>
__device__ __forceinline__ uint4 codes8(uint2 w)
{
    if constexpr (kFmt == SIGE_Q_S8) {
        return make_uint4(s8_pair(__byte_perm(w.x, 0, 0x4140)), s8_pair(__byte_perm(w.x, 0, 0x4342)),
                          s8_pair(__byte_perm(w.y, 0, 0x4140)), s8_pair(__byte_perm(w.y, 0, 0x4342)));
    } else if constexpr (kFmt == SIGE_Q_E4M3) {
        return make_uint4(e4m3_pair(w.x & 0xFFFFu), e4m3_pair(w.x >> 16), e4m3_pair(w.y & 0xFFFFu),
                          e4m3_pair(w.y >> 16));
    } else {
        const uint32_t lo = w.x, hi = w.x << 12;   // even codes in lo, odd ones in hi's upper half
        return make_uint4(s4_pair((lo & 0xFu) | (hi & 0xF0000u)), s4_pair(((lo >> 8) & 0xFu) | ((hi >> 8) & 0xF0000u)),
                          s4_pair(((lo >> 16) & 0xFu) | ((w.x >> 4) & 0xF0000u)),
                          s4_pair(((lo >> 24) & 0xFu) | ((w.x >> 12) & 0xF0000u)));
    }
}

// The first n (1 .. 8) of 8 codes from element e on, at any address, zeros for
// the others: the aligned words that hold them, shifted into place.
__device__ __forceinline__ uint2 codes_any(const uint8_t *codes, int64_t e, uint32_t n, bool s4)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(codes) + (uintptr_t)(s4 ? e >> 1 : e);
    const uint32_t *w = reinterpret_cast<const uint32_t *>(a & ~(uintptr_t)3);
    const uint32_t sh = 8u * (uint32_t)(a & 3) + (s4 ? 4u * (uint32_t)(e & 1) : 0u), bits = s4 ? 4u * n : 8u * n;
    const uint32_t w0 = __ldg(w), w1 = sh + bits > 32u ? __ldg(w + 1) : 0u, w2 = sh + bits > 64u ? __ldg(w + 2) : 0u;
    uint2 r = make_uint2(__funnelshift_r(w0, w1, sh), __funnelshift_r(w1, w2, sh));
    r.x &= bits < 32u ? (1u << bits) - 1u : 0xFFFFFFFFu;
    r.y &= bits < 32u ? 0u : bits < 64u ? (1u << (bits - 32u)) - 1u : 0xFFFFFFFFu;
    return r;
}
// The first n of 8 elements of a query row.
__device__ __forceinline__ uint4 bf16_any(const __nv_bfloat16 *q, int n)
{
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < n)
            w[k >> 1] |= (uint32_t)__ldg(reinterpret_cast<const unsigned short *>(q) + k) << (16 * (k & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// 8 channels of an output row, kAny: the first n of them, at any address.
template <bool kAny>
__device__ __forceinline__ void put8(__nv_bfloat16 *dst, const float *v, float inv, int n)
{
    if constexpr (kAny) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n)
                dst[k] = __float2bfloat16_rn(v[k] * inv);
    } else {
        store8(dst, v, inv);
    }
}

// Swizzled place of 8-channel vector v of row j: block v / 8, 16 bytes at v ^ j.
__device__ __forceinline__ uint32_t place(uint32_t atom, int j, int v)
{
    return (uint32_t)(v >> 3) * atom + (uint32_t)j * 128u + (uint32_t)(((v & 7) ^ (j & 7)) << 4);
}

// One staging thread's share of a chunk of K or V: up to N vectors of 8 codes,
// vector i being (key j, vector v) number t + kStage i of the chunk, v fastest.
// Where they lie in the chunk and in shared memory is worked out once; the next
// chunk's codes are on their way in registers.  kAny: out of aligned words, a row's
// last vector as far as the head goes.
template <int N, int kKeys, bool kAny>
struct Stager {
    uint32_t src[N];      // offset from the chunk's first key: bytes (kAny: codes)
    uint32_t to[N];       // offset in the staged rows (kAny: + codes of the vector) | key << 16 (kKeys: no such vector,
                          // kZero: zeros for padded channels)
    uint2 raw[N];
    static constexpr uint32_t kZero = 0x7FFF;
    const uint8_t *at;    // the next chunk to fetch (kAny: the codes)
    int64_t e0;           // kAny: the next chunk's first code
    uint32_t step;        // bytes (kAny: codes) of a chunk's keys
    int fmt;

    // nv vectors staged a row, the first `real` of them with codes of a head of
    // `head` channels; ch channels a key
    __device__ __forceinline__ void init(int t, int nv, UDiv dnv, int real, int head, int ch, int format, uint32_t atom)
    {
        fmt = format;
        const int sh = !kAny && format == SIGE_Q_S4 ? 1 : 0;
        step = ((uint32_t)kKeys * (uint32_t)ch) >> sh;
        const int dj = (int)udiv(kStage, dnv), dv = kStage - dj * nv;
        int j = (int)udiv((uint32_t)t, dnv), v = t - j * nv;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            src[i] = ((uint32_t)j * (uint32_t)ch + 8u * (uint32_t)v) >> sh;
            to[i] = j >= kKeys ? (uint32_t)kKeys << 16 : place(atom, j, v) | ((v < real ? (uint32_t)j : kZero) << 16);
            if (kAny && j < kKeys)
                to[i] |= (uint32_t)max(0, min(8, head - 8 * v));
            j += dj;
            v += dv;
            if (v >= nv) {
                v -= nv;
                ++j;
            }
        }
    }
    __device__ __forceinline__ void start(const uint8_t *codes, int64_t e)
    {
        if constexpr (kAny) {
            at = codes;
            e0 = e;
        } else {
            at = codes + (fmt == SIGE_Q_S4 ? e >> 1 : e);
        }
    }

    // the next chunk, of which `nkeys` keys exist (zeros for the others)
    __device__ __forceinline__ void fetch(int nkeys)
    {
        const uint32_t lim = (uint32_t)min(nkeys, kKeys) << 16;
        if constexpr (kAny) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                raw[i] = make_uint2(0, 0);
                if (to[i] < lim)
                    raw[i] = codes_any(at, e0 + src[i], to[i] & 15u, fmt == SIGE_Q_S4);
            }
            e0 += step;
            return;
        }
        if (fmt == SIGE_Q_S4) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                raw[i] = make_uint2(to[i] < lim ? __ldg(reinterpret_cast<const uint32_t *>(at + src[i])) : 0u, 0u);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                raw[i] = make_uint2(0, 0);
                if (to[i] < lim)
                    raw[i] = __ldg(reinterpret_cast<const uint2 *>(at + src[i]));
            }
        }
        at += step;
    }

    template <int kFmt>
    __device__ __forceinline__ void store_as(uint32_t base)
    {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (to[i] >> 16 != kKeys)
                sts128(base + (to[i] & 0xFFF0u), codes8<kFmt>(raw[i]));
    }
    __device__ __forceinline__ void store(uint32_t base)
    {
        if (fmt == SIGE_Q_S8)
            store_as<SIGE_Q_S8>(base);
        else if (fmt == SIGE_Q_E4M3)
            store_as<SIGE_Q_E4M3>(base);
        else
            store_as<SIGE_Q_S4>(base);
    }
};

// The scores of a chunk over one 64-channel block: `steps` (1 .. 4) steps of 16
// channels (32 bytes along the swizzled rows of both operands), from one
// elected lane.
__device__ __forceinline__ void mma_s_w(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate, int steps)
{
    asm volatile(
        "{\n .reg .pred p, e, t, e1, e2, e3;\n .reg .b32 l;\n .reg .b64 a1, a2, a3, b1, b2, b3;\n"
        " elect.sync l|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n setp.eq.b32 t, 0, 0;\n"
        " setp.gt.and.s32 e1, %5, 1, e;\n setp.gt.and.s32 e2, %5, 2, e;\n setp.gt.and.s32 e3, %5, 3, e;\n"
        " add.s64 a1, %1, 2;\n add.s64 a2, %1, 4;\n add.s64 a3, %1, 6;\n"
        " add.s64 b1, %2, 2;\n add.s64 b2, %2, 4;\n add.s64 b3, %2, 6;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
        " @e1 tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, t;\n"
        " @e2 tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, t;\n"
        " @e3 tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, t;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(steps)
        : "memory");
}

// O (+)= P V over 64 keys for one 64-channel block of V: four steps of 16 keys (8
// columns of P in tensor memory, 2 KB of V; the last two from b2 on), from one
// elected lane.
__device__ __forceinline__ void mma_pv_w(uint32_t d, uint32_t a, uint64_t b, uint64_t b2, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n .reg .pred p, e, t;\n .reg .b32 l, a1, a2, a3;\n .reg .b64 b1, b3;\n"
        " elect.sync l|e, 0xffffffff;\n setp.ne.b32 p, %5, 0;\n setp.eq.b32 t, 0, 0;\n"
        " add.u32 a1, %1, 8;\n add.u32 a2, %1, 16;\n add.u32 a3, %1, 24;\n"
        " add.s64 b1, %2, 128;\n add.s64 b3, %3, 128;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %4, p;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %4, t;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], %3, %4, t;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %4, t;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "l"(b2), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Pairs of float32.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) { return (uint64_t)hi << 32 | lo; }
__device__ __forceinline__ float lo_of(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi_of(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t lds_2(uint32_t addr)
{
    uint64_t v;
    asm volatile("ld.shared.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts_f1(uint32_t addr, float v) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory"); }
__device__ __forceinline__ void sts_f4(uint32_t addr, const float *v)
{
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]) : "memory");
}
template <int kSoft>
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSoft) : "memory"); }

// 16 tensor-memory lanes x 32 columns, spread over a warp as the accumulator
// fragment of a matrix instruction: register 4 i + e of thread t is lane t / 4
// (+ 8 for e = 2, 3), column 8 i + 2 (t mod 4) + (e mod 2).
__device__ __forceinline__ void ld16x32(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// The same lanes x 16 columns: register 2 i + e is lane t / 4 + 8 e, column
// 4 i + t mod 4 (pairs of bf16 of ld16x32's columns).
__device__ __forceinline__ void st16x16(uint32_t taddr, const uint32_t *v)
{
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// v[j] of a thread is that of row t / 4 + 8 j of the warp's 32: the value of row
// `lane`.
__device__ __forceinline__ float of_row(const float (&v)[4], int lane)
{
    const int src = (lane & 7) * 4;
    const float a = __shfl_sync(0xFFFFFFFFu, v[0], src), b = __shfl_sync(0xFFFFFFFFu, v[1], src);
    const float c = __shfl_sync(0xFFFFFFFFu, v[2], src), d = __shfl_sync(0xFFFFFFFFu, v[3], src);
    return lane < 16 ? (lane < 8 ? a : b) : (lane < 24 ? c : d);
}

// Bounded waits by every lane of a warp: false, in all lanes, when the limit
// expired or another role gave up.
template <bool kPeer>
__device__ __forceinline__ bool wait_w(uint32_t b, uint32_t parity, volatile int *abort_flag, WsHeader *hdr, int where)
{
    return __all_sync(0xFFFFFFFFu, kPeer ? mbar_wait_cluster(b, parity, abort_flag, hdr, where)
                                         : mbar_wait(b, parity, abort_flag, hdr, where));
}

// A unit and the chunks of it that one CTA takes.
struct Unit {
    int slot0, head, n, keys, c_lo, c_hi;
};

struct Work {
    int qblocks, slots, units, split, per, u_first, u_step, rank_split, base;
    int pairs;   // 1: units of two query blocks
};

template <int kKeys>
__device__ __forceinline__ Unit unit_at(const AttnQParams &p, const Work &w, int u)
{
    Unit x;
    x.slot0 = (u % w.qblocks) * (kRows << w.pairs);
    const int rest = u / w.qblocks;
    x.head = rest % p.heads;
    x.n = rest / p.heads;
    x.keys = key_count(p, x.n);
    const int nch = (x.keys + kKeys - 1) / kKeys;
    x.c_lo = (int)((int64_t)w.rank_split * nch / w.split);
    x.c_hi = (int)((int64_t)(w.rank_split + 1) * nch / w.split);
    return x;
}

} // namespace at

using namespace at;

template <int KD, bool kAny>
__global__ void __launch_bounds__(at::Lay<KD>::kThreads, 1) k_attn_qcache_tc(const __grid_constant__ at::Args args)
{
    using L = Lay<KD>;
    constexpr int kKeys = L::kKeys;
    extern __shared__ __align__(1024) uint8_t at_raw[];
    const AttnQParams &p = args.a;
    const uint32_t raw = smem_u32(at_raw);
    const uint32_t sb = (raw + 1023u) & ~1023u;
    uint8_t *smem = at_raw + (sb - raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t bar = sb + L::kOffBar;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kOffBar + kAbort);
    WsHeader *hdr = p.hdr;

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(bar + kTmemSlot),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    pdl_wait();
    Work w;
    w.slots = query_slots(p);
    w.qblocks = (w.slots + kRows - 1) / kRows;
    w.units = w.qblocks * p.N * p.heads;
    {
        // One block of 128 queries fills a CTA when there are CTAs for all of them.
        // With more, two blocks share each chunk's staging where that saves a
        // quarter of the rounds of units over the CTAs: a unit of two blocks takes
        // 1.32 (heads of 40) to 1.45 (of 160) times as long as one of one, whose two
        // groups share the chunks.  2048 keys, 8 heads of 40: 8 items of 3 blocks
        // 44.6 us, 61.0 with single blocks; 25 items of one block 80.8 us, 60.9.
        const int half = ((w.qblocks + 1) >> 1) * p.N * p.heads, ctas = (int)gridDim.x;
        w.pairs = w.units > ctas && 4 * ((half + ctas - 1) / ctas) < 3 * ((w.units + ctas - 1) / ctas);
        if (w.pairs) {
            w.qblocks = (w.qblocks + 1) >> 1;
            w.units = half;
        }
    }
    {
        // the key split: the same on every CTA (it depends on the list's
        // length and the cache's keys); a split unit is its CTAs' only one
        const int nch = (p.keys + kKeys - 1) / kKeys;
        w.split = kCluster;
        while (w.split > 1 && (w.pairs || (int64_t)w.units * w.split > (int64_t)gridDim.x || nch < 4 * w.split))
            w.split >>= 1;
        w.per = kCluster / w.split;
        const int rank = (int)cluster_rank(), sub = rank / w.split;
        w.rank_split = rank - sub * w.split;
        w.base = sub * w.split;
        w.u_first = (int)(blockIdx.x / kCluster) * w.per + sub;
        w.u_step = (int)(gridDim.x / kCluster) * w.per;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < L::kStages; ++i) {
            mbar_init(bar + kBarKvFull + 8u * i, kStage);
            mbar_init(bar + kBarKvEmpty + 8u * i, 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar + kBarSFull + 8u * i, 1);
            mbar_init(bar + kBarPFull + 8u * i, kGroup / 32);
            mbar_init(bar + kBarPvDone + 8u * i, 1);
        }
        mbar_init(bar + kBarSFree, kGroup / 32);
        mbar_init(bar + kBarSFree + 8u, kGroup / 32);
        mbar_init(bar + kBarQFull, kStage);
        mbar_init(bar + kBarQEmpty, 1);
        // one arrival a warp: of every softmax warp of the unit's CTAs; of the
        // warps whose rows this CTA owns (two groups of s CTAs, 128 / s rows of each)
        mbar_init(bar + kBarReady, (uint32_t)(L::kSoft / 32 * w.split));
        mbar_init(bar + kBarPush, (uint32_t)L::kSoft / 32);
        mbar_init(bar + kBarDrain, 1);
        mbar_init(bar + kBarDrain + 8u, 1);
        *abort_flag = 0;
        for (int i = 0; i < L::kStages; ++i)
            *reinterpret_cast<volatile uint64_t *>(smem + L::kOffBar + kBig + 8u * i) = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + L::kOffBar + kTmemSlot);
    cluster_arrive();   // the peers' barriers are initialised before the first remote arrival
    bool joined = false;

    // roles: warps 0 and 1 the products (the lowest numbers: the schedulers serve
    // them first), 4 .. 11 the softmax groups, the others staging
    if (warp < 4 || warp >= 12) {
        if (warp >= 2) {
            // ---- staging
            const int t = (int)threadIdx.x - (warp < 4 ? 64 : 64 + L::kSoft);
            const int nk = args.nk, nkv = args.dhp >> 3;   // (padded to 16 channels)
            constexpr int kPer = (kKeys * KD / 8 + kStage - 1) / kStage;   // vectors of K, and of V, a thread
            Stager<kPer, kKeys, kAny> K, V;
            K.init(t, nkv, args.dkv, nk, p.dh, p.D, p.kfmt, L::kKvAtom);
            V.init(t, args.nv, args.dvv, args.nv, p.dvh, p.Dv, p.vfmt, L::kKvAtom);
            int it = 0, st = 0, nu = 0;
            uint32_t ph = 1;
            bool ok = true;
            for (int u = w.u_first; ok && u < w.units; u += w.u_step) {
                const Unit x = unit_at<kKeys>(p, w, u);
                const int n = x.c_hi - x.c_lo;
                if (n <= 0)
                    continue;
                const int64_t row0 = (int64_t)x.n * p.keys + (int64_t)x.c_lo * kKeys;   // the first chunk's first key
                K.start(p.kc, row0 * p.D + x.head * p.dh);
                V.start(p.vc, row0 * p.Dv + x.head * p.dvh);
                const float *ks = p.ks + row0 * p.kng + x.head * p.dh / p.kgroup;
                const float *vs = p.vs + row0 * p.vng + x.head * p.dvh / p.vgroup;
                const int left = x.keys - x.c_lo * kKeys;   // keys from the first chunk on
                constexpr int kSc = (2 * kKeys + kStage - 1) / kStage;
                float sr[kSc];
                auto fetch = [&](int i) {
                    const int nkeys = left - i * kKeys;
                    K.fetch(nkeys);
                    V.fetch(nkeys);
#pragma unroll
                    for (int e = 0; e < kSc; ++e) {
                        const int k = t + e * kStage, key = k & (kKeys - 1), row = i * kKeys + key;
                        sr[e] = 0.0f;
                        if (k < 2 * kKeys && key < nkeys)
                            sr[e] = k < kKeys ? __ldg(ks + (int64_t)row * p.kng) * args.sc : __ldg(vs + (int64_t)row * p.vng);
                    }
                };
                // the unit's queries, a row a thread, zeros for padding slots and channels
                if (nu > 0 && !wait_w<false>(bar + kBarQEmpty, (nu - 1) & 1, abort_flag, hdr, kSiteQEmpty))
                    break;
                for (int row = t; row < kRows << w.pairs; row += kStage) {
                    const int slot = x.slot0 + row;
                    const int64_t pix = slot < w.slots ? query_pixel(p, x.n, slot) : -1;
                    const uint32_t dst = sb + (row < kRows ? L::kOffQ : L::kOffQ2);
#pragma unroll 1
                    for (int g0 = 0; g0 < nkv; g0 += 4) {
                        uint4 q[4];
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            q[g] = make_uint4(0, 0, 0, 0);
                            if (pix >= 0 && g0 + g < nk) {
                                const __nv_bfloat16 *src = p.q + pix * p.D + x.head * p.dh + 8 * (g0 + g);
                                if constexpr (kAny)
                                    q[g] = bf16_any(src, p.dh - 8 * (g0 + g));
                                else
                                    q[g] = ld_nc16(src);
                            }
                        }
#pragma unroll
                        for (int g = 0; g < 4; ++g)
                            if (g0 + g < nkv)
                                sts128(dst + place(L::kQAtom, row & (kRows - 1), g0 + g), q[g]);
                    }
                }
                fence_async_smem();
                mbar_arrive(bar + kBarQFull);
                ++nu;
#pragma unroll 1
                for (int i = 0; i < n; ++i, ++it) {
                    if (i == 0)
                        fetch(0);
                    if (it >= L::kStages && !wait_w<false>(bar + kBarKvEmpty + 8u * st, ph, abort_flag, hdr, kSiteKvEmpty)) {
                        ok = false;
                        break;
                    }
                    const uint32_t kb = sb + L::kOffK + (uint32_t)st * L::kKvStage;
                    K.store(kb);
                    V.store(kb + L::kAtoms * L::kKvAtom);
                    bool big = false;
#pragma unroll
                    for (int e = 0; e < kSc; ++e) {
                        if (t + e * kStage < 2 * kKeys)
                            sts_f1(sb + L::kOffSc + (uint32_t)st * L::kScStage + (uint32_t)(t + e * kStage) * 4u, sr[e]);
                        big = big || (t + e * kStage >= kKeys && fabsf(sr[e]) >= kBigScale);
                    }
                    big = __any_sync(0xFFFFFFFFu, big);
                    if (lane == 0)
                        asm volatile("st.shared.u8 [%0], %1;" ::"r"(bar + kBig + 8u * st + (uint32_t)(t >> 5)), "r"((uint32_t)big)
                                     : "memory");
                    fence_async_smem();
                    mbar_arrive(bar + kBarKvFull + 8u * st);
                    if (i + 1 < n)
                        fetch(i + 1);
                    if (++st == L::kStages) {
                        st = 0;
                        ph ^= 1;
                    }
                }
            }
            __syncwarp();
        } else {
            // ---- products: warp 0 the scores, warp 1 the weighted values
            const bool scores = warp == 0;
            const uint32_t id_s = idesc_bf16(kKeys);
            // 64-channel blocks: of the last of them, the 16-channel steps of K and
            // the product's shape with V (B, MN-major)
            const int kb = (args.dhp + 63) / 64, vb = (args.dvp + 63) / 64;
            const int ks_last = args.dhp / 16 - 4 * (kb - 1);
            const uint32_t id_o = idesc_bf16(64) | (1u << 16), id_o_last = idesc_bf16(args.dvp - 64 * (vb - 1)) | (1u << 16);
            const uint64_t qd = desc_sw128(sb + L::kOffQ), q2d = desc_sw128(sb + (w.pairs ? L::kOffQ2 : L::kOffQ));
            const uint64_t kd = desc_sw128(sb + L::kOffK), vd = desc_sw128(sb + L::kOffK + L::kAtoms * L::kKvAtom);
            int st = 0, nu = 0;   // stage of the next job's chunk; units so far
            uint32_t ph = 0;
            // jobs of each group so far, mod 4, a byte each.  (The loops are one for
            // all groups: the warps of an SM share a small instruction cache, and
            // these instructions are on the path of every job.)
            uint32_t done = 0;
            bool ok = true;
            for (int u = w.u_first; ok && u < w.units; u += w.u_step) {
                const Unit x = unit_at<kKeys>(p, w, u);
                // job j of the unit: group j mod 2; chunk j, or chunk j / 2 of block
                // j mod 2
                const int jobs = (x.c_hi - x.c_lo) << w.pairs;
                if (jobs <= 0)
                    continue;
                if (scores && !wait_w<false>(bar + kBarQFull, nu & 1, abort_flag, hdr, kSiteQFull)) {
                    ok = false;
                    break;
                }
                ++nu;
#pragma unroll 1
                for (int j = 0; j < jobs; ++j) {
                    const uint32_t g = (uint32_t)j & 1u, n = (done >> (8 * g)) & 3u;
                    const uint32_t b = n & (L::kBufs - 1), buf = L::kBufs * g + b, par = (n / L::kBufs) & 1u;
                    done = (done + (1u << (8 * g))) & 0x03030303u;
                    if (scores) {
                        // (the group has read its last S, or the P V of the
                        // buffer's last job has landed)
                        if (!wait_w<false>(bar + kBarKvFull + 8u * st, ph, abort_flag, hdr, kSiteKvFull) ||
                            !wait_w<false>(bar + (L::kApart ? kBarSFree + 8u * g : kBarPvDone + 8u * buf), par ^ 1u, abort_flag,
                                           hdr, kSiteFree)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t ad = g ? q2d : qd, bd = kd + (uint64_t)((uint32_t)st * (L::kKvStage >> 4));
                        const uint32_t d = tmem + L::tmem_s(g, b);
#pragma unroll
                        for (int c = 0; c < L::kAtoms; ++c)
                            if (c < kb)
                                mma_s_w(d, ad + c * (L::kQAtom >> 4), bd + c * (L::kKvAtom >> 4), id_s, c > 0,
                                        c + 1 < kb ? 4 : ks_last);
                        tc_commit_w(bar + kBarSFull + 8u * buf);
                        if (j + 1 == jobs)
                            tc_commit_w(bar + kBarQEmpty);
                    } else {
                        if (!wait_w<false>(bar + kBarPFull + 8u * buf, par, abort_flag, hdr, kSitePFull)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t d = tmem + L::tmem_o(g), pa = tmem + L::tmem_p(g, b);
                        const uint64_t bd = vd + (uint64_t)((uint32_t)st * (L::kKvStage >> 4));
#pragma unroll
                        for (int k = 0; k < kKeys / 64; ++k)
#pragma unroll
                            for (int c = 0; c < L::kAtoms; ++c)
                                if (c < vb)
                                    mma_pv_w(d + 64u * c, pa + 32u * k, bd + c * (L::kKvAtom >> 4) + 512u * k,
                                             bd + c * (L::kKvAtom >> 4) + 512u * k + (k == 0 && x.keys <= kShort ? 0u : 256u),
                                             c + 1 < vb ? id_o : id_o_last, j >= 2 || k > 0);
                        tc_commit_w(bar + kBarPvDone + 8u * buf);
                        if (!w.pairs || g)
                            tc_commit_w(bar + kBarKvEmpty + 8u * st);
                    }
                    if (!w.pairs || g) {
                        ph ^= st + 1 == L::kStages;
                        st = st + 1 == L::kStages ? 0 : st + 1;
                    }
                }
            }
            if (!ok) {
                // the products in flight finish before this CTA's memory is given up
                const uint32_t drain = bar + kBarDrain + (scores ? 0u : 8u);
                tc_commit_w(drain);
                const long long t0 = clock64();
                while (!mbar_try(drain, 0) && clock64() - t0 < kWaitCycles / 64)
                    ;
            }
            __syncwarp();
        }
    } else {
        // ---- softmax: thread = query row r of group g
        constexpr int kG = 2, kSoft = L::kSoft;
        const int g = (warp >> 2) - 1, tid = (int)threadIdx.x - 128;
        const int r = (warp & 3) * 32 + lane;
        const uint32_t t_row = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t t_o = t_row + L::tmem_o(g);
        const int ng = args.nv;                // 8-channel groups of an output row
        int chunk = 0, m_it = 0;               // chunks of the CTA so far; jobs of this group
        bool ok = true;
        for (int u = w.u_first; u < w.units; u += w.u_step) {
            const Unit x = unit_at<kKeys>(p, w, u);
            const int n = (x.c_hi - x.c_lo) << w.pairs;   // jobs, every kG-th from g on this group's
            // of rows t / 4 + 8 j of the warp: the exponent base, and the sum over
            // this thread's keys
            float mq[4], lq[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                mq[j] = -INFINITY;
                lq[j] = 0.0f;
            }
            // one job; kTail: its chunk is the item's last, with keys to mask
            auto one = [&](int i, auto tail) {
                constexpr bool kTail = decltype(tail)::value;
                const int ci = chunk + (i >> w.pairs), b = m_it & (L::kBufs - 1);
                const int kvalid = x.keys - (x.c_lo + (i >> w.pairs)) * kKeys;
                // (the staged scales are seen through the stage's own barrier; its
                // next phase waits for this chunk's P V)
                if (!wait_w<false>(bar + kBarKvFull + 8u * (ci % L::kStages), (ci / L::kStages) & 1, abort_flag, hdr, kSiteKvFull) ||
                    !wait_w<false>(bar + kBarSFull + 8u * (L::kBufs * g + b), (m_it / L::kBufs) & 1, abort_flag, hdr, kSiteSFull)) {
                    ok = false;
                    return;
                }
                tc_fence_after();
                const uint32_t sc = sb + L::kOffSc + (uint32_t)(ci % L::kStages) * L::kScStage;
                // (kBigScale; read where it is needed: a register is dear)
                auto big = [&]() { return lds_2(bar + kBig + 8u * (uint32_t)(ci % L::kStages)) != 0; };
                const uint32_t t_s = t_row + L::tmem_s(g, b), t_p = t_row + L::tmem_p(g, b);
                // The scores are read in the fragment layout: a thread has a quarter
                // of the keys for four rows, so it reads a quarter of the scales,
                // once for the four.  (With a row a thread every lane reads every
                // scale: 512 bytes a key pair and warp through shared memory, which
                // bounded the kernel.)  Packed float32 instructions throughout.
                const uint32_t sq = sc + 8u * (uint32_t)(lane & 3);
                const int k0 = 2 * (lane & 3);
                // One pass: the weights are formed with the exponent base of the
                // group's jobs so far while the scores' maximum is found.  bf16 and
                // float32 weights keep their precision up to 2^kSlack above the
                // base, so the base moves (and the pass is run again) only when the
                // maximum has grown by more than that, or for the group's first job.
                float top[4];      // the job's largest score, less the base
                uint64_t ls[4];    // sums of weights
                auto pass = [&](auto first) {
                    constexpr bool kFirst = decltype(first)::value;   // the maximum only, of the scores themselves
                    uint64_t nm[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        nm[j] = kFirst ? 0 : pair(__float_as_uint(-mq[j]), __float_as_uint(-mq[j]));
                        top[j] = -INFINITY;
                        ls[j] = 0;
                    }
#pragma unroll 1
                    for (int h = 0; h < kKeys / 32; ++h) {
                        uint32_t sr[2][16], pk[2][8];
                        ld16x32(t_s + 32u * h, sr[0]);
                        ld16x32(t_s + 32u * h + (16u << 16), sr[1]);
                        ld_wait();
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint64_t s2 = lds_2(sq + 4u * (32 * h + 8 * q));
                            const uint64_t v2 = kFirst ? 0 : lds_2(sq + 4u * (kKeys + 32 * h + 8 * q));
                            const int kk = 32 * h + 8 * q + k0;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t *e = sr[j >> 1] + 4 * q + 2 * (j & 1);
                                const uint64_t d = kFirst ? mul2(pair(e[0], e[1]), s2) : fma2(pair(e[0], e[1]), s2, nm[j]);
                                float x0 = lo_of(d), x1 = hi_of(d);
                                if (kTail) {   // (masked keys: weight 0)
                                    x0 = kk < kvalid ? x0 : -INFINITY;
                                    x1 = kk + 1 < kvalid ? x1 : -INFINITY;
                                }
                                top[j] = fmaxf(top[j], fmaxf(x0, x1));
                                if constexpr (!kFirst) {
                                    const uint64_t w2 = pair(__float_as_uint(ex2(x0)), __float_as_uint(ex2(x1)));
                                    ls[j] = add2(ls[j], w2);
                                    const uint64_t y = mul2(w2, v2);
                                    pk[j >> 1][2 * q + (j & 1)] = pack_bf16x2(lo_of(y), hi_of(y));
                                }
                            }
                        }
                        if constexpr (!kFirst) {
                            st16x16(t_p + 16u * h, pk[0]);
                            st16x16(t_p + 16u * h + (16u << 16), pk[1]);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        top[j] = fmaxf(top[j], __shfl_xor_sync(0xFFFFFFFFu, top[j], 1));
                        top[j] = fmaxf(top[j], __shfl_xor_sync(0xFFFFFFFFu, top[j], 2));
                    }
                };
                // the weights of an item of at most kShort keys, in two terms
                auto brief = [&]() {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {   // (16 rows at a time: few registers)
                        uint32_t sr[16], hi[8], lo[8];
                        ld16x32(t_s + ((16u * half) << 16), sr);
                        ld_wait();
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint64_t s2 = lds_2(sq + 32u * q), v2 = lds_2(sq + 4u * (kKeys + 8 * q));
#pragma unroll
                            for (int i2 = 0; i2 < 2; ++i2) {
                                const int j = 2 * half + i2;
                                const uint32_t nm = __float_as_uint(-mq[j]);
                                const uint64_t d = fma2(pair(sr[4 * q + 2 * i2], sr[4 * q + 2 * i2 + 1]), s2, pair(nm, nm));
                                const float x0 = 8 * q + k0 < kvalid ? lo_of(d) : -INFINITY;
                                const float x1 = 8 * q + k0 + 1 < kvalid ? hi_of(d) : -INFINITY;
                                const uint64_t w2 = pair(__float_as_uint(ex2(x0)), __float_as_uint(ex2(x1)));
                                ls[j] = q == 0 ? w2 : add2(ls[j], w2);
                                const uint64_t y = mul2(w2, v2);
                                const uint32_t t = pack_bf16x2(lo_of(y), hi_of(y));
                                hi[2 * q + i2] = t;
                                lo[2 * q + i2] = pack_bf16x2(lo_of(y) - bf16_lo(t), hi_of(y) - bf16_hi(t));
                            }
                        }
                        const uint32_t to = t_p + ((16u * half) << 16);
                        st16x16(to, hi);
                        st16x16(to + 16u, lo);
                        if (kKeys > 64) {
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                hi[k] = 0;
                            st16x16(to + 32u, hi);
                            st16x16(to + 48u, hi);
                        }
                    }
                };
                // the group's previous P V has landed: P may be written, O rescaled.
                // (Each phase of the barrier is waited for in turn: a parity tells
                // two neighbouring phases apart, no more.)
                if (i >= kG) {
                    const int pb = (m_it - 1) & (L::kBufs - 1);
                    if (!wait_w<false>(bar + kBarPvDone + 8u * (L::kBufs * g + pb), ((m_it - 1) / L::kBufs) & 1, abort_flag, hdr,
                                       kSitePvDone)) {
                        ok = false;
                        return;
                    }
                    tc_fence_after();
                }
                // A first job has no base yet, and where P lies over the scores they
                // cannot be read again: the maximum first.  With large values the base
                // has to lie kRoom above it.
                bool move = i < kG || !L::kApart || big();
                if (move) {
                    pass(std::true_type());
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        top[j] -= i < kG ? 0.0f : mq[j];
                }
#pragma unroll 1
                while (true) {
                    if (move) {
                        float corr[4];
                        bool grow = false;
                        const bool wide = big();
                        const float room = wide ? kRoom : 0.0f;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            // (a first job: from -inf to its maximum; a row whose
                            // scores are all -inf or NaN keeps a base of -inf)
                            const bool up = i < kG || top[j] > (wide ? -kRoom : L::kApart ? 0.0f : 8.0f);
                            top[j] += room;
                            corr[j] = up && i >= kG ? ex2(-top[j]) : 1.0f;
                            if (up) {
                                mq[j] = i < kG ? top[j] : mq[j] + top[j];
                                lq[j] *= corr[j];
                                grow = grow || i >= kG;
                            }
                        }
                        if (__any_sync(0xFFFFFFFFu, grow)) {
                            const float f = of_row(corr, lane);
#pragma unroll 1
                            for (int pc = 0; pc < args.dvp; pc += 16) {
                                float v[16];
                                tmem_ld16(t_o + (uint32_t)pc, v);
#pragma unroll
                                for (int q = 0; q < 16; ++q)
                                    v[q] *= f;
                                st16(t_o + (uint32_t)pc, v);
                            }
                        }
                    }
                    if (kTail && x.keys <= kShort) {   // (one job, and the maximum is known)
                        brief();
                        break;
                    }
                    pass(std::false_type());
                    if (move || !__any_sync(0xFFFFFFFFu, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) > kSlack))
                        break;
                    move = true;
                }
                if (L::kApart) {   // the next S may come
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(bar + kBarSFree + 8u * g);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    lq[j] += lo_of(ls[j]) + hi_of(ls[j]);
                st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar + kBarPFull + 8u * (L::kBufs * g + b));
            };
            for (int i = g; ok && i < n; i += kG, ++m_it) {
                if (x.keys - (x.c_lo + (i >> w.pairs)) * kKeys >= kKeys)
                    one(i, std::false_type());
                else
                    one(i, std::true_type());
            }
            chunk += x.c_hi - x.c_lo;
            // the group's last P V of the unit has landed
            const bool mine = n > g;
            if (ok && mine)
                ok = wait_w<false>(bar + kBarPvDone + 8u * (L::kBufs * g + ((m_it - 1) & (L::kBufs - 1))), ((m_it - 1) / L::kBufs) & 1,
                                   abort_flag, hdr, kSitePvDone);
            tc_fence_after();
            // this thread's own row from here on
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                lq[j] += __shfl_xor_sync(0xFFFFFFFFu, lq[j], 1);
                lq[j] += __shfl_xor_sync(0xFFFFFFFFu, lq[j], 2);
            }
            const float m_used = of_row(mq, lane), l = of_row(lq, lane);
            if (w.split > 1) {
                // ---- merge of a split unit's kG s partial rows: each is pushed to
                // the CTA that owns the row, over the memory of the ring, once
                // every CTA of the unit has finished its products
                const int s = w.split, rows = kRows / s;   // (32 or more: a warp's rows have one owner)
                if (!joined) {
                    cluster_wait();
                    joined = true;
                }
                tc_fence_before();
                __syncwarp();
                if (lane < s)
                    mbar_arrive_peer(map_peer(bar + kBarReady, (uint32_t)(w.base + lane)));
                ok = wait_w<true>(bar + kBarReady, 0, abort_flag, hdr, kSiteReady) && ok;
                if (!ok)
                    continue;
                {
                    const int owner = r / rows;
                    const uint32_t slot = (uint32_t)((w.rank_split * kG + g) * rows + (r - owner * rows));   // of kSoft
                    const uint32_t dst = map_peer(sb + L::kOffPush + slot * 16u, (uint32_t)(w.base + owner));
#pragma unroll 1
                    for (int pc = 0; pc < args.dvp; pc += 16) {
                        float v[16];
                        if (mine)
                            tmem_ld16(t_o + (uint32_t)pc, v);
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            st_peer_f32x4(dst + (uint32_t)(pc / 4 + q) * (kSoft * 16u), mine ? v[4 * q] : 0.0f,
                                          mine ? v[4 * q + 1] : 0.0f, mine ? v[4 * q + 2] : 0.0f, mine ? v[4 * q + 3] : 0.0f);
                    }
                    st_peer_f32x2(map_peer(sb + L::kOffMl + slot * 8u, (uint32_t)(w.base + owner)), m_used, mine ? l : -1.0f);
                    __syncwarp();   // the warp's pushes, then one arrival that releases them
                    if (lane == 0)
                        mbar_arrive_peer(map_peer(bar + kBarPush, (uint32_t)(w.base + owner)));
                }
                if (!wait_w<true>(bar + kBarPush, 0, abort_flag, hdr, kSitePush)) {
                    ok = false;
                    continue;
                }
                for (int item = tid; item < rows * ng; item += kSoft) {
                    const int j = item % rows, gi = item / rows;
                    const int slot = x.slot0 + w.rank_split * rows + j;
                    const int64_t pix = slot < w.slots ? query_pixel(p, x.n, slot) : -1;
                    if (pix < 0)
                        continue;
                    float mm = -INFINITY;
                    for (int i = 0; i < kG * s; ++i)
                        mm = fmaxf(mm, lds_f2(sb + L::kOffMl + (uint32_t)(i * rows + j) * 8u).x);
                    float sum = 0.0f, acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                    for (int i = 0; i < kG * s; ++i) {
                        const float2 ml = lds_f2(sb + L::kOffMl + (uint32_t)(i * rows + j) * 8u);
                        if (ml.y == -1.0f)   // a part without a chunk
                            continue;
                        const float wt = ex2(ml.x - mm);
                        sum = fmaf(ml.y, wt, sum);
                        const uint32_t src = sb + L::kOffPush + (uint32_t)(i * rows + j) * 16u + (uint32_t)(2 * gi) * (kSoft * 16u);
                        const float4 y0 = lds_f4(src), y1 = lds_f4(src + kSoft * 16u);
                        acc[0] = fmaf(wt, y0.x, acc[0]); acc[1] = fmaf(wt, y0.y, acc[1]);
                        acc[2] = fmaf(wt, y0.z, acc[2]); acc[3] = fmaf(wt, y0.w, acc[3]);
                        acc[4] = fmaf(wt, y1.x, acc[4]); acc[5] = fmaf(wt, y1.y, acc[5]);
                        acc[6] = fmaf(wt, y1.z, acc[6]); acc[7] = fmaf(wt, y1.w, acc[7]);
                    }
                    put8<kAny>(p.o + pix * p.Dv + x.head * p.dvh + 8 * gi, acc, x.keys > 0 ? 1.0f / sum : 0.0f, p.dvh - 8 * gi);
                }
                continue;
            }
            // ---- the unit's rows
            const int slot = x.slot0 + (w.pairs ? (g & 1) * kRows : 0) + r;
            const int64_t pix = slot < w.slots ? query_pixel(p, x.n, slot) : -1;
            __nv_bfloat16 *dst = p.o + pix * p.Dv + x.head * p.dvh;
            if (w.pairs) {   // a block each: nothing to merge
                const float inv = mine ? 1.0f / l : 0.0f;   // (no key at all: zeros)
#pragma unroll 1
                for (int pc = 0; pc < args.dvp && ok; pc += 16) {
                    float v[16];
                    if (mine)
                        tmem_ld16(t_o + (uint32_t)pc, v);
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        v[q] = mine ? v[q] : 0.0f;
                    if (pix >= 0)
                        put8<kAny>(dst + pc, v, inv, p.dvh - pc);
                    if (pix >= 0 && pc / 8 + 1 < ng)
                        put8<kAny>(dst + pc + 8, v + 8, inv, p.dvh - pc - 8);
                }
                tc_fence_before();
                continue;
            }
            // the two groups share the block: each keeps the 8-channel groups of
            // its parity and merges them with the other's copy of them, 64
            // channels at a time
            const int pt = (g ^ 1) * kGroup + r;
            float wa = 0.0f, wb = 0.0f, inv = 0.0f;
            bool both = false;   // neither group's wait has expired
#pragma unroll 1
            for (int p0 = 0; p0 < args.dvp; p0 += 64) {
                float o[32];
                soft_sync<kSoft>();   // the last rows have been read
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float v[16];
                    const bool in = ok && mine && p0 + 16 * k < args.dvp;
                    if (in)
                        tmem_ld16(t_o + (uint32_t)(p0 + 16 * k), v);
                    const uint32_t at = sb + L::kOffX + (uint32_t)(2 * k * kSoft + tid) * 16u;
                    float m[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const float a = in ? v[q] : 0.0f, c = in ? v[8 + q] : 0.0f;
                        m[q] = g ? a : c;
                        o[8 * k + q] = g ? c : a;
                    }
                    sts_f4(at, m);
                    sts_f4(at + kSoft * 16u, m + 4);
                }
                if (p0 == 0)   // (a sum of -1: no key; -2: a wait expired, the row is not written)
                    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(sb + L::kOffMl + (uint32_t)tid * 8u), "f"(m_used),
                                 "f"(!ok ? -2.0f : mine ? l : -1.0f) : "memory");
                soft_sync<kSoft>();
                if (p0 == 0) {
                    const float2 ml = lds_f2(sb + L::kOffMl + (uint32_t)pt * 8u);
                    const bool other = ml.y != -1.0f;
                    both = ok && ml.y != -2.0f;
                    const float mm = fmaxf(mine ? m_used : -INFINITY, other ? ml.x : -INFINITY);
                    wa = mine ? ex2(m_used - mm) : 0.0f;
                    wb = other ? ex2(ml.x - mm) : 0.0f;
                    const float sum = (mine ? l * wa : 0.0f) + (other ? ml.y * wb : 0.0f);
                    inv = mine || other ? 1.0f / sum : 0.0f;   // (no key at all: zeros)
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int gi = p0 / 8 + 2 * k + g;
                    if (both && pix >= 0 && gi < ng) {
                        const uint32_t src = sb + L::kOffX + (uint32_t)(2 * k * kSoft + pt) * 16u;
                        const float4 y0 = lds_f4(src), y1 = lds_f4(src + kSoft * 16u);
                        float *oo = o + 8 * k;
                        oo[0] = fmaf(y0.x, wb, oo[0] * wa); oo[1] = fmaf(y0.y, wb, oo[1] * wa);
                        oo[2] = fmaf(y0.z, wb, oo[2] * wa); oo[3] = fmaf(y0.w, wb, oo[3] * wa);
                        oo[4] = fmaf(y1.x, wb, oo[4] * wa); oo[5] = fmaf(y1.y, wb, oo[5] * wa);
                        oo[6] = fmaf(y1.z, wb, oo[6] * wa); oo[7] = fmaf(y1.w, wb, oo[7] * wa);
                        put8<kAny>(dst + 8 * gi, oo, inv, p.dvh - 8 * gi);
                    }
                }
            }
            tc_fence_before();
        }
    }
    if (!joined)
        cluster_wait();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
    }
    // no CTA leaves while a peer may still address its shared memory
    cluster_arrive();
    cluster_wait();
}

// ------------------------------------------------------------------ host

bool attention_qcache_tc_scope(int dh, int dvh) { return dh > 0 && dvh > 0 && dh <= 192 && dvh <= 192; }

template <int KD, bool kAny>
static int launch_kd(const at::Args &a, int64_t units_max, cudaStream_t stream)
{
    constexpr auto kernel = k_attn_qcache_tc<KD, kAny>;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return SIGE_ERR_CUDA;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = at::kCluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(at::Lay<KD>::kThreads);
    cfg.dynamicSmemBytes = at::Lay<KD>::kBytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    static std::atomic<int> clusters_of[64];   // co-resident clusters, per device
    int ncl = clusters_of[dev].load(std::memory_order_acquire);
    if (ncl == 0) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)at::Lay<KD>::kBytes) != cudaSuccess) {
            cudaGetLastError();
            return SIGE_ERR_CUDA;
        }
        cfg.gridDim = dim3(at::kCluster * (device_sm_count() / at::kCluster));
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&ncl, kernel, &cfg) != cudaSuccess || ncl < 1) {
            cudaGetLastError();
            return SIGE_ERR_CUDA;
        }
        clusters_of[dev].store(ncl, std::memory_order_release);
    }
    prefer_max_shared_of<kernel>();
    cfg.numAttrs = 2;
    // every unit a launch can have needs at most one cluster
    cfg.gridDim = dim3((unsigned)(at::kCluster * std::max<int64_t>(1, std::min<int64_t>(ncl, units_max))));
    if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) {
        cudaGetLastError();
        return SIGE_ERR_CUDA;
    }
    count_launch();
    return launch_check();
}

int launch_attention_qcache_tc(const AttnQParams &p, cudaStream_t stream)
{
    if (!attention_qcache_tc_scope(p.dh, p.dvh))
        return 1;
    const int64_t units_max = (p.slots + at::kRows - 1) / at::kRows * p.N * p.heads;
    // (units and the bytes of a chunk's rows are counted in 32 bits)
    if (units_max > INT32_MAX / 16 || p.D > (1 << 24) || p.Dv > (1 << 24))
        return 1;
    at::Args a{};
    a.a = p;
    a.dhp = (p.dh + 15) / 16 * 16;
    a.dvp = (p.dvh + 15) / 16 * 16;
    a.nk = (p.dh + 7) / 8;
    a.nv = (p.dvh + 7) / 8;
    a.sc = (float)(1.4426950408889634 / std::sqrt((double)p.dh));
    a.dkv = udiv_make((uint32_t)(a.dhp / 8));
    a.dvv = udiv_make((uint32_t)a.nv);
    // 16-byte query and output vectors, 8 codes at once, or element by element
    const bool any = p.dh % 8 || p.dvh % 8 || !aligned_to(p.q, 16) || !aligned_to(p.o, 16) ||
                     !aligned_to(p.kc, p.kfmt == SIGE_Q_S4 ? 4 : 8) || !aligned_to(p.vc, p.vfmt == SIGE_Q_S4 ? 4 : 8);
    const int kd = std::max(a.dhp, a.dvp);
    if (any)
        return kd <= 64    ? launch_kd<64, true>(a, units_max, stream)
               : kd <= 128 ? launch_kd<128, true>(a, units_max, stream)
                           : launch_kd<192, true>(a, units_max, stream);
    return kd <= 64    ? launch_kd<64, false>(a, units_max, stream)
           : kd <= 128 ? launch_kd<128, false>(a, units_max, stream)
                       : launch_kd<192, false>(a, units_max, stream);
}

} // namespace sige
