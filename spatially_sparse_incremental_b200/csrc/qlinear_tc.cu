// Product of 8-bit integers on the tensor cores (sige_qlinear): the integer
// sums by tcgen05.mma kind::i8 (exact, int32 in tensor memory), the two scales,
// bias and residual in the epilogue, one rounding into the cached output.
//
// A work unit is 128 tokens x `bn` (256 .. 32) output channels, K in chunks of
// 128 bytes (four MMAs of 32).  bn and the K split depend on the number of
// tokens, which only the device knows for a tile list, so every CTA derives
// them at its start.
//   * warp 0 loads the operands by TMA into a ring of stages, 128-byte rows
//     with the 128-byte swizzle (the K-major operands of the MMA): weights and
//     whole maps by boxes of rows, the tokens of a tile list straight from the
//     cache, a 4 x 4 or 8 x 8 tile a box or (other tiles) four tokens a
//     tile::gather4, one copy a lane;
//   * warp 1 issues the MMAs into one of two accumulators of up to 256
//     columns, so that the next unit's products run under this one's epilogue;
//   * warps 2 .. 9 (two warps to each quarter of the tensor memory's lanes,
//     each with half of the columns) finish the outputs.
// Where units are few and K is long (cut_cost), a cluster's CTAs split a unit's K
// chunks and exchange their int32 sums through distributed shared memory, each
// finishing a slice of the columns; integer sums do not depend on the split.
// 20 tokens of a list x 5120 -> 1280: 10.2 us, 21.0 without; one token of a map
// 6.6 and 8.4.
//
// k_qlinear_whole is the same for whole maps (16384 x 640 -> 5120 61 us, 72 by
// the general kernel; 1280 -> 320 with residual 10.3 and 13.7; 16 tokens x 1280 ->
// 1280 4.0 and 5.1), k_qlinear_staged for codes that TMA cannot copy.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "qlinear.cuh"
#include "tc_ptx.cuh"

namespace sige {
namespace qt {

constexpr int kEpiWarps = 8;
constexpr int kEpiThreads = 32 * kEpiWarps;
constexpr int kThreads = 64 + kEpiThreads;
constexpr int kRows = 128;
constexpr int kChunk = 128;              // bytes of K a stage
constexpr int kMaxBn = 256;
constexpr int kSplitBn = 64;             // widest unit whose K is split
constexpr int kCluster = 4;
constexpr int kMaxStages = 9;

constexpr uint32_t kRing = 196608;       // 4 stages of 128 + 256 rows, more of narrower ones
constexpr uint32_t kOffRecv = kRing;     // sums pushed by the other CTAs of a split unit (k_qlinear_whole: the
                                         // output tiles of the warps)
constexpr uint32_t kRecvBytes = (kCluster - 1) * kRows * (kSplitBn / kCluster) * 4;
constexpr uint32_t kOffCol = kOffRecv + kRecvBytes;          // per accumulator: column scales and biases
constexpr uint32_t kOffBar = kOffCol + 2 * 2 * kMaxBn * 4;
constexpr uint32_t kBarFull = 0;                             // + 8 stage
constexpr uint32_t kBarEmpty = 8 * kMaxStages;
constexpr uint32_t kBarAccFull = 16 * kMaxStages;            // + 8 accumulator
constexpr uint32_t kBarAccEmpty = kBarAccFull + 16;
constexpr uint32_t kBarRecv = kBarAccEmpty + 16;
constexpr uint32_t kBarDrain = kBarRecv + 8;
constexpr uint32_t kTmemSlot = kBarDrain + 8;
constexpr uint32_t kAbort = kTmemSlot + 4;
constexpr uint32_t kSmem = kOffBar + 256 + 1024;             // + alignment slack
static_assert(kEpiWarps * 2048 <= kRecvBytes, "output tiles");
static_assert(kAbort + 4 <= 256, "barrier block");
static_assert(kSmem <= 227 * 1024, "shared memory");

// wait sites (the detail of a recorded SIGE_ERR_TIMEOUT)
constexpr int kSiteEmpty = 301, kSiteFull = 302, kSiteAccEmpty = 303, kSiteAccFull = 304, kSiteRecv = 305;

struct Plan {
    int bn, stages, split, nch;
    uint32_t slots, rblocks, cblocks, units;
};

__host__ __device__ inline int least(int a, int b) { return a < b ? a : b; }

// How a product of many tokens is cut: candidate i < 8 is units of 32 (i + 1)
// columns, then 64 columns with K split 2 and 4 ways and 32 columns split 2
// ways (16 columns or more for each CTA to finish).
constexpr int kCuts = 11;
__host__ __device__ inline void cut_at(int i, int *bn, int *split)
{
    *bn = i < 8 ? 32 * (i + 1) : i == 10 ? 32 : 64;
    *split = i < 8 ? 1 : i == 9 ? 4 : 2;
}

// What a call's kind adds: cycles of a token row of a chunk (copied by boxes, or
// gathered four a copy, about 60 a copy) and of a split's exchange (a whole map
// gives up k_qlinear_whole for it: 16 tokens x 1280 -> 1280 4.2 us, split 5.9).
struct Costs {
    uint32_t token, split;
};
constexpr Costs kMapCosts = {2, 4300};
__host__ __device__ inline Costs list_costs(int tile_rows) { return {tile_rows ? 2u : 15u, 1300}; }

// Estimated cycles of a cut: rounds of units, each the longer of its chunks and
// its outputs (about 12 cycles a column); a fill and a drain; the exchange of a
// split, by quarters of 32 rows.  A chunk: the operands' way into shared memory
// at about 60 bytes a cycle (measured longer than the products, 2 bn cycles);
// 250 for the issue of a small one.  rows: tokens of a unit.  0xFFFFFFFF: not
// possible.
__host__ __device__ inline uint32_t cut_cost(int i, uint32_t rblocks, int rows, Costs k, int Co, int nch, int grid, int cluster)
{
    int bn, split;
    cut_at(i, &bn, &split);
    const uint32_t units = rblocks * (((uint32_t)Co + bn - 1) / bn);
    if (split > cluster || (split > 1 && (units * (uint32_t)split > (uint32_t)grid || nch < 2 * split)))
        return 0xFFFFFFFFu;
    const uint32_t rounds = (units * (uint32_t)split + grid - 1) / grid;
    uint32_t chunk = (uint32_t)bn * 17u / 8u + (uint32_t)rows * k.token;
    chunk = chunk < 250u ? 250u : chunk;
    const uint32_t mul = (uint32_t)((nch + split - 1) / split) * chunk, out = 12u * (uint32_t)bn;
    const uint32_t exchange = split > 1 ? k.split + 300u * (uint32_t)((rows + 31) / 32) : 0u;
    const float c = (float)rounds * (float)(mul > out ? mul : out) + (float)(1000u + out / split + exchange);
    return c < 2e9f ? (uint32_t)c : 2000000000u;
}

// The launch's work for `slots` tokens on `grid` CTAs in clusters of `cluster`.  On the device the whole warp calls it: a lane
// prices each cut.
__host__ __device__ inline Plan make_plan(uint32_t slots, Costs k, int Co, int C, int grid, int cluster)
{
    Plan q;
    q.slots = slots;
    q.nch = (C + kChunk - 1) / kChunk;
    q.rblocks = (slots + kRows - 1) / kRows;
    const int rows = slots < (uint32_t)kRows ? (int)slots : kRows;
#ifdef __CUDA_ARCH__
    const int lane = (int)(threadIdx.x & 31);
    const uint32_t mine = cut_cost(least(lane, kCuts - 1), q.rblocks, rows, k, Co, q.nch, grid, cluster);
    const int best = __ffs(__ballot_sync(0xFFFFFFFFu, mine == __reduce_min_sync(0xFFFFFFFFu, mine))) - 1;
#else
    int best = 0;
    for (int i = 1; i < kCuts; ++i)
        if (cut_cost(i, q.rblocks, rows, k, Co, q.nch, grid, cluster) <
            cut_cost(best, q.rblocks, rows, k, Co, q.nch, grid, cluster))
            best = i;
#endif
    cut_at(best, &q.bn, &q.split);
    q.cblocks = ((uint32_t)Co + q.bn - 1) / q.bn;
    q.units = q.rblocks * q.cblocks;
    q.stages = q.bn > 128 ? 4 : q.bn > 64 ? 6 : q.bn > 32 ? 8 : 9;
    return q;
}
static_assert(4 * (kRows + 256) * kChunk <= kRing && 6 * (kRows + 128) * kChunk <= kRing &&
              8 * (kRows + 64) * kChunk <= kRing && 9 * (kRows + 32) * kChunk <= kRing && 9 <= kMaxStages, "ring");

// kind::i8, A and B signed, D int32, both K-major, M = 128.
__device__ __forceinline__ uint32_t idesc_s8(int n)
{
    return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// The `steps` (1 .. 4) products of a stage, 32 channels each (32 bytes along the
// swizzled rows), and the commit that releases the stage, from one elected lane
// of the converged warp.
__device__ __forceinline__ void mma_s8_commit_w(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate,
                                                int steps, uint32_t bar)
{
    asm volatile(
        "{\n .reg .pred p, e, t, e1, e2, e3;\n .reg .b32 l;\n .reg .b64 a1, a2, a3, b1, b2, b3;\n"
        " elect.sync l|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n setp.eq.b32 t, 0, 0;\n"
        " setp.gt.and.s32 e1, %5, 1, e;\n setp.gt.and.s32 e2, %5, 2, e;\n setp.gt.and.s32 e3, %5, 3, e;\n"
        " add.s64 a1, %1, 2;\n add.s64 a2, %1, 4;\n add.s64 a3, %1, 6;\n"
        " add.s64 b1, %2, 2;\n add.s64 b2, %2, 4;\n add.s64 b3, %2, 6;\n"
        " @e tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n"
        " @e1 tcgen05.mma.cta_group::1.kind::i8 [%0], a1, b1, %3, t;\n"
        " @e2 tcgen05.mma.cta_group::1.kind::i8 [%0], a2, b2, %3, t;\n"
        " @e3 tcgen05.mma.cta_group::1.kind::i8 [%0], a3, b3, %3, t;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%6];\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(steps), "r"(bar)
        : "memory");
}

// A whole stage from two boxes (128 bytes of K from byte x on, rows ya and yb)
// and the bytes its barrier waits for, from one elected lane of the converged
// warp.
__device__ __forceinline__ void tma_stage_w(uint32_t da, const CUtensorMap *ma, int ya, uint32_t db, const CUtensorMap *mb,
                                            int yb, uint32_t bar, uint32_t bytes, int x)
{
    asm volatile(
        "{\n .reg .pred e;\n .reg .b32 l;\n elect.sync l|e, 0xffffffff;\n"
        " @e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%6], %7;\n"
        " @e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%8, %2}], [%6];\n"
        " @e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%3], [%4, {%8, %5}], [%6];\n}\n"
        ::"r"(da), "l"(reinterpret_cast<uint64_t>(ma)), "r"(ya), "r"(db), "l"(reinterpret_cast<uint64_t>(mb)), "r"(yb),
        "r"(bar), "r"(bytes), "r"(x)
        : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2, int c3)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
                 : "memory");
}

// Four rows of the token map into four 128-byte rows of a stage.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int r0, int r1,
                                            int r2, int r3)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(r0), "r"(r1), "r"(r2), "r"(r3)
                 : "memory");
}

// n columns of this warp's 32 tensor-memory lanes, without a wait.
__device__ __forceinline__ void ld_cols(uint32_t taddr, int (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void ld_done() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void st_peer_s32x4(uint32_t addr, int a, int b, int c, int d)
{
    asm volatile("st.shared::cluster.v4.s32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
__device__ __forceinline__ int4 lds_s32x4(uint32_t addr)
{
    int4 v;
    asm volatile("ld.shared.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ float4 lds_f32x4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kEpiThreads) : "memory"); }

// After a wait that expired: the copies in flight (the last of `it` issued) land,
// and the products in flight finish, before the CTA's memory is given up; both
// bounded.
__device__ __noinline__ void drain_copies(uint32_t bar, int it, int stages)
{
    for (int i = 0; i < min(it, stages); ++i) {
        const int k = it - 1 - i, s = k % stages;
        const long long t0 = clock64();
        while (!mbar_try(bar + kBarFull + 8u * s, (k / stages) & 1) && clock64() - t0 < kWaitCycles / 64)
            ;
    }
}
__device__ __noinline__ void drain_products(uint32_t bar)
{
    tc_commit_w(bar + kBarDrain);
    const long long t0 = clock64();
    while (!mbar_try(bar + kBarDrain, 0) && clock64() - t0 < kWaitCycles / 64)
        ;
}

struct Args {
    QLinearParams q;
    int vec;       // y and the residual take 32-byte accesses of 16 columns
    int width;     // elements of y an access takes otherwise (put_rows)
    int tile_rows; // tokens that one box copies (a tile's; a whole map's of a unit), 0: four tokens a copy
    Plan plan;     // of a whole map (a list's is made on the device)
};

// 16 sums of one token, scaled and biased: scales and biases from shared
// memory (col: kMaxBn scales, then kMaxBn biases).  kBig: sa may be a large scale
// (is_big).
template <bool kBig>
__device__ __forceinline__ void scale16(const int *acc, uint32_t col, float sa, float *v)
{
    const TokenScale t = kBig ? token_scale(sa) : TokenScale{sa, 1.0f};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float4 s = lds_f32x4(col + 16u * q), b = lds_f32x4(col + 4u * kMaxBn + 16u * q);
        v[4 * q] = qlinear_value(acc[4 * q], t, s.x, b.x);
        v[4 * q + 1] = qlinear_value(acc[4 * q + 1], t, s.y, b.y);
        v[4 * q + 2] = qlinear_value(acc[4 * q + 2], t, s.z, b.z);
        v[4 * q + 3] = qlinear_value(acc[4 * q + 3], t, s.w, b.w);
    }
}

// 32 bytes (a whole memory sector).
__device__ __forceinline__ void st_v8(void *dst, const uint32_t *v)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void ld_v8(const void *src, uint32_t *v)
{
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "l"(src));
}

// The outputs of a whole map leave through shared memory and TMA: v holds 64
// bytes of columns (32 bf16 or 16 float32) of this lane's row, tile 2 KB of the
// warp, the rows' 16-byte pieces at piece ^ ((row / 2) mod 4) (the 64-byte
// swizzle of the output map, and no bank conflicts).  Storing them from the
// registers, 32 bytes of 32 different lines an instruction, bounded a call of
// wide outputs (16384 x 640 x 5120: 73 us, 45 us without the stores).
template <int kE>   // bytes of an output element
__device__ __forceinline__ void put_tile(const float *v, uint32_t tile, const CUtensorMap *map, int col, int row, int lane)
{
    // the previous tile has been read
    if (lane == 0)
        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
    const uint32_t own = tile + 64u * lane, sw = (uint32_t)(lane >> 1) & 3u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint4 x;
        if constexpr (kE == 2) {
            const float *u = v + 8 * k;
            x = make_uint4(pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]), pack_bf16x2(u[4], u[5]), pack_bf16x2(u[6], u[7]));
        } else {
            x = make_uint4(__float_as_uint(v[4 * k]), __float_as_uint(v[4 * k + 1]), __float_as_uint(v[4 * k + 2]),
                           __float_as_uint(v[4 * k + 3]));
        }
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(own + (((uint32_t)k ^ sw) << 4)), "r"(x.x), "r"(x.y),
                     "r"(x.z), "r"(x.w)
                     : "memory");
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0)
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];\n"
                     "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
                     "r"(tile), "r"(col), "r"(row)
                     : "memory");
}

// + residual, for 16 columns of one token from element e on (32-byte aligned).
__device__ __forceinline__ void add_residual16(const QLinearParams &p, int64_t e, float *v)
{
    uint32_t w[8];
    if (p.dtype == SIGE_BF16) {
        ld_v8(p.residual + e * 2, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            v[2 * k] += bf16_lo(w[k]);
            v[2 * k + 1] += bf16_hi(w[k]);
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            ld_v8(p.residual + e * 4 + 32 * h, w);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[8 * h + k] += __uint_as_float(w[k]);
        }
    }
}

// 16 outputs of one token (y and the residual at element e, 32-byte aligned
// rows): a thread writes whole sectors of its own row.
__device__ __forceinline__ void put16(const QLinearParams &p, int64_t e, float *v)
{
    if (p.residual)
        add_residual16(p, e, v);
    uint32_t w[8];
    if (p.dtype == SIGE_BF16) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            w[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
        st_v8(p.y + e * 2, w);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                w[k] = __float_as_uint(v[8 * h + k]);
            st_v8(p.y + e * 4 + 32 * h, w);
        }
    }
}

// 16 columns from c on of a warp's 32 rows, where a row's columns are no whole
// sectors (or not all there): lane r leaves row r's values in shared memory (2 KB
// of the warp, 16-byte pieces at piece ^ ((row / 2) mod 4)), then neighbouring
// lanes take neighbouring columns, kW elements each.  A lane for each row's
// columns stored 2 bytes of 32 different lines an instruction: 16384 x 640 ->
// 5112 812 us.
template <int kE, int kW>
__device__ __noinline__ void put_rows_as(const QLinearParams &p, uint32_t tile, int pix, int col)
{
    constexpr int kLanes = 16 / kW;   // of a row
    constexpr int kRowsAt = 32 / kLanes, kPass = 32 / kRowsAt, kGo = kPass < 8 ? kPass : 8;   // passes under way at once
    const int lane = (int)(threadIdx.x & 31), c = col + (lane % kLanes) * kW;
    const uint32_t k0 = (uint32_t)(c - col);
#pragma unroll 1
    for (int r0 = 0; r0 < 32; r0 += kGo * kRowsAt) {
        float v[kGo][kW];
        int64_t e[kGo];   // byte offset, -1: nothing to store
#pragma unroll
        for (int i = 0; i < kGo; ++i) {
            const int row = r0 + i * kRowsAt + lane / kLanes, at = __shfl_sync(0xFFFFFFFFu, pix, row);
            e[i] = at < 0 || c >= p.Co ? -1 : ((int64_t)at * p.Co + c) * kE;
            const uint32_t src = tile + 64u * (uint32_t)row, sw = (uint32_t)(row >> 1) & 3u;
            if constexpr (kW >= 4) {
#pragma unroll
                for (int k = 0; k < kW / 4; ++k) {
                    const float4 x = lds_f32x4(src + (((k0 / 4 + k) ^ sw) << 4));
                    v[i][4 * k] = x.x; v[i][4 * k + 1] = x.y; v[i][4 * k + 2] = x.z; v[i][4 * k + 3] = x.w;
                }
            } else {
#pragma unroll
                for (int k = 0; k < kW; ++k)
                    asm volatile("ld.shared.f32 %0, [%1];"
                                 : "=f"(v[i][k]) : "r"(src + (((k0 / 4) ^ sw) << 4) + 4u * (k0 % 4 + k)) : "memory");
            }
        }
        if (p.residual) {
            uint4 w[kGo];
#pragma unroll
            for (int i = 0; i < kGo; ++i) {
                w[i] = make_uint4(0, 0, 0, 0);
                if (e[i] >= 0) {
                    if constexpr (kE * kW == 16)
                        w[i] = *reinterpret_cast<const uint4 *>(p.residual + e[i]);
                    else if constexpr (kE * kW == 4)
                        w[i].x = *reinterpret_cast<const uint32_t *>(p.residual + e[i]);
                    else
                        w[i].x = *reinterpret_cast<const uint16_t *>(p.residual + e[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < kGo; ++i) {
                const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                for (int k = 0; k < kW; ++k)
                    v[i][k] += kE == 4 ? __uint_as_float(x[k & 3]) : k & 1 ? bf16_hi(x[k >> 1]) : bf16_lo(x[k >> 1]);
            }
        }
#pragma unroll
        for (int i = 0; i < kGo; ++i) {
            if (e[i] < 0)
                continue;
            uint8_t *dst = p.y + e[i];
            const float *u = v[i];
            if constexpr (kE == 2 && kW == 8)
                *reinterpret_cast<uint4 *>(dst) = make_uint4(pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]),
                                                             pack_bf16x2(u[4], u[5]), pack_bf16x2(u[6], u[7]));
            else if constexpr (kE == 4 && kW == 4)
                *reinterpret_cast<float4 *>(dst) = make_float4(u[0], u[1], u[2], u[3]);
            else if constexpr (kE == 2 && kW == 2)
                *reinterpret_cast<uint32_t *>(dst) = pack_bf16x2(u[0], u[1]);
            else if constexpr (kE == 2)
                *reinterpret_cast<__nv_bfloat16 *>(dst) = __float2bfloat16_rn(u[0]);
            else
                *reinterpret_cast<float *>(dst) = u[0];
        }
    }
    __syncwarp();
}
__device__ __noinline__ void put_rows(const Args &a, uint32_t tile, int pix, int col)
{
    const QLinearParams &p = a.q;
    if (p.dtype == SIGE_BF16) {
        if (a.width == 8)
            put_rows_as<2, 8>(p, tile, pix, col);
        else if (a.width == 2)
            put_rows_as<2, 2>(p, tile, pix, col);
        else
            put_rows_as<2, 1>(p, tile, pix, col);
    } else {
        if (a.width == 4)
            put_rows_as<4, 4>(p, tile, pix, col);
        else
            put_rows_as<4, 1>(p, tile, pix, col);
    }
}
// The widest access of put_rows: aligned at every row, and a divisor of the columns.
inline int row_width(const QLinearParams &p)
{
    const int esz = p.dtype == SIGE_BF16 ? 2 : 4;
    for (int w = 16 / esz; w > 1; w = w == 8 ? 2 : 1)
        if (p.Co % w == 0 && aligned_to(p.y, (uintptr_t)(w * esz)) && aligned_to(p.residual, (uintptr_t)(w * esz)))
            return w;
    return 1;
}

// 16 columns from c on of the warp's tokens (pix: this lane's, -1: none): whole
// sectors of a lane's own row, or put_rows.
__device__ __forceinline__ void put_cols(const Args &a, float *v, int64_t pix, int c, uint32_t tile)
{
    if (a.vec && c + 16 <= a.q.Co) {
        if (pix >= 0)
            put16(a.q, pix * a.q.Co + c, v);
    } else if (c < a.q.Co) {
        const int lane = (int)(threadIdx.x & 31);
        const uint32_t own = tile + 64u * (uint32_t)lane, sw = (uint32_t)(lane >> 1) & 3u;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(own + (((uint32_t)k ^ sw) << 4)), "f"(v[4 * k]),
                         "f"(v[4 * k + 1]), "f"(v[4 * k + 2]), "f"(v[4 * k + 3])
                         : "memory");
        __syncwarp();
        put_rows(a, tile, (int)pix, c);
    }
}

} // namespace qt

using namespace qt;

__global__ void __launch_bounds__(qt::kThreads, 1)
    k_qlinear_tc(const __grid_constant__ qt::Args args, const __grid_constant__ CUtensorMap tw,
                 const __grid_constant__ CUtensorMap tw64, const __grid_constant__ CUtensorMap tw32,
                 const __grid_constant__ CUtensorMap tbox)
{
    extern __shared__ __align__(1024) uint8_t qt_raw[];
    const QLinearParams &p = args.q;
    const uint32_t raw = smem_u32(qt_raw);
    const uint32_t sb = (raw + 1023u) & ~1023u;
    uint8_t *smem = qt_raw + (sb - raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t bar = sb + kOffBar;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOffBar + kAbort);
    WsHeader *hdr = p.hdr;
    uint32_t csize;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(csize));

    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(bar + kBarFull + 8u * i, 1);
            mbar_init(bar + kBarEmpty + 8u * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar + kBarAccFull + 8u * i, 1);
            mbar_init(bar + kBarAccEmpty + 8u * i, kEpiWarps);
        }
        mbar_init(bar + kBarDrain, 1);
        *abort_flag = 0;
    }
    if (warp == 0 && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tw)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tbox)) : "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(bar + kTmemSlot),
                     "r"(2 * kMaxBn));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    pdl_wait();
    const Plan plan = p.px.idx ? make_plan((uint32_t)pixel_slots(p.px), list_costs(args.tile_rows), p.Co, p.C, (int)gridDim.x, (int)csize)
                               : args.plan;
    const int split_n = plan.split;
    const int per = (int)csize / split_n;                  // units a cluster takes at a time
    const int rank = csize > 1 ? (int)cluster_rank() : 0;
    const int sub = rank / split_n, split = rank - sub * split_n;
    const uint32_t u_first = (blockIdx.x / csize) * (uint32_t)per + (uint32_t)sub;
    const uint32_t u_step = (gridDim.x / csize) * (uint32_t)per;
    const int c_lo = split * plan.nch / split_n, c_hi = (split + 1) * plan.nch / split_n;   // never empty
    if (threadIdx.x == 0) {
        // pushed by the warps of the unit's other CTAs whose rows hold a token
        const uint32_t left = u_first < plan.units ? plan.slots - u_first / plan.cblocks * kRows : 0;
        mbar_init(bar + kBarRecv, max(1u, (uint32_t)(split_n - 1) * (kEpiWarps / 4) * min(4u, (left + 31) / 32)));
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + kOffBar + kTmemSlot);
    // the peers' barriers are initialised before the first push
    if (csize > 1)
        cluster_arrive();
    bool joined = false;

    const uint32_t stage_bytes = (uint32_t)(kRows + plan.bn) * kChunk;
    if (warp == 0) {
        // ---- operands
        const bool lists = p.px.idx != nullptr;
        const bool tiles = lists && args.tile_rows;   // whole tiles by boxes
        // weight rows: one box for a whole map; for a list (whose bn the host
        // does not know) boxes of 128, 64 and 32, one a lane
        const int n128 = plan.bn >> 7, n64 = (plan.bn >> 6) & 1, nw = n128 + n64 + ((plan.bn >> 5) & 1);
        const CUtensorMap *wmap = lane < n128 ? &tw : lane < n128 + n64 ? &tw64 : &tw32;
        const int wofs = lane < n128 ? 128 * lane : lane < n128 + n64 ? 128 * n128 : 128 * n128 + 64 * n64;
        constexpr uint32_t wdst = kRows * kChunk;          // weights behind the tokens
        const int per_copy = tiles ? args.tile_rows : 4;   // tokens a copy of a list, one copy a lane
        int it = 0, st = 0;
        uint32_t ph = 1;
        bool ok = true;
        for (uint32_t u = u_first; ok && u < plan.units; u += u_step) {
            const uint32_t rb = u / plan.cblocks;
            const int cb = (int)(u - rb * plan.cblocks);
            const int wrow = cb * plan.bn;
            const uint32_t s_first = rb * kRows;
            // the copies that hold a token of the list: what lies in the other
            // rows of a stage enters only products that are not written
            const int nt = lists ? (int)((min(plan.slots - s_first, (uint32_t)kRows) + per_copy - 1) / per_copy) : 0;
            const uint32_t bytes = lists ? (uint32_t)(plan.bn + nt * per_copy) * kChunk
                                         : (uint32_t)(plan.bn + args.tile_rows) * kChunk;
            // this lane's four tokens of the unit, or its tile (a clipped slot
            // reads the first token's row or tile)
            int t0 = 0, t1 = 0, t2 = 0, t3 = 0;
            if (tiles) {
                const uint32_t s0 = s_first + (uint32_t)(lane * args.tile_rows);
                if (lane < nt && pixel_of(p.px, s0) >= 0) {
                    const uint32_t tn = udiv(s0, p.px.dbb), t = udiv(tn, p.px.dN);
                    const int2 org = __ldg(reinterpret_cast<const int2 *>(p.px.idx) + t);
                    t0 = org.y;
                    t1 = org.x;
                    t2 = (int)(tn - t * (uint32_t)p.px.N);
                }
            } else if (lists) {
                const uint32_t s0 = s_first + 4 * lane;
                int rows[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    rows[k] = s0 + k < plan.slots ? (int)max((int64_t)0, pixel_of(p.px, s0 + k)) : 0;
                t0 = rows[0]; t1 = rows[1]; t2 = rows[2]; t3 = rows[3];
            }
            for (int c = c_lo; c < c_hi; ++c, ++it) {
                if (it >= plan.stages && !mbar_wait_w(bar + kBarEmpty + 8u * st, ph, abort_flag, hdr, kSiteEmpty)) {
                    ok = false;
                    break;
                }
                const uint32_t full = bar + kBarFull + 8u * st;
                const uint32_t dst = sb + (uint32_t)st * stage_bytes;
                if (!lists) {
                    tma_stage_w(dst + wdst, &tw, wrow, dst, &tbox, (int)s_first, full, bytes, c * kChunk);
                } else {
                    if (lane == 0)
                        mbar_expect_tx(full, bytes);
                    __syncwarp();
                    if (lane < nw)
                        tma_load_2d(dst + wdst + (uint32_t)wofs * kChunk, wmap, full, c * kChunk, wrow + wofs);
                    if (lane < nt) {
                        const uint32_t d = dst + (uint32_t)(lane * per_copy) * kChunk;
                        if (tiles)
                            tma_load_4d(d, &tbox, full, c * kChunk, t0, t1, t2);
                        else
                            tma_gather4(d, &tbox, full, c * kChunk, t0, t1, t2, t3);
                    }
                    __syncwarp();
                }
                if (++st == plan.stages) {
                    st = 0;
                    ph ^= 1;
                }
            }
        }
        if (!ok)
            drain_copies(bar, it, plan.stages);
        __syncwarp();
    } else if (warp == 1) {
        // ---- products
        const uint32_t id = idesc_s8(plan.bn);
        const uint64_t ring = desc_sw128(sb);
        const int last_steps = (p.C - (plan.nch - 1) * kChunk + 31) / 32;   // of the last chunk's 32-channel steps
        int st = 0, nu = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (uint32_t u = u_first; ok && u < plan.units; u += u_step, ++nu) {
            const int ab = nu & 1;
            if (nu >= 2 && !mbar_wait_w(bar + kBarAccEmpty + 8u * ab, ((nu >> 1) & 1) ^ 1, abort_flag, hdr, kSiteAccEmpty)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t d = tmem + (uint32_t)ab * kMaxBn;
            for (int c = c_lo; c < c_hi; ++c) {
                if (!mbar_wait_w(bar + kBarFull + 8u * st, ph, abort_flag, hdr, kSiteFull)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t ad = ring + (uint64_t)((uint32_t)st * (stage_bytes >> 4));
                mma_s8_commit_w(d, ad, ad + ((kRows * kChunk) >> 4), id, c > c_lo,
                                c + 1 < plan.nch ? 4 : last_steps, bar + kBarEmpty + 8u * st);
                if (++st == plan.stages) {
                    st = 0;
                    ph ^= 1;
                }
            }
            if (ok)
                tc_commit_w(bar + kBarAccFull + 8u * ab);
        }
        if (!ok)
            drain_products(bar);
        __syncwarp();
    } else {
        // ---- outputs
        const int et = (int)threadIdx.x - 64;
        const int r = (warp & 3) * 32 + lane;              // row of the unit = tensor-memory lane
        const int half = (warp - 2) >> 2;
        const uint32_t t_row = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        // put_rows' memory: that of the pushed sums or, where there are any, the
        // ring's, idle once a split unit's products (its CTA's only ones) are done
        const uint32_t tile = sb + (split_n > 1 ? 0u : kOffRecv) + 2048u * (uint32_t)(warp - 2);
        int nu = 0;
        bool ok = true;
        for (uint32_t u = u_first; u < plan.units; u += u_step, ++nu) {
            if (!ok) {   // a warp whose wait expired goes on meeting the others
                epi_sync();
                continue;
            }
            const int ab = nu & 1;
            const uint32_t rb = u / plan.cblocks;
            const int cb = (int)(u - rb * plan.cblocks);
            const uint32_t col = sb + kOffCol + (uint32_t)ab * 2 * kMaxBn * 4;
            float *colp = reinterpret_cast<float *>(smem + kOffCol + (uint32_t)ab * 2 * kMaxBn * 4);
            if (et < plan.bn) {
                const int c = cb * plan.bn + et;
                colp[et] = c < p.Co ? __ldg(p.sw + c) : 0.0f;
                colp[kMaxBn + et] = c < p.Co && p.bias ? __ldg(p.bias + c) : 0.0f;
            }
            const uint32_t s = rb * kRows + (uint32_t)r;
            const int64_t pix = s < plan.slots ? pixel_of(p.px, s) : -1;
            const float rs = pix >= 0 ? __ldg(p.sa + pix) : 0.0f;
            const bool live = rb * kRows + (uint32_t)((warp & 3) * 32) < plan.slots;   // the warp's rows hold a token
            epi_sync();
            if (!mbar_wait_w(bar + kBarAccFull + 8u * ab, (nu >> 1) & 1, abort_flag, hdr, kSiteAccFull)) {
                ok = false;
                continue;
            }
            tc_fence_after();
            const uint32_t t_acc = t_row + (uint32_t)ab * kMaxBn;
            // this CTA's columns: all, or its slice of a split unit
            const int cw = plan.bn / split_n, col0 = split * cw;
            if (split_n > 1) {
                if (!joined) {
                    cluster_wait();
                    joined = true;
                }
                // push the other slices to their owners: 16 columns at a time,
                // [sender][4 columns][row] of 16 bytes
                for (int o = 1; live && o < split_n; ++o) {
                    const int to = (split + o) & (split_n - 1);
                    const int from = ((split - to) & (split_n - 1)) - 1;   // this CTA among the owner's senders
                    for (int g = 16 * half; g < cw; g += 32) {
                        int acc[16];
                        ld_cols(t_acc + (uint32_t)(to * cw + g), acc);
                        ld_done();
                        const uint32_t dst = map_peer(sb + kOffRecv + (uint32_t)((from * (cw / 4) + g / 4) * kRows + r) * 16,
                                                      (uint32_t)(sub * split_n + to));
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            st_peer_s32x4(dst + (uint32_t)q * kRows * 16, acc[4 * q], acc[4 * q + 1], acc[4 * q + 2],
                                          acc[4 * q + 3]);
                    }
                    __syncwarp();   // the warp's pushes, then one arrival for them
                    if (lane == 0)
                        mbar_arrive_peer(map_peer(bar + kBarRecv, (uint32_t)(sub * split_n + to)));
                }
                if (live && !__all_sync(0xFFFFFFFFu, mbar_wait_cluster(bar + kBarRecv, 0, abort_flag, hdr, kSiteRecv))) {
                    ok = false;
                    continue;
                }
            }
            if (split_n == 1) {
                // 32 columns at a time, the next ones on their way
                int acc[2][32];
                auto load = [&](int g, int (&r)[32]) {
                    ld_cols(t_acc + (uint32_t)g, *reinterpret_cast<int (*)[16]>(r));
                    ld_cols(t_acc + (uint32_t)g + 16u, *reinterpret_cast<int (*)[16]>(r + 16));
                };
                auto finish = [&](int g, int (&q)[32]) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float v[16];
                        scale16<true>(q + 16 * h, col + 4u * (uint32_t)(g + 16 * h), rs, v);
                        put_cols(args, v, pix, cb * plan.bn + g + 16 * h, tile);
                    }
                };
                int g = 32 * half;
                if (g < cw) {
                    load(g, acc[0]);
                    ld_done();
                    while (true) {
                        if (g + 64 < cw)
                            load(g + 64, acc[1]);
                        finish(g, acc[0]);
                        if ((g += 64) >= cw)
                            break;
                        ld_done();
                        if (g + 64 < cw)
                            load(g + 64, acc[0]);
                        finish(g, acc[1]);
                        if ((g += 64) >= cw)
                            break;
                        ld_done();
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar + kBarAccEmpty + 8u * ab);
                continue;
            }
            for (int g = 16 * half; live && g < cw; g += 32) {
                int acc[16];
                ld_cols(t_acc + (uint32_t)(col0 + g), acc);
                ld_done();
                for (int f = 0; f < split_n - 1; ++f) {
                    const uint32_t src = sb + kOffRecv + (uint32_t)((f * (cw / 4) + g / 4) * kRows + r) * 16;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int4 v = lds_s32x4(src + (uint32_t)q * kRows * 16);
                        acc[4 * q] += v.x;
                        acc[4 * q + 1] += v.y;
                        acc[4 * q + 2] += v.z;
                        acc[4 * q + 3] += v.w;
                    }
                }
                float v[16];
                scale16<true>(acc, col + 4u * (uint32_t)(col0 + g), rs, v);
                put_cols(args, v, pix, cb * plan.bn + col0 + g, tile);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar + kBarAccEmpty + 8u * ab);
        }
    }
    if (csize > 1 && !joined)
        cluster_wait();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * kMaxBn));
    }
    // no CTA leaves while a peer may still address its shared memory
    if (csize > 1) {
        cluster_arrive();
        cluster_wait();
    }
}

// The same for a whole map whose units are not split and whose
// outputs TMA can store: the loops that bound the large products, with nothing
// else in them.  kE: bytes of an output element.
template <int kE>
__global__ void __launch_bounds__(qt::kThreads, 1)
    k_qlinear_whole(const __grid_constant__ qt::Args args, const __grid_constant__ CUtensorMap tw,
                    const __grid_constant__ CUtensorMap tbox, const __grid_constant__ CUtensorMap ty)
{
    extern __shared__ __align__(1024) uint8_t qt_raw[];
    const QLinearParams &p = args.q;
    const Plan &plan = args.plan;
    const uint32_t raw = smem_u32(qt_raw);
    const uint32_t sb = (raw + 1023u) & ~1023u;
    uint8_t *smem = qt_raw + (sb - raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t bar = sb + kOffBar;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOffBar + kAbort);
    WsHeader *hdr = p.hdr;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(bar + kBarFull + 8u * i, 1);
            mbar_init(bar + kBarEmpty + 8u * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar + kBarAccFull + 8u * i, 1);
            mbar_init(bar + kBarAccEmpty + 8u * i, kEpiWarps);
        }
        mbar_init(bar + kBarDrain, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0 && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tw)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tbox)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&ty)) : "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(bar + kTmemSlot),
                     "r"(2 * kMaxBn));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + kOffBar + kTmemSlot);
    pdl_wait();

    const uint32_t stage_bytes = (uint32_t)(kRows + plan.bn) * kChunk;
    if (warp == 0) {
        // ---- operands
        int it = 0, st = 0;
        uint32_t ph = 1;
        bool ok = true;
        for (uint32_t u = blockIdx.x; ok && u < plan.units; u += gridDim.x) {
            const uint32_t rb = u / plan.cblocks;
            const int cb = (int)(u - rb * plan.cblocks);
            for (int c = 0; c < plan.nch; ++c, ++it) {
                if (it >= plan.stages && !mbar_wait_w(bar + kBarEmpty + 8u * st, ph, abort_flag, hdr, kSiteEmpty)) {
                    ok = false;
                    break;
                }
                const uint32_t dst = sb + (uint32_t)st * stage_bytes;
                tma_stage_w(dst + kRows * kChunk, &tw, cb * plan.bn, dst, &tbox, (int)rb * kRows, bar + kBarFull + 8u * st,
                            (uint32_t)(plan.bn + args.tile_rows) * kChunk, c * kChunk);
                if (++st == plan.stages) {
                    st = 0;
                    ph ^= 1;
                }
            }
        }
        if (!ok)
            drain_copies(bar, it, plan.stages);
        __syncwarp();
    } else if (warp == 1) {
        // ---- products
        const uint32_t id = idesc_s8(plan.bn);
        const uint64_t ring = desc_sw128(sb);
        const int last_steps = (p.C - (plan.nch - 1) * kChunk + 31) / 32;
        int st = 0, nu = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (uint32_t u = blockIdx.x; ok && u < plan.units; u += gridDim.x, ++nu) {
            const int ab = nu & 1;
            if (nu >= 2 && !mbar_wait_w(bar + kBarAccEmpty + 8u * ab, ((nu >> 1) & 1) ^ 1, abort_flag, hdr, kSiteAccEmpty)) {
                ok = false;
                break;
            }
            tc_fence_after();
            for (int c = 0; c < plan.nch; ++c) {
                if (!mbar_wait_w(bar + kBarFull + 8u * st, ph, abort_flag, hdr, kSiteFull)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t ad = ring + (uint64_t)((uint32_t)st * (stage_bytes >> 4));
                mma_s8_commit_w(tmem + (uint32_t)ab * kMaxBn, ad, ad + ((kRows * kChunk) >> 4), id, c > 0,
                                c + 1 < plan.nch ? 4 : last_steps, bar + kBarEmpty + 8u * st);
                if (++st == plan.stages) {
                    st = 0;
                    ph ^= 1;
                }
            }
            if (ok)
                tc_commit_w(bar + kBarAccFull + 8u * ab);
        }
        if (!ok)
            drain_products(bar);
        __syncwarp();
    } else {
        // ---- outputs: a warp's rows are its quarter of the tensor memory's
        // lanes, its columns every other group of 64 bytes
        constexpr int kCols = 64 / kE;
        const int et = (int)threadIdx.x - 64, r = (warp & 3) * 32 + lane, half = (warp - 2) >> 2;
        const uint32_t t_row = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t tile = sb + kOffRecv + (uint32_t)(warp - 2) * 2048u;
        float *colp = reinterpret_cast<float *>(smem + kOffCol);
        // a unit's scales (thread: a column's, and its row's) are on their way
        // under the unit before
        float n_sw = 0.0f, n_bias = 0.0f, n_sa = 0.0f;
        auto fetch = [&](uint32_t u) {
            const uint32_t rb = u / plan.cblocks;
            const int c = (int)(u - rb * plan.cblocks) * plan.bn + et;
            const bool in = et < plan.bn && c < p.Co;
            const int64_t row = (int64_t)rb * kRows + r;
            n_sw = in ? __ldg(p.sw + c) : 0.0f;
            n_bias = in && p.bias ? __ldg(p.bias + c) : 0.0f;
            n_sa = row < p.rows ? __ldg(p.sa + row) : 0.0f;
        };
        if (blockIdx.x < plan.units)
            fetch(blockIdx.x);
        int nu = 0;
        bool ok = true;
        for (uint32_t u = blockIdx.x; u < plan.units; u += gridDim.x, ++nu) {
            const int ab = nu & 1;
            const uint32_t rb = u / plan.cblocks;
            const int c0 = (int)(u - rb * plan.cblocks) * plan.bn;
            const uint32_t col = sb + kOffCol + (uint32_t)ab * 2 * kMaxBn * 4;
            colp[ab * 2 * kMaxBn + et] = n_sw;
            colp[ab * 2 * kMaxBn + kMaxBn + et] = n_bias;
            const float sa = n_sa;
            const int row0 = (int)rb * kRows + (warp & 3) * 32;
            const int64_t e0 = ((int64_t)row0 + lane) * p.Co + c0;
            const bool has_res = p.residual && row0 + lane < p.rows;
            uint32_t res[16];
            auto residual = [&](int g) {   // this row's 64 bytes from column g of the unit on
                if (has_res && c0 + g < p.Co) {
                    ld_v8(p.residual + (e0 + g) * kE, res);
                    if (c0 + g + kCols / 2 < p.Co)
                        ld_v8(p.residual + (e0 + g) * kE + 32, res + 8);
                }
            };
            residual(half * kCols);
            if (u + gridDim.x < plan.units)
                fetch(u + gridDim.x);
            epi_sync();   // (every warp of every unit comes here: a wait that expired keeps a warp in the loop)
            if (ok)
                ok = mbar_wait_w(bar + kBarAccFull + 8u * ab, (nu >> 1) & 1, abort_flag, hdr, kSiteAccFull);
            if (!ok)
                continue;
            tc_fence_after();
            const uint32_t t_acc = t_row + (uint32_t)ab * kMaxBn;
            auto finish = [&](auto big) {
#pragma unroll 1
                for (int g = half * kCols; g < plan.bn && c0 + g < p.Co; g += 2 * kCols) {
                    int acc[kCols];
                    float v[kCols];
#pragma unroll
                    for (int q = 0; q < kCols; q += 16)
                        ld_cols(t_acc + (uint32_t)(g + q), *reinterpret_cast<int (*)[16]>(acc + q));
                    ld_done();
#pragma unroll
                    for (int q = 0; q < kCols; q += 16)
                        scale16<decltype(big)::value>(acc + q, col + 4u * (uint32_t)(g + q), sa, v + q);
                    if (p.residual) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            if constexpr (kE == 2) {
                                v[2 * k] += bf16_lo(res[k]);
                                v[2 * k + 1] += bf16_hi(res[k]);
                            } else {
                                v[k] += __uint_as_float(res[k]);
                            }
                        }
                        if (g + 2 * kCols < plan.bn)
                            residual(g + 2 * kCols);
                    }
                    if (row0 < p.rows)
                        put_tile<kE>(v, tile, &ty, c0 + g, row0, lane);
                }
            };
            // (a loop of its own for warps with such a token: their multiplication more
            // took 16384 x 640 -> 5120 from 60.1 to 61.3 us in one loop for all)
            if (__any_sync(0xFFFFFFFFu, is_big(sa)))
                finish(std::true_type());
            else
                finish(std::false_type());
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar + kBarAccEmpty + 8u * ab);
        }
        if (lane == 0)
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");   // the outputs have left shared memory
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * kMaxBn));
    }
}

namespace qt {

// k_qlinear_staged: 8 warps stage and finish, one issues.
constexpr int kStagedThreads = kEpiThreads + 32;
constexpr int kStagedStages = 4, kStagedBn = 128;
constexpr uint32_t kStagedStage = (kRows + kStagedBn) * kChunk;
constexpr uint32_t kOffStagedTile = kStagedStages * kStagedStage;            // put_rows' memory
constexpr uint32_t kOffStagedCol = kOffStagedTile + kEpiWarps * 2048;        // per unit parity: scales and biases
constexpr uint32_t kOffStagedRow = kOffStagedCol + 2 * 2 * kMaxBn * 4;       // the unit's rows of tokens and channels
constexpr uint32_t kOffStagedBar = kOffStagedRow + (kRows + kStagedBn) * 8;
constexpr uint32_t kStagedSmem = kOffStagedBar + 256 + 1024;
constexpr int kSiteStagedEmpty = 311, kSiteStagedFull = 312, kSiteStagedAccEmpty = 313, kSiteStagedAccFull = 314;

} // namespace qt

// The product for codes that TMA cannot copy (channels that are not a multiple of
// 16, addresses that are not): the same units of 128 tokens x bn (128 .. 32)
// channels, the stages filled by the CTA's warps: lane l takes aligned word l of
// a row's 128 bytes of K (32 rows a warp and chunk, the next chunk's on their
// way), shifts its neighbour's bytes in and leaves 4 bytes; a row's last word's
// neighbour comes from the lane that is the row's number.  Bound by that staging,
// about 3200 cycles a chunk of 128 x 128.  16384 x 300 -> 5120 810 us with four
// products an instruction on CUDA cores, 332 us with 16 bytes of a row a lane
// (every word fetched from L2 again and again), 230 us here; 16384 x 1280 -> 320
// 51 us, 9.2 by TMA.
__global__ void __launch_bounds__(qt::kStagedThreads, 1) k_qlinear_staged(const __grid_constant__ qt::Args args)
{
    extern __shared__ __align__(1024) uint8_t qt_raw[];
    const QLinearParams &p = args.q;
    const uint32_t raw = smem_u32(qt_raw);
    const uint32_t sb = (raw + 1023u) & ~1023u;
    uint8_t *smem = qt_raw + (sb - raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t bar = sb + kOffStagedBar;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOffStagedBar + kAbort);
    WsHeader *hdr = p.hdr;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStagedStages; ++i) {
            mbar_init(bar + kBarFull + 8u * i, kEpiWarps);
            mbar_init(bar + kBarEmpty + 8u * i, 1);
        }
        mbar_init(bar + kBarAccFull, 1);
        mbar_init(bar + kBarAccEmpty, kEpiWarps);
        mbar_init(bar + kBarDrain, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kEpiWarps) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(bar + kTmemSlot),
                     "r"(kStagedBn));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    pdl_wait();
    const int64_t slots = pixel_slots(p.px);
    const int64_t rblocks = (slots + kRows - 1) / kRows;
    // the widest units that leave no CTA without one
    int bn = kStagedBn;
    while (bn > 32 && rblocks * ((p.Co + bn - 1) / bn) < (int64_t)gridDim.x)
        bn >>= 1;
    const int cblocks = (p.Co + bn - 1) / bn, nch = (p.C + kChunk - 1) / kChunk;
    const int64_t units = rblocks * cblocks;
    const int last_steps = (p.C - (nch - 1) * kChunk + 31) / 32;   // of the last chunk's 32-channel steps
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + kOffStagedBar + kTmemSlot);

    if (warp == kEpiWarps) {
        // ---- products
        const uint32_t id = idesc_s8(bn);
        const uint64_t ring = desc_sw128(sb);
        int st = 0, nu = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int64_t u = blockIdx.x; ok && u < units; u += gridDim.x, ++nu) {
            if (nu > 0 && !mbar_wait_w(bar + kBarAccEmpty, (nu - 1) & 1, abort_flag, hdr, kSiteStagedAccEmpty)) {
                ok = false;
                break;
            }
            tc_fence_after();
            for (int c = 0; c < nch; ++c) {
                if (!mbar_wait_w(bar + kBarFull + 8u * st, ph, abort_flag, hdr, kSiteStagedFull)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t ad = ring + (uint64_t)((uint32_t)st * (kStagedStage >> 4));
                mma_s8_commit_w(tmem, ad, ad + ((kRows * kChunk) >> 4), id, c > 0, c + 1 < nch ? 4 : last_steps,
                                bar + kBarEmpty + 8u * st);
                if (++st == kStagedStages) {
                    st = 0;
                    ph ^= 1;
                }
            }
            if (ok)
                tc_commit_w(bar + kBarAccFull);
        }
        if (!ok)
            drain_products(bar);
        __syncwarp();
    } else {
        // ---- staging, then outputs
        const int et = (int)threadIdx.x;
        const int r = (warp & 3) * 32 + lane, half = warp >> 2;
        const uint32_t t_row = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t tile = sb + kOffStagedTile + 2048u * (uint32_t)warp;
        // a warp's rows: every 8th token, then every 8th channel
        const int mine = 16 + bn / kEpiWarps;
        unsigned long long *rowp = reinterpret_cast<unsigned long long *>(smem + kOffStagedRow);
        int it = 0, st = 0, nu = 0;
        uint32_t ph = 1;
        bool ok = true;
        for (int64_t u = blockIdx.x; u < units; u += gridDim.x, ++nu) {
            const int64_t rb = u / cblocks;
            const int c0 = (int)(u - rb * cblocks) * bn;
            // (every warp has staged the last unit: it has met the others since)
            if (et < kRows) {
                const int64_t s = rb * kRows + et;
                const int64_t pix = s < slots ? pixel_of(p.px, (uint32_t)s) : -1;
                rowp[et] = pix >= 0 ? reinterpret_cast<unsigned long long>(p.a + pix * p.C) : 0ull;
            } else {
                const int ch = c0 + et - kRows;
                rowp[et] = et - kRows < bn && ch < p.Co ? reinterpret_cast<unsigned long long>(p.w + (int64_t)ch * p.C) : 0ull;
            }
            epi_sync();
            if (ok) {
                // row i of the warp: its place in the table and in a stage
                auto place_of = [&](int i) { return warp + 8 * i; };
                const unsigned long long own = lane < mine ? rowp[place_of(lane)] : 0ull;
                // bits of every row's offset in a word (the same for every chunk)
                const uint32_t low = __ballot_sync(0xFFFFFFFFu, own & 1), high = __ballot_sync(0xFFFFFFFFu, own & 2);
                uint32_t w[32], w33 = 0;
                auto fetch = [&](int c) {
                    const int n = min(kChunk, p.C - c * kChunk);   // bytes of a row
                    if (own) {
                        const unsigned long long a = own + (unsigned)(c * kChunk);
                        w33 = (int)(a & 3) + n > kChunk ? __ldg(reinterpret_cast<const uint32_t *>(a & ~3ull) + 32) : 0u;
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        if (i < mine) {
                            const unsigned long long row = rowp[place_of(i)], a = row + (unsigned)(c * kChunk);
                            w[i] = 0;
                            if (row && 4 * lane < (int)(a & 3) + n)
                                w[i] = __ldg(reinterpret_cast<const uint32_t *>(a & ~3ull) + lane);
                        }
                    }
                };
                fetch(0);
                for (int c = 0; c < nch; ++c, ++it) {
                    // (rows without a token or a channel are zeros: leaving them out by a
                    // branch takes the rows out of step, 300 -> 420 us when it was tried)
                    const int left = p.C - c * kChunk - 4 * lane;   // bytes of this lane's word
                    const uint32_t mask = left >= 4 ? 0xFFFFFFFFu : left > 0 ? (1u << (8 * left)) - 1u : 0u;
                    uint32_t x[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        if (i < mine) {
                            const uint32_t sh = ((low >> i) & 1u) * 8u + ((high >> i) & 1u) * 16u;
                            const uint32_t up = __shfl_down_sync(0xFFFFFFFFu, w[i], 1), end = __shfl_sync(0xFFFFFFFFu, w33, i);
                            x[i] = __funnelshift_r(w[i], lane == 31 ? end : up, sh) & mask;
                        }
                    }
                    if (c + 1 < nch)
                        fetch(c + 1);
                    if (it >= kStagedStages && !mbar_wait_w(bar + kBarEmpty + 8u * st, ph, abort_flag, hdr, kSiteStagedEmpty)) {
                        ok = false;
                        break;
                    }
                    // (row & 7 is the warp's number)
                    const uint32_t dst = sb + (uint32_t)st * kStagedStage + 4u * (uint32_t)(lane & 3) +
                                         (((uint32_t)(lane >> 2) ^ (uint32_t)warp) << 4);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (i < mine)
                            asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst + (uint32_t)place_of(i) * kChunk), "r"(x[i]) : "memory");
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(bar + kBarFull + 8u * st);
                    if (++st == kStagedStages) {
                        st = 0;
                        ph ^= 1;
                    }
                }
            }
            const uint32_t col = sb + kOffStagedCol + (uint32_t)(nu & 1) * 2 * kMaxBn * 4;
            float *colp = reinterpret_cast<float *>(smem + kOffStagedCol + (uint32_t)(nu & 1) * 2 * kMaxBn * 4);
            if (et < bn) {
                const int c = c0 + et;
                colp[et] = c < p.Co ? __ldg(p.sw + c) : 0.0f;
                colp[kMaxBn + et] = c < p.Co && p.bias ? __ldg(p.bias + c) : 0.0f;
            }
            const int64_t s = rb * kRows + r;
            const int64_t pix = s < slots ? pixel_of(p.px, (uint32_t)s) : -1;
            const float rs = pix >= 0 ? __ldg(p.sa + pix) : 0.0f;
            epi_sync();   // (met by every warp, after an expired wait too)
            if (ok)
                ok = mbar_wait_w(bar + kBarAccFull, nu & 1, abort_flag, hdr, kSiteStagedAccFull);
            if (!ok)
                continue;
            tc_fence_after();
            for (int g = 16 * half; g < bn && c0 + g < p.Co; g += 32) {
                int acc[16];
                ld_cols(t_row + (uint32_t)g, acc);
                ld_done();
                float v[16];
                scale16<true>(acc, col + 4u * (uint32_t)g, rs, v);
                put_cols(args, v, pix, c0 + g, tile);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar + kBarAccEmpty);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kEpiWarps) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kStagedBn));
    }
}

// ------------------------------------------------------------------ host

// 128-byte columns of a matrix of `rows` rows of C codes, box_rows rows a copy.
static bool encode_rows(CUtensorMap *map, const void *base, int64_t rows, int C, int box_rows, CUtensorMapL2promotion l2,
                        PFN_cuTensorMapEncodeTiled_v12000 encode)
{
    cuuint64_t dims[2] = {(cuuint64_t)C, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)C};
    cuuint32_t box[2] = {(cuuint32_t)qt::kChunk, (cuuint32_t)box_rows};
    cuuint32_t es[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, l2,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The token map [N][H][W][C], one b x b tile a copy (zeros outside the map).
static bool encode_tiles(CUtensorMap *map, const QLinearParams &p, PFN_cuTensorMapEncodeTiled_v12000 encode)
{
    const cuuint64_t C = (cuuint64_t)p.C, W = (cuuint64_t)p.px.W, H = (cuuint64_t)p.px.H;
    cuuint64_t dims[4] = {C, W, H, (cuuint64_t)p.px.N};
    cuuint64_t strides[3] = {C, C * W, C * W * H};
    cuuint32_t box[4] = {(cuuint32_t)qt::kChunk, (cuuint32_t)p.px.b, (cuuint32_t)p.px.b, 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t *>(p.a), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The output [rows][Co], 64 bytes of columns x 32 rows a copy.
static bool encode_out(CUtensorMap *map, const QLinearParams &p, int esz, PFN_cuTensorMapEncodeTiled_v12000 encode)
{
    cuuint64_t dims[2] = {(cuuint64_t)p.Co, (cuuint64_t)p.rows};
    cuuint64_t strides[1] = {(cuuint64_t)p.Co * esz};
    cuuint32_t box[2] = {(cuuint32_t)(64 / esz), 32};
    cuuint32_t es[2] = {1, 1};
    return encode(map, esz == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, p.y, dims, strides,
                  box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool qlinear_tma_scope(int c) { return c % 16 == 0; }

static int launch_staged(const QLinearParams &p, cudaStream_t stream)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return SIGE_ERR_CUDA;
    static std::atomic<int> smem_set[64];
    if (!smem_set[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(k_qlinear_staged, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)qt::kStagedSmem) != cudaSuccess) {
            cudaGetLastError();
            return SIGE_ERR_CUDA;
        }
        smem_set[dev].store(1, std::memory_order_release);
    }
    prefer_max_shared_of<k_qlinear_staged>();
    qt::Args a{};
    a.q = p;
    const int esz = p.dtype == SIGE_BF16 ? 2 : 4;
    a.vec = (int64_t)p.Co * esz % 32 == 0 && aligned_to(p.y, 32) && aligned_to(p.residual, 32);
    a.width = qt::row_width(p);
    const int64_t most = (p.slots + qt::kRows - 1) / qt::kRows * ((p.Co + 31) / 32);
    const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(most, device_sm_count()));
    if (launch_pdl(k_qlinear_staged, dim3(grid), dim3(qt::kStagedThreads), qt::kStagedSmem, stream, a) != cudaSuccess) {
        cudaGetLastError();
        return SIGE_ERR_CUDA;
    }
    count_launch();
    return launch_check();
}

int launch_qlinear(const QLinearParams &p, cudaStream_t stream)
{
    // (the TMA kernels count units in 32 bits)
    const int64_t narrowest = ((p.slots + qt::kRows - 1) / qt::kRows) * (((int64_t)p.Co + 31) / 32);
    if (!qlinear_tma_scope(p.C) || !aligned_to(p.a, 16) || !aligned_to(p.w, 16) || narrowest > INT32_MAX / 8)
        return launch_staged(p, stream);
    const PFN_cuTensorMapEncodeTiled_v12000 encode = get_encode();
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return SIGE_ERR_CUDA;
    if (!encode)
        return SIGE_ERR_CUDA;
    qt::Args a{};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = qt::kCluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(qt::kThreads);
    cfg.dynamicSmemBytes = qt::kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    static std::atomic<int> clusters_of[64];   // co-resident clusters, per device
    int ncl = clusters_of[dev].load(std::memory_order_acquire);
    if (ncl == 0) {
        if (cudaFuncSetAttribute(k_qlinear_tc, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)qt::kSmem) != cudaSuccess ||
            cudaFuncSetAttribute(k_qlinear_whole<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)qt::kSmem) != cudaSuccess ||
            cudaFuncSetAttribute(k_qlinear_whole<4>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)qt::kSmem) != cudaSuccess) {
            cudaGetLastError();
            return SIGE_ERR_CUDA;
        }
        cfg.gridDim = dim3(qt::kCluster * (device_sm_count() / qt::kCluster));
        cfg.attrs = attr + 1;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&ncl, k_qlinear_tc, &cfg) != cudaSuccess || ncl < 1) {
            cudaGetLastError();
            return SIGE_ERR_CUDA;
        }
        cfg.attrs = attr;
        clusters_of[dev].store(ncl, std::memory_order_release);
    }
    prefer_max_shared(k_qlinear_tc);
    a.q = p;
    const int esz = p.dtype == SIGE_BF16 ? 2 : 4;
    a.vec = (int64_t)p.Co * esz % 32 == 0 && aligned_to(p.y, 32) && aligned_to(p.residual, 32);
    a.width = qt::row_width(p);
    // a whole map of enough units needs no cluster (every SM takes part); a
    // list's length is known on the device only
    const int sms = device_sm_count();
    const int most = qt::kCluster * ncl;
    bool solo = false, whole = false;
    if (!p.px.idx) {
        a.plan = qt::make_plan((uint32_t)p.slots, qt::kMapCosts, p.Co, p.C, most, qt::kCluster);
        solo = a.plan.split == 1;
        if (solo)
            a.plan = qt::make_plan((uint32_t)p.slots, qt::kMapCosts, p.Co, p.C, sms, 1);
        cfg.gridDim = dim3(solo ? (unsigned)std::min<int64_t>(sms, a.plan.units)
                                : (a.plan.units * a.plan.split + qt::kCluster - 1) / qt::kCluster * qt::kCluster);
    } else {
        // no more clusters than the narrowest units of a full list can use
        cfg.gridDim = dim3((unsigned)(qt::kCluster * std::max<int64_t>(1, std::min<int64_t>(ncl, narrowest))));
    }
    cfg.numAttrs = solo ? 1 : 2;
    // how the operands are copied.  A whole map: one box of weight rows and one
    // of tokens a stage.  A list: tiles of 4 x 4 or 8 x 8 (a divisor of 128
    // tokens) by a box each, 5.7 us where four tokens a copy took 8.8 (25 tiles
    // of 4 x 4, C 320 -> 320); four tokens a copy otherwise.
    CUtensorMap tw, tw64, tw32, tbox, ty{};
    const CUtensorMapL2promotion l2 = CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
    bool good;
    if (!p.px.idx) {
        // (rows of a box past the map's end are zeros, but not for nothing: one
        // token x 5120 -> 1280 with boxes of 128 rows 8.4 us, 32 tokens 6.8)
        a.tile_rows = (int)std::min<int64_t>((p.slots + 7) / 8 * 8, qt::kRows);
        good = encode_rows(&tw, p.w, p.Co, p.C, a.plan.bn, l2, encode) &&
               encode_rows(&tbox, p.a, p.rows, p.C, a.tile_rows, l2, encode);
        tw64 = tw32 = tw;
        whole = solo && a.vec && encode_out(&ty, p, esz, encode);
    } else {
        good = encode_rows(&tw, p.w, p.Co, p.C, 128, l2, encode) && encode_rows(&tw64, p.w, p.Co, p.C, 64, l2, encode) &&
               encode_rows(&tw32, p.w, p.Co, p.C, 32, l2, encode);
        if (p.px.b == 4 || p.px.b == 8) {
            a.tile_rows = p.px.b * p.px.b;
            good = good && encode_tiles(&tbox, p, encode);
        } else {
            good = good && encode_rows(&tbox, p.a, p.rows, p.C, 1, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, encode);
        }
    }
    if (!good)
        return SIGE_ERR_CUDA;
    const cudaError_t err = !whole      ? cudaLaunchKernelEx(&cfg, k_qlinear_tc, a, tw, tw64, tw32, tbox)
                            : esz == 2 ? cudaLaunchKernelEx(&cfg, k_qlinear_whole<2>, a, tw, tbox, ty)
                                       : cudaLaunchKernelEx(&cfg, k_qlinear_whole<4>, a, tw, tbox, ty);
    if (err != cudaSuccess) {
        cudaGetLastError();
        return SIGE_ERR_CUDA;
    }
    count_launch();
    return launch_check();
}

} // namespace sige
