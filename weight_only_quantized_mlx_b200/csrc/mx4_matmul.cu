// Y = A W^T with both operands in MX4, on the block-scaled tensor instruction
// (tcgen05.mma kind::mxf4): E2M1 codes straight from memory, one E8M0 scale per
// 32 columns applied inside the tensor core, fp32 sums in TMEM.
//
//   tile: 256 weight rows (two MMA M = 128 halves) x BN activation rows (MMA N,
//         up to 224), over all of K in k-blocks of 256 columns (one 128-byte row
//         of codes, four MMAs of K = 64 per half).  Where tiles leave SMs idle, the
//         S blocks of a cluster take a range of K of one tile each and add their
//         sums through distributed shared memory, in rank order.
//   warp 0      TMA: the codes of both operands (128-byte swizzle)
//   warp 1      allocates TMEM; one lane copies each k-block's scales into TMEM
//               (tcgen05.cp) and issues the MMAs
//   warps 2, 3 and 12, 13  scales of the weight rows and of the activation rows,
//               128 rows each: 8 bytes a row and k-block, loaded two k-blocks
//               ahead (16 bytes for two of them where alignment allows: a row's
//               sector is then fetched half as often), put into the 128 x 4
//               order that tcgen05.cp and
//               the MMA expect (row r, group g of a set of four: byte
//               (r % 32) 16 + (r / 32) 4 + g)
//   warps 4-11  read the accumulators (tcgen05.ld) as BF16 into registers,
//               hand TMEM back and store Y while the next tile's MMAs run
//
// TMEM (512 columns): 2 x 224 columns of sums, 2 x 32 columns of scales (a
// k-block's: two halves and two sets of four columns for the weight, two sets of
// eight for the activations).  Why 256 x 224: at the 4-bit rate a k-block of
// codes must arrive in about half a microsecond, so the bytes from L2 per
// multiply bound the kernel, and this is the squarest tile that leaves TMEM
// room for scales.  Columns behind K and rows behind the operands read as zero
// codes under scale 1.
//
// Measured: 8192 x 14336 x 4096 222 us (4.3 PFLOP/s), 8192 x 4096 x 14336 200 us (4.8),
// 509 x 4100 x 14368 38 us (1.6), 64 x 4096 x 14336 16 us.  With parts cut out (the
// first two and the third, when they took 235, 202 and 38 us): no loads of scales 205,
// 182, 30; no copies of scales to TMEM 231, 190, 37; neither 186, 162, 29; no codes
// 198, 175, 35; MMAs alone 151, 129, 24.
//
// All waits are bounded; after one gives up the producers and the MMA thread
// issue nothing more and wait (bounded) for what they issued.
#include <cooperative_groups.h>

#include "device_common.cuh"
#include "kernels.h"
#include "mx4_common.cuh"
#include "tensor_map.h"

namespace mlxq {
namespace {

constexpr int kBM = 256;                     // weight rows per tile
constexpr int kMaxBN = 224;                  // activation rows per tile
constexpr int kBK = 256;                     // columns per k-block
constexpr int kStages = 3;
constexpr uint32_t kStageW = kBM * 128;      // codes of the weight rows
constexpr uint32_t kStageX = kMaxBN * 128;   // codes of the activation rows
constexpr uint32_t kStageS = 2048;           // scales of one operand: [half][set][32][16]
constexpr uint32_t kStageBytes = kStageW + kStageX + 2 * kStageS;
constexpr int kFirstEpilogue = 4;
constexpr int kFirstXScales = kFirstEpilogue + 8;
constexpr int kThreads = (kFirstXScales + 2) * 32;
constexpr uint32_t kAccCols = kMaxBN;        // TMEM columns of one half's sums
constexpr uint32_t kScaleCol = 2 * kAccCols; // then two buffers of 32 columns of scales
static_assert(kScaleCol + 2 * 32 <= 512, "TMEM columns");

struct MatmulParams {
    uint16_t* Y;
    const uint8_t* w_scales;
    const uint8_t* a_scales;
    int N, m, G;        // weight rows, activation rows, scale bytes per row
    int BN, num_kb, S;
    uint32_t idesc;
    unsigned int* status;
};

__device__ __forceinline__ void umma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// 32 rows x 16 bytes of shared memory -> four TMEM columns, in all four lane quadrants
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// K-major operand, rows of 128 bytes, 128-byte swizzle, 8-row groups 1024 bytes apart
__device__ __forceinline__ uint64_t codes_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | static_cast<uint64_t>(1u) << 16 |
           static_cast<uint64_t>(1024u >> 4) << 32 | static_cast<uint64_t>(1u) << 46 | static_cast<uint64_t>(2u) << 61;
}
// 32 rows of 16 bytes, no swizzle, 8-row groups 128 bytes apart
__device__ __forceinline__ uint64_t scales_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | static_cast<uint64_t>(1u) << 16 |
           static_cast<uint64_t>(128u >> 4) << 32 | static_cast<uint64_t>(1u) << 46;
}

// The eight scale bytes of one row and k-block, from the table's byte e on: words
// now, bytes when they are due, so that the loads of many rows are in flight
// together.  SCALES_PAIR: rows are multiples of 16 bytes, the table is 16-byte
// aligned and the k-blocks come in pairs, which share a load.  SCALES_WIDE:
// 8 bytes.  SCALES_ANY: the bytes start anywhere in a word; words that the table does
// not have all of are not read.
enum ScaleLoads { SCALES_ANY, SCALES_WIDE, SCALES_PAIR };
__device__ __forceinline__ uint32_t ldg_if(const uint8_t* p, bool read) {
    uint32_t v;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %2, 0;\n\t"
        "mov.u32 %0, 0;\n\t"
        "@p ld.global.nc.u32 %0, [%1];\n\t}"
        : "=r"(v)
        : "l"(p), "r"(static_cast<uint32_t>(read)));
    return v;
}
template <ScaleLoads LOADS>
constexpr int kScaleWords = LOADS == SCALES_ANY ? 3 : (LOADS == SCALES_WIDE ? 2 : 4);
template <ScaleLoads LOADS>
__device__ __forceinline__ void load_words(uint32_t (&w)[kScaleWords<LOADS>], const uint8_t* scales, int64_t e, int64_t table, bool live) {
    if constexpr (LOADS == SCALES_PAIR) {
        uint4 v = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
        if (live) v = __ldg(reinterpret_cast<const uint4*>(scales + e));
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    } else if constexpr (LOADS == SCALES_WIDE) {
        uint2 v = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
        if (live) v = __ldg(reinterpret_cast<const uint2*>(scales + e));
        w[0] = v.x;
        w[1] = v.y;
    } else {
        const int64_t at = e & ~int64_t{3};
#pragma unroll
        for (int i = 0; i < 3; ++i) w[i] = ldg_if(scales + at + 4 * i, live && at + 4 * i + 4 <= table);
    }
}
// `left`: blocks left in the row; behind them, and where there is no row, 127 (scale 1).
__device__ __forceinline__ uint2 scale_bytes(const uint32_t (&w)[3], const uint8_t* scales, int64_t e, int64_t table, bool live, int left) {
    if (!live) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    const uint32_t sh = 8u * static_cast<uint32_t>(e & 3);
    uint32_t lo = __funnelshift_r(w[0], w[1], sh), hi = __funnelshift_r(w[1], w[2], sh);
    if (e + 8 > (table & ~int64_t{3})) {  // the table's last bytes, not a whole word
        lo = hi = 0;
        for (int i = 0; i < 4; ++i) {
            if (e + i < table) lo |= static_cast<uint32_t>(__ldg(scales + e + i)) << (8 * i);
            if (e + 4 + i < table) hi |= static_cast<uint32_t>(__ldg(scales + e + 4 + i)) << (8 * i);
        }
    }
    const uint32_t k0 = left >= 4 ? 0xFFFFFFFFu : (1u << (8 * left)) - 1u;
    const uint32_t k1 = left >= 8 ? 0xFFFFFFFFu : (left > 4 ? (1u << (8 * (left - 4))) - 1u : 0u);
    return make_uint2((lo & k0) | (0x7F7F7F7Fu & ~k0), (hi & k1) | (0x7F7F7F7Fu & ~k1));
}

template <ScaleLoads LOADS>
__global__ void __launch_bounds__(kThreads, 1)
    k_mx4_matmul(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_a, const MatmulParams p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[3 * kStages + 3];
    __shared__ uint32_t tmem_slot;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;  // swizzle atoms
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles_n = (p.N + kBM - 1) / kBM, tiles = tiles_n * ((p.m + p.BN - 1) / p.BN);
    // S == 1: block b takes tiles b, b + gridDim.x, ...; else cluster c takes tile c alone
    const int S = p.S, rank = static_cast<int>(blockIdx.x) % S, first = static_cast<int>(blockIdx.x) / S;
    const int stride = S == 1 ? static_cast<int>(gridDim.x) : tiles;
    const int kb0 = static_cast<int>(static_cast<int64_t>(p.num_kb) * rank / S);
    const int num_kb = static_cast<int>(static_cast<int64_t>(p.num_kb) * (rank + 1) / S) - kb0;

    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * static_cast<uint32_t>(s); };                 // codes landed
    auto sfull = [&](int s) { return bar0 + 8u * static_cast<uint32_t>(kStages + s); };      // scales written
    auto empty = [&](int s) { return bar0 + 8u * static_cast<uint32_t>(2 * kStages + s); };  // stage read
    const uint32_t acc_full = bar0 + 8u * 3 * kStages, acc_empty = acc_full + 8u, drain = acc_full + 16u;
    auto W_of = [&](int s) { return base + static_cast<uint32_t>(s) * kStageBytes; };
    auto X_of = [&](int s) { return W_of(s) + kStageW; };
    auto SW_of = [&](int s) { return X_of(s) + kStageX; };
    auto SX_of = [&](int s) { return SW_of(s) + kStageS; };

    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(sfull(s), 4);
            mbar_init(empty(s), 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, 8);
        mbar_init(drain, 1);
        mbar_fence_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = tmem_slot;
    pdl_wait();

    if (warp == 0) {
        // ---------------- codes ----------------
        if (lane == 0) {
            prefetch_tmap(&tm_w);
            prefetch_tmap(&tm_a);
            const uint64_t pol = policy_evict_last();  // every tile of codes serves many tiles of Y
            const uint32_t bytes = kStageW + static_cast<uint32_t>(p.BN) * 128u;
            bool ok = true;
            int it = 0;
            for (int tile = first; tile < tiles && ok; tile += stride) {
                const int n0 = (tile % tiles_n) * kBM, m0 = (tile / tiles_n) * p.BN;
                for (int kb = 0; kb < num_kb; ++kb, ++it) {
                    const int s = it % kStages;
                    if (it >= kStages) ok = mbar_wait(empty(s), ((it / kStages) - 1) & 1, p.status);
                    if (!ok) break;
                    mbar_arrive_expect_tx(full(s), bytes);
                    tma_load_2d(W_of(s), &tm_w, (kb0 + kb) * 128, n0, full(s), pol);
                    tma_load_2d(X_of(s), &tm_a, (kb0 + kb) * 128, m0, full(s), pol);
                }
            }
            // every issued copy has landed before the block may exit
            for (int u = it > kStages ? it - kStages : 0; u < it; ++u)
                if (!mbar_wait(full(u % kStages), (u / kStages) & 1, p.status)) break;
        }
    } else if (warp == 1) {
        // ---------------- MMA ----------------
        if (lane == 0) {
            bool ok = true;
            int it = 0, t = 0;
            for (int tile = first; tile < tiles && ok; tile += stride, ++t) {
                if (t >= 1) ok = mbar_wait(acc_empty, (t - 1) & 1, p.status);
                if (!ok) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                for (int kb = 0; kb < num_kb; ++kb, ++it) {
                    const int s = it % kStages;
                    ok = mbar_wait(full(s), (it / kStages) & 1, p.status) && mbar_wait(sfull(s), (it / kStages) & 1, p.status);
                    if (!ok) break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    // scales of the k-block: weight half h, set q at sc + 8h + 4q; activations set q at sc + 16 + 8q
                    const uint32_t sc = tmem + kScaleCol + 32u * (it & 1);
                    const uint64_t sw = scales_desc(SW_of(s)), sx = scales_desc(SX_of(s));
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        copy_scales(sc + 4u * q, sw + 32u * q);                 // 512 bytes apart
                        copy_scales(sc + 8u + 4u * q, sw + 64u + 32u * q);      // half 1, 1024 bytes on
                        copy_scales(sc + 16u + 8u * q, sx + 32u * q);
                        if (p.BN > 128) copy_scales(sc + 20u + 8u * q, sx + 64u + 32u * q);
                    }
                    const uint64_t a0 = codes_desc(W_of(s)), a1 = codes_desc(W_of(s) + 128u * 128u), b = codes_desc(X_of(s));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint32_t acc = (kb != 0 || kk != 0) ? 1u : 0u;
                        // the two scales of this K = 64 are bytes 0, 1 or 2, 3 of a column
                        const uint32_t id = p.idesc | static_cast<uint32_t>(2 * (kk & 1)) << 4 | static_cast<uint32_t>(2 * (kk & 1)) << 29;
                        const uint32_t q = static_cast<uint32_t>(kk >> 1);
                        umma_mxf4(tmem, a0 + 2u * kk, b + 2u * kk, id, sc + 4u * q, sc + 16u + 8u * q, acc);
                        umma_mxf4(tmem + kAccCols, a1 + 2u * kk, b + 2u * kk, id, sc + 8u + 4u * q, sc + 16u + 8u * q, acc);
                    }
                    commit(empty(s));
                }
                if (ok) commit(acc_full);
            }
            // everything this thread issued has finished before TMEM is freed
            commit(drain);
            mbar_wait(drain, 0, p.status);
        }
        __syncwarp();
    } else if (warp < kFirstEpilogue || warp >= kFirstXScales) {
        // ---------------- scales ----------------
        const bool weight = warp < kFirstEpilogue;
        const int half = warp & 1;  // rows 128 half ..
        const uint8_t* scales = weight ? p.w_scales : p.a_scales;
        const int rows = weight ? p.N : p.m, span = weight ? kBM : p.BN;
        const int64_t table = static_cast<int64_t>(rows) * p.G;
        constexpr int kWords = kScaleWords<LOADS>;
        constexpr int kAhead = LOADS == SCALES_PAIR ? 2 : 1;  // k-blocks of a load
        auto first_row = [&](int tile) { return weight ? (tile % tiles_n) * kBM : (tile / tiles_n) * p.BN; };
        auto load = [&](uint32_t (&v)[4][kWords], int tile, int kb) {
            const int r0 = first_row(tile);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = half * 128 + lane + 32 * i;
                load_words<LOADS>(v[i], scales, static_cast<int64_t>(r0 + r) * p.G + (kb0 + kb) * 8, table, r < span && r0 + r < rows);
            }
        };
        bool ok = true;
        int it = 0, ltile = first, lkb = 0;  // what is loaded next
        uint32_t v[2][4][kWords];
        auto load_next = [&](uint32_t (&d)[4][kWords]) {
            if (ltile < tiles) load(d, ltile, lkb);
            if ((lkb += kAhead) >= num_kb) {
                lkb = 0;
                ltile += stride;
            }
        };
        if (LOADS != SCALES_PAIR) load_next(v[0]);
        load_next(v[1]);
        for (int tile = first; tile < tiles && ok; tile += stride) {
            const int r0 = first_row(tile);
            for (int kb = 0; kb < num_kb; ++kb, ++it) {
                const int s = it % kStages;
                uint2 c[4];
                auto advance = [&]() {  // the loaded words are due, others take their place
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < kWords; ++j) v[0][i][j] = v[1][i][j];
                    load_next(v[1]);
                };
                if constexpr (LOADS == SCALES_PAIR) {
                    if ((kb & 1) == 0) advance();
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        c[i] = (kb & 1) == 0 ? make_uint2(v[0][i][0], v[0][i][1]) : make_uint2(v[0][i][2], v[0][i][3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (LOADS == SCALES_WIDE) {
                            c[i] = make_uint2(v[0][i][0], v[0][i][1]);
                        } else {
                            const int r = half * 128 + lane + 32 * i;
                            c[i] = scale_bytes(v[0][i], scales, static_cast<int64_t>(r0 + r) * p.G + (kb0 + kb) * 8, table,
                                               r < span && r0 + r < rows, p.G - (kb0 + kb) * 8);
                        }
                    }
                    advance();
                }
                if (it >= kStages) ok = mbar_wait(empty(s), ((it / kStages) - 1) & 1, p.status);
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    ok = false;
                    break;
                }
                const uint32_t dst = (weight ? SW_of(s) : SX_of(s)) + 1024u * half + static_cast<uint32_t>(lane) * 16u;
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(c[0].x), "r"(c[1].x), "r"(c[2].x), "r"(c[3].x) : "memory");
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst + 512u), "r"(c[0].y), "r"(c[1].y), "r"(c[2].y), "r"(c[3].y)
                             : "memory");
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(sfull(s));
            }
        }
    } else {
        // ---------------- epilogue ----------------
        const int e = warp - kFirstEpilogue, half = e >> 2, quad = warp & 3;  // TMEM lanes 32 quad ..
        const int64_t N = p.N;
        int t = 0;
        for (int tile = first; tile < tiles; tile += stride, ++t) {
            const int n = (tile % tiles_n) * kBM + half * 128 + quad * 32 + lane, m0 = (tile / tiles_n) * p.BN;
            const bool ok = mbar_wait(acc_full, t & 1, p.status);
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t src = tmem + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(half) * kAccCols;
            if (S > 1) {  // the one tile's sums, [BN][256] over the stages, which no copy or MMA uses any more
                const uint32_t dst = base + static_cast<uint32_t>(half * 128 + quad * 32 + lane) * 4u;
                for (int c = 0; c < p.BN; c += 16) {
                    uint32_t r[16];
                    tmem_ld16(src + static_cast<uint32_t>(c), r);
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst + static_cast<uint32_t>(c + i) * 1024u), "r"(r[i]) : "memory");
                }
                break;
            }
            uint32_t y[kMaxBN / 2];  // BF16 pairs: columns 2i, 2i + 1
#pragma unroll
            for (int c = 0; c < kMaxBN / 16; ++c) {
                if (c * 16 < p.BN) {
                    uint32_t r[16];
                    tmem_ld16(src + 16u * c, r);
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[c * 8 + i] = pack_bf16x2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
                }
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty);
            if (n < p.N) {
                uint16_t* out = p.Y + static_cast<int64_t>(m0) * N + n;
                const int rows = min(p.BN, p.m - m0);
#pragma unroll
                for (int i = 0; i < kMaxBN / 2; ++i) {
                    if (2 * i < rows) out[0] = static_cast<uint16_t>(y[i]);
                    if (2 * i + 1 < rows) out[N] = static_cast<uint16_t>(y[i] >> 16);
                    out += 2 * N;
                }
            }
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncwarp();
    if (S > 1) {
        cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
        cluster.sync();  // all ranges' sums are there
        const int n0 = (first % tiles_n) * kBM, m0 = (first / tiles_n) * p.BN, cols = min(p.BN, p.m - m0);
        const int mine = cols > rank ? (cols - rank - 1) / S + 1 : 0;  // activation rows rank, rank + S, ...
        for (int i = threadIdx.x; i < mine * (kBM / 4); i += kThreads) {
            const int c = rank + (i >> 6) * S, r = (i & 63) * 4;
            float4 v[8];  // all ranks' sums of four weight rows, in flight together
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q < S)
                    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\tld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
                                 : "=f"(v[q].x), "=f"(v[q].y), "=f"(v[q].z), "=f"(v[q].w)
                                 : "r"(base + static_cast<uint32_t>(c * kBM + r) * 4u), "r"(q));
            float4 sum = v[0];
#pragma unroll
            for (int q = 1; q < 8; ++q)
                if (q < S) {
                    sum.x += v[q].x;
                    sum.y += v[q].y;
                    sum.z += v[q].z;
                    sum.w += v[q].w;
                }
            uint16_t* out = p.Y + static_cast<int64_t>(m0 + c) * p.N + n0 + r;
            const uint32_t lo = pack_bf16x2(sum.x, sum.y), hi = pack_bf16x2(sum.z, sum.w);
            if (n0 + r < p.N) out[0] = static_cast<uint16_t>(lo);
            if (n0 + r + 1 < p.N) out[1] = static_cast<uint16_t>(lo >> 16);
            if (n0 + r + 2 < p.N) out[2] = static_cast<uint16_t>(hi);
            if (n0 + r + 3 < p.N) out[3] = static_cast<uint16_t>(hi >> 16);
        }
        cluster.sync();  // no block leaves while a peer reads its sums
    }
    __syncthreads();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

// Activation rows per tile and ranges of K: the pair that ends first.  A k-block
// takes about 0.72 us and 0.9 ns per activation row (measured 0.8 at 64 rows, 0.9
// at 224: an MMA of few columns is hardly shorter than one of many), so tiles are
// wide and idle SMs are filled by splitting K, which costs about 3 us and the
// exchange of sums.
void pick_plan(int64_t m, int64_t N, int num_kb, int sms, int* bn_out, int* s_out) {
    int64_t best = INT64_MAX;
    for (int S = 1; S <= 8 && S <= num_kb; S *= 2) {
        for (int bn = 16; bn <= kMaxBN; bn += 16) {
            if (S > 1 && bn * kBM * 4 > static_cast<int>(kStages * kStageBytes)) continue;
            const int64_t tiles = ((N + kBM - 1) / kBM) * ((m + bn - 1) / bn);
            // (a cluster wants its SMs in one GPC: not every SM finds one)
            if (S > 1 && tiles * S > sms - 4 * S) continue;
            const int64_t kb = (num_kb + S - 1) / S, waves = S > 1 ? 1 : (tiles + sms - 1) / sms;
            const int64_t cost = waves * kb * (720 + bn * 9 / 10) + (S > 1 ? 3000 + bn * 10 : 0);  // ns
            if (cost < best) {
                best = cost;
                *bn_out = bn;
                *s_out = S;
            }
        }
    }
}

template <ScaleLoads LOADS>
cudaError_t launch(unsigned grid, const CUtensorMap& tm_w, const CUtensorMap& tm_a, const MatmulParams& p, cudaStream_t stream) {
    static std::atomic<int> configured[64];
    const size_t smem = kStages * kStageBytes + 1024;
    cudaError_t e = ensure_dynamic_smem(k_mx4_matmul<LOADS>, smem, configured);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.S);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.S > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k_mx4_matmul<LOADS>, tm_w, tm_a, p);
}

}  // namespace

cudaError_t launch_mx4_matmul(const Mx4View& w, const Mx4View& a, void* y, cudaStream_t stream) {
    if (w.cols == 0) return cudaMemsetAsync(y, 0, static_cast<size_t>(a.rows * w.rows * 2), stream);  // empty sums
    const int sms = device_info().sm_count;
    MatmulParams p{};
    p.Y = static_cast<uint16_t*>(y);
    p.w_scales = w.scales;
    p.a_scales = a.scales;
    p.N = static_cast<int>(w.rows);
    p.m = static_cast<int>(a.rows);
    p.G = static_cast<int>(w.cols / kMxBlock);
    p.num_kb = static_cast<int>((w.cols + kBK - 1) / kBK);
    pick_plan(a.rows, w.rows, p.num_kb, sms, &p.BN, &p.S);
    const uintptr_t tables = reinterpret_cast<uintptr_t>(w.scales) | reinterpret_cast<uintptr_t>(a.scales);
    const bool wide = p.G % 8 == 0 && (tables & 7u) == 0;
    // Pairs halve the sectors fetched, which counts where many tiles run (8192 x 14336 x
    // 4096: 238 -> 222 us, 8192 x 4096 x 14336: 205 -> 200); with K split, latency
    // counts, and they measured slower (64 x 4096 x 14336: 16.2 -> 16.6 us).
    const bool pair = p.S == 1 && p.G % 16 == 0 && (tables & 15u) == 0;
    // kind::mxf4: A and B E2M1 (1), scales UE8M0 (bit 23), N / 8, M / 128
    p.idesc = 1u << 7 | 1u << 10 | static_cast<uint32_t>(p.BN / 8) << 17 | 1u << 23 | 1u << 27;
    p.status = device_status_ptr();
    CUtensorMap tm_w, tm_a;
    if (!encode_2d(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.codes, static_cast<uint64_t>(w.cols / 2), static_cast<uint64_t>(w.rows),
                   static_cast<uint64_t>(w.cols / 2), 128, kBM, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_2d(&tm_a, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.codes, static_cast<uint64_t>(a.cols / 2), static_cast<uint64_t>(a.rows),
                   static_cast<uint64_t>(a.cols / 2), 128, static_cast<uint32_t>(p.BN), CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    const int64_t tiles = ((w.rows + kBM - 1) / kBM) * ((a.rows + p.BN - 1) / p.BN);
    if (tiles > 0x3FFFFFFF) return cudaErrorInvalidValue;
    const unsigned grid = static_cast<unsigned>(p.S > 1 ? tiles * p.S : (tiles < sms ? tiles : sms));
    return pair ? launch<SCALES_PAIR>(grid, tm_w, tm_a, p, stream)
                : (wide ? launch<SCALES_WIDE>(grid, tm_w, tm_a, p, stream) : launch<SCALES_ANY>(grid, tm_w, tm_a, p, stream));
}

}  // namespace mlxq
