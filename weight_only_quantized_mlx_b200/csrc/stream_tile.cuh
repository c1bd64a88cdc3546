// Weight streaming for a few activation rows, shared by the MX4 gemm and the
// expert layer.
//
// A warp works on tiles of 16 weight rows (two halves of 8: rows g of half A
// and half B belong to lanes 4g .. 4g + 3) and walks K in steps of 64 bytes of
// codes per row: lane (g, t) owns bytes 16t .. 16t + 15 of the step in its two
// rows.  It copies exactly those bytes with cp.async into its own ring in
// shared memory (kDepth steps in flight per warp, no block barrier), turns
// them into BF16 and feeds them to mma.sync m16n8k16 as the A operand, with
// the activations (8 columns per MMA) as B.  A sum over k may be taken in any
// order, so each MMA's k slots hold whatever columns the lane's bytes hold;
// the B fragment is loaded in the same order.
//
// The step's scales ride along: one 4-byte copy per lane, the four lanes of a
// row pair fetch what the quad needs.
#pragma once

#include "device_common.cuh"
#include "kernels.h"
#include "mx4_common.cuh"

namespace mlxq {

constexpr int kStreamWarps = 16;
constexpr int kStreamThreads = kStreamWarps * 32;
constexpr int kDepth = 8;                        // ring stages per warp
constexpr uint32_t kStageBytes = 512 + 512 + 128;  // codes of half A, of half B, scales
constexpr uint32_t kRingBytes = kDepth * kStageBytes;
constexpr uint32_t kAreaBytes = 16 * 68 * 4;     // a warp's partial sums: 16 rows x up to 64 columns (padded)

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 ldg128(const void* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A step of one tile for the lane: which rows, and where in K.
struct StepRows {
    int64_t row_a, row_b;  // weight rows of this lane in half A and half B
    bool live_a, live_b;   // false: read nothing (zeros)
};

// ---- 8-bit group-affine weights: 64 columns per step, 16 codes per lane ------------------
struct Q8Fmt {
    static constexpr int kStepCols = 64;
    static constexpr int kLaneCols = 16;

    struct Mat {
        const uint8_t* codes;
        const uint16_t* tables[2];  // scales, biases
        int64_t row_bytes;          // K
        int G, log_gs;
    };

    static __host__ Mat make(const WeightView& v) {
        int lg = 0;
        while ((1 << lg) < v.gs) ++lg;
        return Mat{reinterpret_cast<const uint8_t*>(v.packed), {v.scales, v.biases}, v.K, static_cast<int>(v.G), lg};
    }

    // lane t of a quad copies: 0 scale A, 1 bias A, 2 scale B, 3 bias B.  The
    // table entry sits in one half of an aligned 4-byte word (group size 32:
    // the step's two groups are the two halves; G is even there).
    static __device__ __forceinline__ void issue(const Mat& wa, const Mat& wb, uint32_t slot, int lane, const StepRows& r,
                                                 int step) {
        const int t = lane & 3;
        const int64_t off = static_cast<int64_t>(step) * 64 + 16 * t;
        const uint32_t dst = slot + static_cast<uint32_t>(lane) * 16u;
        cp_async16(dst, wa.codes + (r.live_a ? r.row_a * wa.row_bytes + off : 0), r.live_a ? 16u : 0u);
        cp_async16(dst + 512u, wb.codes + (r.live_b ? r.row_b * wb.row_bytes + off : 0), r.live_b ? 16u : 0u);
        const bool live = (t & 2) ? r.live_b : r.live_a;
        const int64_t e = ((t & 2) ? r.row_b : r.row_a) * wa.G + ((step * 64) >> wa.log_gs);
        const uint16_t* table = (t & 2) ? wb.tables[t & 1] : wa.tables[t & 1];
        cp_async4(slot + 1024u + static_cast<uint32_t>(lane) * 4u, table + (live ? (e & ~int64_t{1}) : 0), live ? 4u : 0u);
    }

    // One step: acc[n] += W(16 rows) x(8 columns n) over the step's k.
    // xp[n]: this lane's activation row of column tile n (0: column unused).
    template <int NT>
    static __device__ __forceinline__ void consume(const Mat& w, uint32_t slot, int lane, uint32_t row_parity, int step,
                                                   const uint16_t* const (&xp)[NT], int nt, float (&acc)[NT][4]) {
        const int t = lane & 3;
        const uint4 ca = lds128(slot + static_cast<uint32_t>(lane) * 16u);
        const uint4 cb = lds128(slot + 512u + static_cast<uint32_t>(lane) * 16u);
        const uint4 tb = lds128(slot + 1024u + static_cast<uint32_t>(lane & ~3) * 4u);
        // which half of the table words: the parity of row * G + group (both rows have one parity)
        const uint32_t hi = w.log_gs == 5 ? (t >> 1) : ((row_parity & w.G) ^ ((step * 64) >> w.log_gs)) & 1u;
        const uint32_t sel = hi ? 0x3244u : 0x1044u;  // halfword to the top of an fp32
        const float sa = __uint_as_float(__byte_perm(tb.x, 0u, sel)), ba = __uint_as_float(__byte_perm(tb.y, 0u, sel));
        const float sb = __uint_as_float(__byte_perm(tb.z, 0u, sel)), bb = __uint_as_float(__byte_perm(tb.w, 0u, sel));
        const uint32_t wa[4] = {ca.x, ca.y, ca.z, ca.w}, wb[4] = {cb.x, cb.y, cb.z, cb.w};
        const int64_t k0 = static_cast<int64_t>(step) * 64 + 16 * t;
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            uint32_t a[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                a[j][0] = pair<0>(wa[i + j], sa, ba);
                a[j][1] = pair<0>(wb[i + j], sb, bb);
                a[j][2] = pair<2>(wa[i + j], sa, ba);
                a[j][3] = pair<2>(wb[i + j], sb, bb);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (n >= nt) break;
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (xp[n]) x = ldg128(xp[n] + k0 + 4 * i);
                mma_bf16(acc[n], a[0][0], a[0][1], a[0][2], a[0][3], x.x, x.y);
                mma_bf16(acc[n], a[1][0], a[1][1], a[1][2], a[1][3], x.z, x.w);
            }
        }
    }

    // codes J and J + 1 of a word -> bf16(fma(s, q, b)) in two halves
    template <int J>
    static __device__ __forceinline__ uint32_t pair(uint32_t w, float s, float b) {
        const float q0 = __fsub_rn(code_magic<J>(w), kMagic), q1 = __fsub_rn(code_magic<J + 1>(w), kMagic);
        return pack_bf16x2(__fmaf_rn(s, q0, b), __fmaf_rn(s, q1, b));
    }
};

// ---- MX4 weights: 128 columns per step, 32 codes (one block) per lane ---------------------
struct Mx4Fmt {
    static constexpr int kStepCols = 128;
    static constexpr int kLaneCols = 32;

    struct Mat {
        const uint8_t* codes;
        const uint8_t* scales;
        int64_t row_bytes;     // K / 2
        int64_t scale_bytes;   // rows * G, the end of the table
        int G;                 // K / 32
    };

    static __host__ Mat make(const Mx4View& v) {
        return Mat{v.codes, v.scales, v.cols / 2, v.rows * (v.cols / kMxBlock), static_cast<int>(v.cols / kMxBlock)};
    }

    // The four scale bytes of a row and step start anywhere in a word: lane t
    // of a quad copies aligned word (t & 1) of row half t >> 1, bytes behind
    // the table left out.
    static __device__ __forceinline__ void issue(const Mat& wa, const Mat& wb, uint32_t slot, int lane, const StepRows& r,
                                                 int step) {
        const int t = lane & 3;
        const int64_t off = static_cast<int64_t>(step) * 64 + 16 * t;
        const bool in = off < wa.row_bytes;  // the last step of a row may be short
        const uint32_t dst = slot + static_cast<uint32_t>(lane) * 16u;
        const bool la = r.live_a && in, lb = r.live_b && in;
        cp_async16(dst, wa.codes + (la ? r.row_a * wa.row_bytes + off : 0), la ? 16u : 0u);
        cp_async16(dst + 512u, wb.codes + (lb ? r.row_b * wb.row_bytes + off : 0), lb ? 16u : 0u);
        const bool live = (t & 2) ? r.live_b : r.live_a;
        const int64_t e = ((((t & 2) ? r.row_b : r.row_a) * wa.G + 4 * static_cast<int64_t>(step)) & ~int64_t{3}) + 4 * (t & 1);
        const int64_t left = live ? wa.scale_bytes - e : 0;
        cp_async4(slot + 1024u + static_cast<uint32_t>(lane) * 4u, ((t & 2) ? wb.scales : wa.scales) + (left > 0 ? e : 0),
                  left > 4 ? 4u : (left > 0 ? static_cast<uint32_t>(left) : 0u));
    }

    template <int NT>
    static __device__ __forceinline__ void consume(const Mat& w, uint32_t slot, int lane, uint32_t row_low, int step,
                                                   const uint16_t* const (&xp)[NT], int nt, float (&acc)[NT][4]) {
        const int t = lane & 3;
        const uint4 ca = lds128(slot + static_cast<uint32_t>(lane) * 16u);
        const uint4 cb = lds128(slot + 512u + static_cast<uint32_t>(lane) * 16u);
        const uint4 tb = lds128(slot + 1024u + static_cast<uint32_t>(lane & ~3) * 4u);
        const int64_t k0 = static_cast<int64_t>(step) * 128 + 32 * t;
        const bool in = k0 < 2 * w.row_bytes;
        // byte (row * G + 4 step + t) & 3 .. of the two words; rows of both halves are congruent
        const uint32_t sh = 8u * ((row_low * static_cast<uint32_t>(w.G)) & 3u);
        uint32_t ea = in ? (__funnelshift_r(tb.x, tb.y, sh) >> (8 * t)) & 255u : 0u;
        uint32_t eb = in ? (__funnelshift_r(tb.z, tb.w, sh) >> (8 * t)) & 255u : 0u;
        // W = code 2^-126 * 2^(E - 1): one exact product while E <= 128 (scales up
        // to 2); larger scales (and NaN) take a second factor
        const bool big = __any_sync(0xFFFFFFFFu, ea > 128u || eb > 128u);
        const uint32_t fa = scale_factor(ea), fb = scale_factor(eb);
        const uint32_t wa[4] = {ca.x, ca.y, ca.z, ca.w}, wb[4] = {cb.x, cb.y, cb.z, cb.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t a[4], b[4];
            a[0] = mul_bf16x2(e2m1_pair<0>(wa[i]), fa);
            a[1] = mul_bf16x2(e2m1_pair<1>(wa[i]), fa);
            a[2] = mul_bf16x2(e2m1_pair<2>(wa[i]), fa);
            a[3] = mul_bf16x2(e2m1_pair<3>(wa[i]), fa);
            b[0] = mul_bf16x2(e2m1_pair<0>(wb[i]), fb);
            b[1] = mul_bf16x2(e2m1_pair<1>(wb[i]), fb);
            b[2] = mul_bf16x2(e2m1_pair<2>(wb[i]), fb);
            b[3] = mul_bf16x2(e2m1_pair<3>(wb[i]), fb);
            if (big) {
                const uint32_t ga = scale_rest(ea), gb = scale_rest(eb);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    a[j] = mul_bf16x2(a[j], ga);
                    b[j] = mul_bf16x2(b[j], gb);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (n >= nt) break;
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (xp[n] && in) x = ldg128(xp[n] + k0 + 8 * i);
                mma_bf16(acc[n], a[0], b[0], a[1], b[1], __byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632));
                mma_bf16(acc[n], a[2], b[2], a[3], b[3], __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
            }
        }
    }

    // 2^(min(E, 128) - 1), twice: exponent field min(E, 128) + 126 (at most 254);
    // E = 0 is field 126 as well as 2^-127 * 2^126 = 1/2 asks.
    static __device__ __forceinline__ uint32_t scale_factor(uint32_t e) { return ((min(e, 128u) + 126u) << 7) * 0x00010001u; }
    // the rest: 2^(E - 128) for E > 128, NaN for 255, else 1
    static __device__ __forceinline__ uint32_t scale_rest(uint32_t e) {
        return (e == 255u ? 0x7FFFu : (e > 128u ? (e - 1u) << 7 : 0x3F80u)) * 0x00010001u;
    }
};

// How many warps share a tile's K (1, 2, 4, 8, 16): the choice that ends
// first, counting a tile as its steps plus about two steps for joining the
// warps' sums where more than one shares it.
__device__ __forceinline__ int pick_k_warps(int tiles, int steps) {
    int best = 1, best_cost = 0x7FFFFFFF;
#pragma unroll
    for (int wk = 1; wk <= kStreamWarps; wk *= 2) {
        const int groups = kStreamWarps / wk;
        const int cost = ((tiles + groups - 1) / groups) * ((steps + wk - 1) / wk + (wk > 1 ? 2 : 0));
        if (cost < best_cost) {
            best_cost = cost;
            best = wk;
        }
    }
    return best;
}

// Which activation rows an expert's MMA columns hold.  A slot is token * top_k
// + choice.  NT == 1 (up to 8 tokens): column = token, eight entries per
// expert, -1 where the token did not choose it.  Otherwise: the expert's slots
// one after another, `cnt` of them, padded with -1 to a multiple of 8.
struct Columns {
    const int16_t* cols;
    const int16_t* off;  // first entry of active expert a
    const int16_t* cnt;
    int top_k;
    __device__ __forceinline__ int slot(int a, int c) const { return cols[off[a] + c]; }
};

// A warp's share of a phase: its group of k_warps warps takes the tiles
// group, group + groups, ...; within a tile it takes the steps kw, kw +
// k_warps, ... of the concatenated experts.
struct Share {
    int tiles, steps, experts;  // steps of one expert; experts concatenated along K
    int k_warps, groups, group, kw;
    __device__ __forceinline__ Share(int tiles_, int steps_, int experts_, int warp)
        : tiles(tiles_), steps(steps_), experts(experts_) {
        k_warps = pick_k_warps(tiles, steps * experts);
        groups = kStreamWarps / k_warps;
        group = warp / k_warps;
        kw = warp - group * k_warps;
    }
    __device__ __forceinline__ int own_steps() const {  // per tile
        const int all = steps * experts;
        return kw < all ? (all - kw + k_warps - 1) / k_warps : 0;
    }
};

struct Cursor {
    int tile, a, step;
    __device__ __forceinline__ explicit Cursor(const Share& s) : tile(s.group), a(s.kw / s.steps), step(s.kw % s.steps) {
        if (a >= s.experts) tile = s.tiles;  // no step of any tile is this warp's
    }
    __device__ __forceinline__ void next(const Share& s) {
        step += s.k_warps;
        while (step >= s.steps) {
            step -= s.steps;
            ++a;
        }
        if (a >= s.experts) {
            a = s.kw / s.steps;
            step = s.kw % s.steps;
            tile += s.groups;
        }
    }
};

// Barrier of the warps that share a tile.
__device__ __forceinline__ void group_sync(int group, int k_warps) {
    if (k_warps == 1) __syncwarp();
    else named_bar_sync(1u + static_cast<uint32_t>(group), static_cast<uint32_t>(k_warps) * 32u);
}

// y[token][row] = sum over experts a and columns k of W_a[row, k] h[slot][k]
// for the rows row_lo .. row_hi - 1 of y: a block's whole share of the down
// projection, or (EXPERTS false, one "expert", slot = token) of a gemm.  Tiles
// are 16 rows; every expert's slice of a tile goes into one accumulator, so
// the sum over experts needs no second pass and no atomics: with up to 8
// tokens (NT == 1) column = token and the fragment itself accumulates, else
// each warp adds an expert's columns to its own [16][tokens] sums in shared
// memory.  The warps that share a tile join in warp order, so results do not
// depend on timing.  `ready` runs once the ring has been filled for the first
// time (weights only) and before h is read; false ends the phase.
template <class F, int NT, bool EXPERTS, class Ready>
__device__ __forceinline__ void stream_rows(const typename F::Mat& w, int64_t rows_per_expert, int row_lo, int row_hi,
                                            int experts, const int16_t* act, const Columns& cm, const uint16_t* h, int K,
                                            int tokens, uint16_t* y, int64_t y_stride, uint32_t ring, uint8_t* areas,
                                            Ready ready) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const Share sh((row_hi - row_lo + 15) / 16, (K + F::kStepCols - 1) / F::kStepCols, experts, warp);
    float* area = reinterpret_cast<float*>(areas + warp * kAreaBytes);
    const float* group_area = reinterpret_cast<const float*>(areas + sh.group * sh.k_warps * kAreaBytes);
    constexpr int kAreaFloats = kAreaBytes / 4;
    constexpr int kStride = NT * 8 + 1;          // NT > 1: floats per row of the area
    constexpr int kBatch = NT == 1 ? 8 : 1;      // tiles between two joins

    Cursor pc(sh);
    uint32_t pslot = 0;
    auto issue = [&]() {
        if (pc.tile < sh.tiles) {
            const int64_t base = EXPERTS ? static_cast<int64_t>(act[pc.a]) * rows_per_expert : 0;
            const int r = row_lo + pc.tile * 16 + g;
            const StepRows rows{base + r, base + r + 8, r < row_hi, r + 8 < row_hi};
            F::issue(w, w, ring + pslot * kStageBytes, lane, rows, pc.step);
            pc.next(sh);
        }
        cp_async_commit();
        pslot = (pslot + 1) % kDepth;
    };
#pragma unroll 1
    for (int i = 0; i < kDepth - 1; ++i) issue();
    if (!ready()) {
        cp_async_wait<0>();
        return;
    }

    uint32_t cslot = 0;
    const int own = sh.own_steps();
    for (int tile0 = sh.group; tile0 < sh.tiles; tile0 += sh.groups * kBatch) {
        int batch = 0;
        for (; batch < kBatch; ++batch) {
            const int tile = tile0 + batch * sh.groups;
            if (tile >= sh.tiles) break;
            float acc[NT][4];
            const uint16_t* xp[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
                xp[n] = nullptr;
            }
            if (NT > 1) {
                for (int i = lane; i < 16 * kStride; i += 32) area[i] = 0.f;
                __syncwarp();
            }
            auto scatter = [&](int a, int nt) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (n >= nt) break;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int c = n * 8 + 2 * t + i;
                        int token = c;
                        if (EXPERTS) {
                            const int s = cm.slot(a, c);
                            token = s < 0 ? -1 : s / cm.top_k;
                        }
                        if (token >= 0) {
                            area[g * kStride + token] += acc[n][i];
                            area[(g + 8) * kStride + token] += acc[n][2 + i];
                        }
                    }
                    acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
                }
                __syncwarp();
            };
            int a = -1, nt = 0;
            int ca = sh.kw / sh.steps, step = sh.kw % sh.steps;
            for (int it = 0; it < own; ++it) {
                if (ca != a) {
                    if (NT > 1 && a >= 0) scatter(a, nt);
                    a = ca;
                    nt = NT == 1 ? 1 : (EXPERTS ? (cm.cnt[a] + 7) / 8 : (tokens + 7) / 8);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const int c = n * 8 + g;
                        const int s = n < nt ? (EXPERTS ? cm.slot(a, c) : (c < tokens ? c : -1)) : -1;
                        xp[n] = s >= 0 ? h + static_cast<int64_t>(s) * K : nullptr;
                    }
                }
                cp_async_wait<kDepth - 2>();
                __syncwarp();  // the quad's scales have landed; the slot refilled below is read out
                issue();
                const uint32_t low = (EXPERTS ? static_cast<uint32_t>(act[a]) * static_cast<uint32_t>(rows_per_expert) : 0u) +
                                     static_cast<uint32_t>(row_lo + tile * 16 + g);
                F::template consume<NT>(w, ring + cslot * kStageBytes, lane, low, step, xp, nt, acc);
                cslot = (cslot + 1) % kDepth;
                step += sh.k_warps;
                while (step >= sh.steps) {
                    step -= sh.steps;
                    ++ca;
                }
            }
            if (NT == 1) {
                reinterpret_cast<float4*>(area)[batch * 32 + lane] = make_float4(acc[0][0], acc[0][1], acc[0][2], acc[0][3]);
            } else if (a >= 0) {
                scatter(a, nt);
            }
        }
        group_sync(sh.group, sh.k_warps);
        const int me = sh.kw * 32 + lane, all = sh.k_warps * 32;
        if (NT == 1) {
            for (int i = me; i < batch * 32; i += all) {
                float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int v = 0; v < sh.k_warps; ++v) {
                    const float4 p = reinterpret_cast<const float4*>(group_area + v * kAreaFloats)[i];
                    s.x += p.x;
                    s.y += p.y;
                    s.z += p.z;
                    s.w += p.w;
                }
                const int r = row_lo + (tile0 + (i >> 5) * sh.groups) * 16 + ((i & 31) >> 2), c = 2 * (i & 3);
                const uint32_t lo = pack_bf16x2(s.x, s.y), hi = pack_bf16x2(s.z, s.w);
                if (c < tokens && r < row_hi) y[c * y_stride + r] = static_cast<uint16_t>(lo);
                if (c + 1 < tokens && r < row_hi) y[(c + 1) * y_stride + r] = static_cast<uint16_t>(lo >> 16);
                if (c < tokens && r + 8 < row_hi) y[c * y_stride + r + 8] = static_cast<uint16_t>(hi);
                if (c + 1 < tokens && r + 8 < row_hi) y[(c + 1) * y_stride + r + 8] = static_cast<uint16_t>(hi >> 16);
            }
        } else {
            const int r0 = row_lo + tile0 * 16;
            for (int i = me; i < 16 * tokens; i += all) {
                const int r = i & 15, c = i >> 4;
                float s = 0.f;
                for (int v = 0; v < sh.k_warps; ++v) s += group_area[v * kAreaFloats + r * kStride + c];
                if (r0 + r < row_hi) y[c * y_stride + r0 + r] = static_cast<uint16_t>(pack_bf16x2(s, 0.f));
            }
        }
        group_sync(sh.group, sh.k_warps);
    }
    cp_async_wait<0>();
}

}  // namespace mlxq
