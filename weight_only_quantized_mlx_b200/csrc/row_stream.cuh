// Weight streaming for a few activation rows: copies, dequantisation and
// products of one step for 8-bit group-affine and MX4 weights, and the phase in
// which a block's warps share the activations (gate and up of the expert layer,
// the MX4 gemm).
//
// A warp works on tiles of 16 weight rows (two halves of 8: rows g of half A
// and half B belong to lanes 4g .. 4g + 3) and walks K in steps of 64 bytes of
// codes per row.  Lane (g, t) copies bytes 16t .. 16t + 15 of the step in its
// two rows with cp.async into the warp's own ring in shared memory (several steps
// in flight per warp, no block barrier).  The codes become 16-bit operands in
// registers and go to mma.sync m16n8k16 as A, with the activations (8 columns
// per MMA) as B.  A sum over k may be taken in any order, so each MMA's k slots
// hold whatever columns the lane's codes belong to; activations are kept in the
// matching order, in "pieces" of 8 columns (16 bytes).
//
// The step's scales ride along: one 4-byte copy per lane, the four lanes of a
// row pair fetch what the quad needs.
#pragma once

#include <type_traits>

#include "device_common.cuh"
#include "kernels.h"
#include "mx4_common.cuh"

namespace mlxq {

constexpr int kStreamWarps = 16;
constexpr int kStreamThreads = kStreamWarps * 32;
constexpr uint32_t kStageBytes = 512 + 512 + 128;  // codes of half A, of half B, scales

// Stages of a warp's ring: six where latency counts; with more columns four, the
// room of the others holds activations.
template <int NT>
struct Ring {
    static constexpr int kDepth = NT == 1 ? 6 : 4;
    static constexpr uint32_t kBytes = kDepth * kStageBytes;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A column's unit: 2^(f - 141) with f the largest BF16 exponent field among its
// activations (15 .. 254; infinities and NaN stay what they are in any unit).
// The largest lies in [2^14, 2^15) units, the upper end of FP16.
constexpr uint32_t kXTop = 14;
__device__ __forceinline__ uint32_t x_field(uint32_t field) { return min(max(field, 1u + kXTop), 254u); }
__device__ __forceinline__ float x_unit(uint32_t field) { return __uint_as_float((x_field(field) - kXTop) << 23); }
__device__ __forceinline__ float x_inverse(uint32_t field) { return __uint_as_float((254u + kXTop - x_field(field)) << 23); }  // 1 / unit

// Columns' units from their fields; a column behind the last one has that one's.
struct FieldUnit {
    const uint32_t* field;
    int cols;
    __device__ __forceinline__ float operator()(int c) const { return x_unit(field[min(c, cols - 1)]); }
};

// ---- 8-bit group-affine weights: 64 columns per step, 16 codes per lane ------------------
struct Q8Fmt {
    static constexpr int kStepCols = 64;
    static constexpr int kPieces = 2;  // 8-column pieces of a lane and step

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

    static __device__ __forceinline__ int group(const Mat& w, int step) { return (step * 64) >> w.log_gs; }

    // Where a lane copies a tile from, at the present step.  Lane t of a quad also
    // copies table entries: 0 scale A, 1 bias A, 2 scale B, 3 bias B.  An entry
    // sits in one half of an aligned 4-byte word (group size 32: the step's two
    // groups are the two halves; G is even there).  A dead half walks the
    // matrix's first row and reads no bytes of it.
    struct Feed {
        const uint8_t *a, *b, *table;
        uint32_t na, nb, nt;  // bytes to read: 16 or 0, 4 or 0
        uint32_t odd;         // parity of the row's first table entry
        int step;
    };
    static __device__ __forceinline__ void start(Feed& f, const Mat& wa, const Mat& wb, int64_t row_a, int64_t row_b, bool live_a,
                                                 bool live_b, int lane, int step) {
        const int t = lane & 3, off = step * 64 + 16 * t;
        f.a = wa.codes + (live_a ? row_a * wa.row_bytes : 0) + off;
        f.b = wb.codes + (live_b ? row_b * wb.row_bytes : 0) + off;
        f.na = live_a ? 16u : 0u;
        f.nb = live_b ? 16u : 0u;
        const bool live = (t & 2) ? live_b : live_a;
        const int64_t e = live ? ((t & 2) ? row_b : row_a) * wa.G : 0;
        f.odd = static_cast<uint32_t>(e) & 1u;
        f.table = reinterpret_cast<const uint8_t*>(((t & 2) ? wb.tables[t & 1] : wa.tables[t & 1]) + (e - f.odd));
        f.nt = live ? 4u : 0u;
        f.step = step;
    }
    // Copy the step into the stage at slot and go on by `by` steps.
    static __device__ __forceinline__ void issue(const Mat& w, Feed& f, uint32_t slot, int lane, int by) {
        const uint32_t dst = slot + static_cast<uint32_t>(lane) * 16u;
        cp_async16(dst, f.a, f.na);
        cp_async16(dst + 512u, f.b, f.nb);
        const uint32_t e = (f.odd + static_cast<uint32_t>(group(w, f.step))) >> 1;
        cp_async4(dst + 1024u - static_cast<uint32_t>(lane) * 12u, f.table + 4u * e, f.nt);
        f.a += by * 64;
        f.b += by * 64;
        f.step += by;
    }

    // What a lane needs to read its scales: the parity of its row's first entry.
    static __device__ __forceinline__ uint32_t row_key(const Mat& w, uint32_t row) { return row & static_cast<uint32_t>(w.G) & 1u; }

    // One step: acc[n] += W(16 rows) x(8 columns n) / kUnit, n < N, over the step's k.
    static constexpr float kUnit = 1.f;
    // x(i, n): this lane's piece i of column tile n.
    template <int NT, int N, class X>
    static __device__ __forceinline__ void consume(const Mat& w, uint32_t slot, int lane, uint32_t key, int step,
                                                   float (&acc)[NT][4], X x) {
        const int t = lane & 3;
        const uint4 ca = lds128(slot + static_cast<uint32_t>(lane) * 16u);
        const uint4 cb = lds128(slot + 512u + static_cast<uint32_t>(lane) * 16u);
        const uint4 tb = lds128(slot + 1024u + static_cast<uint32_t>(lane & ~3) * 4u);
        const uint32_t hi = w.log_gs == 5 ? static_cast<uint32_t>(t >> 1) : (key + static_cast<uint32_t>(group(w, step))) & 1u;
        const uint32_t sel = hi ? 0x3244u : 0x1044u;  // halfword to the top of an fp32
        const float sa = __uint_as_float(__byte_perm(tb.x, 0u, sel)), ba = __uint_as_float(__byte_perm(tb.y, 0u, sel));
        const float sb = __uint_as_float(__byte_perm(tb.z, 0u, sel)), bb = __uint_as_float(__byte_perm(tb.w, 0u, sel));
        const float2 sa2 = make_float2(sa, sa), ba2 = make_float2(ba, ba), sb2 = make_float2(sb, sb), bb2 = make_float2(bb, bb);
        const uint32_t wa[4] = {ca.x, ca.y, ca.z, ca.w}, wb[4] = {cb.x, cb.y, cb.z, cb.w};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t a[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                a[j][0] = pair<0>(wa[2 * i + j], sa2, ba2);
                a[j][1] = pair<0>(wb[2 * i + j], sb2, bb2);
                a[j][2] = pair<2>(wa[2 * i + j], sa2, ba2);
                a[j][3] = pair<2>(wb[2 * i + j], sb2, bb2);
            }
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const uint4 v = x(i, n);
                mma_bf16(acc[n], a[0][0], a[0][1], a[0][2], a[0][3], v.x, v.y);
                mma_bf16(acc[n], a[1][0], a[1][1], a[1][2], a[1][3], v.z, v.w);
            }
        }
    }

    // codes J and J + 1 of a word -> bf16(fma(s, q, b)) in two halves
    template <int J>
    static __device__ __forceinline__ uint32_t pair(uint32_t w, float2 s, float2 b) {
        const float2 q = __fadd2_rn(make_float2(code_magic<J>(w), code_magic<J + 1>(w)), make_float2(-kMagic, -kMagic));
        const float2 v = __ffma2_rn(s, q, b);
        return pack_bf16x2(v.x, v.y);
    }

    // Rows of h, each value the sum of two BF16 parts.  A quad's loads of one piece (lanes t
    // = 0 .. 3, 16 bytes each) are 64 bytes, the second parts' 64 bytes behind, so that
    // eight lanes read whole lines.  h_row: length of a row; place: where column k's first part is
    // (the second: 32 on).
    static constexpr bool kPair = true;
    static __host__ __device__ __forceinline__ int h_row(int cols) { return (cols + kStepCols - 1) / kStepCols * (2 * kStepCols); }
    static __device__ __forceinline__ int place(int k) { return (k & ~63) * 2 + (k >> 3 & 1) * 64 + (k >> 4 & 3) * 8 + (k & 7); }

    // shared activations: BF16 as they are; piece r of a step (columns 8r ..) is lane t = r / 2's piece i = r % 2
    static constexpr bool kScaled = false;
    static __device__ __forceinline__ int piece_index(int r) { return r % kPieces; }
    static __device__ __forceinline__ int piece_lane(int r) { return r / kPieces; }
    template <int NT, int N>
    static __device__ __forceinline__ void consume_shared(const Mat& w, uint32_t slot, int lane, uint32_t key, int step,
                                                          float (&acc)[NT][4], uint32_t x, uint32_t piece_stride,
                                                          const uint32_t (&xo)[NT], bool&, const uint32_t*, int) {
        consume<NT, N>(w, slot, lane, key, step, acc,
                       [&](int i, int n) { return lds128(x + static_cast<uint32_t>(i) * piece_stride + xo[n]); });
    }
};

// ---- MX4 weights: 128 columns per step, 32 codes (one block) per lane ---------------------
struct Mx4Fmt {
    static constexpr int kStepCols = 128;
    static constexpr int kPieces = 4;

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
    // the table left out.  The last step of a row may be short.
    struct Feed {
        const uint8_t *a, *b, *table;
        int ca, cb;  // bytes of codes from the lane's first one to the row's end
        int ct;      // scale bytes left in the table
    };
    static __device__ __forceinline__ void start(Feed& f, const Mat& wa, const Mat& wb, int64_t row_a, int64_t row_b, bool live_a,
                                                 bool live_b, int lane, int step) {
        const int t = lane & 3, off = step * 64 + 16 * t;
        f.a = wa.codes + (live_a ? row_a * wa.row_bytes : 0) + off;
        f.b = wb.codes + (live_b ? row_b * wb.row_bytes : 0) + off;
        f.ca = live_a ? static_cast<int>(wa.row_bytes) - off : 0;
        f.cb = live_b ? static_cast<int>(wa.row_bytes) - off : 0;
        const bool live = (t & 2) ? live_b : live_a;
        // (a dead half reads the first row's scales: any will do, its codes are zeros)
        const int64_t e = (live ? (((t & 2) ? row_b : row_a) * wa.G) & ~int64_t{3} : 0) + 4 * (t & 1) + 4 * step;
        const int64_t left = wa.scale_bytes - e;
        f.table = ((t & 2) ? wb.scales : wa.scales) + e;
        f.ct = left > 0x40000000 ? 0x40000000 : static_cast<int>(left);
    }
    // Copy the step into the stage at slot and go on by `by` steps.  (A copy of no
    // bytes does not touch its source, which may lie behind the matrix.)
    static __device__ __forceinline__ void issue_at(Feed& f, uint32_t dst, uint32_t tdst, int by) {
        cp_async16(dst, f.a, f.ca > 0 ? 16u : 0u);
        cp_async16(dst + 512u, f.b, f.cb > 0 ? 16u : 0u);
        cp_async4(tdst, f.table, static_cast<uint32_t>(min(max(f.ct, 0), 4)));
        f.a += by * 64;
        f.b += by * 64;
        f.table += by * 4;
        f.ca -= by * 64;
        f.cb -= by * 64;
        f.ct -= by * 4;
    }
    static __device__ __forceinline__ void issue(const Mat&, Feed& f, uint32_t slot, int lane, int by) {
        const uint32_t dst = slot + static_cast<uint32_t>(lane) * 16u;
        issue_at(f, dst, dst + 1024u - static_cast<uint32_t>(lane) * 12u, by);
    }

    // the shift that brings a row's first scale byte to the bottom of its first word
    static __device__ __forceinline__ uint32_t row_key(const Mat& w, uint32_t row) {
        return 8u * ((row * static_cast<uint32_t>(w.G)) & 3u);
    }

    template <int NT, int N, class X>
    static __device__ __forceinline__ void consume(const Mat& w, uint32_t slot, int lane, uint32_t key, int step,
                                                   float (&acc)[NT][4], X x) {
        const int t = lane & 3;
        const uint4 ca = lds128(slot + static_cast<uint32_t>(lane) * 16u);
        const uint4 cb = lds128(slot + 512u + static_cast<uint32_t>(lane) * 16u);
        const uint4 tb = lds128(slot + 1024u + static_cast<uint32_t>(lane & ~3) * 4u);
        const bool in = step * 64 + 16 * t < static_cast<int>(w.row_bytes);
        uint32_t ea = (__funnelshift_r(tb.x, tb.y, key) >> (8 * t)) & 255u;
        uint32_t eb = (__funnelshift_r(tb.z, tb.w, key) >> (8 * t)) & 255u;
        if (!in) ea = eb = 0u;  // codes there are zeros; another row's scale must not make them NaN
        // W / 4 = code 2^-126 * 2^(E - 3): one exact product while E <= 128 (scales up
        // to 2); larger scales (and NaN) take a second factor
        const bool big = __any_sync(0xFFFFFFFFu, max(ea, eb) > 128u);
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
            for (int n = 0; n < N; ++n) {
                const uint4 v = x(i, n);
                mma_bf16(acc[n], a[0], b[0], a[1], b[1], v.x, v.y);
                mma_bf16(acc[n], a[2], b[2], a[3], b[3], v.z, v.w);
            }
        }
    }

    // Weights are multiplied as W / kUnit: 6 * 2^127 is beyond BF16 where its product
    // with x need not be (and a quarter of the least, 2^-130, BF16 still holds).
    static constexpr float kUnit = 4.f;
    // 2^(min(E, 128) - 3), twice: exponent field min(E, 128) + 124; E = 0 is field 124
    // as well as 2^-127 * 2^126 / 4 = 1/8 asks.
    static __device__ __forceinline__ uint32_t scale_factor(uint32_t e) { return ((min(e, 128u) + 124u) << 7) * 0x00010001u; }
    // the rest: 2^(E - 128) for E > 128, NaN for 255, else 1
    static __device__ __forceinline__ uint32_t scale_rest(uint32_t e) {
        return (e == 255u ? 0x7FFFu : (e > 128u ? (e - 1u) << 7 : 0x3F80u)) * 0x00010001u;
    }

    // rows of h as for 8 bits; and a word of codes comes apart as 0 4 1 5 2 6 3 7
    static constexpr bool kPair = true;
    static __host__ __device__ __forceinline__ int h_row(int cols) { return (cols + kStepCols - 1) / kStepCols * (2 * kStepCols); }
    static __device__ __forceinline__ int place(int k) {
        return (k & ~127) * 2 + (k >> 3 & 3) * 64 + (k >> 5 & 3) * 8 + ((k & 3) << 1 | (k >> 2 & 1));
    }
};

// ---- MX4 weights with shared activations: products in FP16 ---------------------------------
// cvt.rn.f16x2.e2m1x2 turns a byte of codes into two FP16 values in one
// instruction (3.1 against 6.4 SM cycles per word of 8 codes for the BF16 form
// above, which has to place bits and multiply), so the codes go to the tensor
// pipe unscaled: an MMA pair covers one block of 32 columns, and its fp32 result
// is multiplied by the rows' block scales as it is added to the sums.
// Activations are held as FP16 in units that bring their column's largest power of
// two to 2^14: a BF16 value's 8 bits then fit down to 2^-31 of the column's largest
// magnitude, so products are exact; smaller values are off by at most 2^-39 of the
// largest.  A block's sum is below 32 * 6 * 2^15 < 2^23 units.
struct Mx4HalfFmt : Mx4Fmt {
    // the 16-byte unit of block b in row g sits at unit b ^ (g / 2), so that the
    // 32 lanes' word loads (row g, word t) touch 32 banks
    static __device__ __forceinline__ void issue(const Mat&, Feed& f, uint32_t slot, int lane, int by) {
        const int g = lane >> 2, t = lane & 3;
        issue_at(f, slot + static_cast<uint32_t>(g * 64 + ((t ^ (g >> 1)) & 3) * 16), slot + 1024u + static_cast<uint32_t>(lane) * 4u, by);
    }

    // rows of h: FP16 in units of their largest power of two, in order
    static constexpr bool kPair = false;

    static constexpr bool kScaled = true;
    static __device__ __forceinline__ int piece_index(int r) { return r >> 2; }  // block
    static __device__ __forceinline__ int piece_lane(int r) { return r & 3; }

    // acc holds sums in the columns' units while `plain`, and turns to plain
    // numbers, for the rest of the tile, at the first step with a scale outside
    // 2^-63 .. 2^64: there each product meets scale and unit in the order that
    // does not leave fp32 on the way.
    // MT tiles of 16 rows, their stages one behind the other: each piece of the
    // activations is read once for all of them.
    // x(b, n): this lane's piece of block b and column tile n; unit(c): column c's unit.
    template <int MT, int NT, int N, class X, class Unit>
    static __device__ __forceinline__ void consume_tiles(const Mat& w, uint32_t slot, int lane, const uint32_t (&key)[MT], int step,
                                                         float (&acc)[MT][NT][4], bool& plain, X x, Unit unit) {
        const int g = lane >> 2, t = lane & 3;
        const int left = w.G - 4 * step;  // blocks left in the row; behind it codes are zeros, and scales must not be NaN
        uint32_t ea[MT], eb[MT], mid = 0x80808080u;  // the two top bits of every byte differ: 64 .. 191
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const uint4 tb = lds128(slot + j * kStageBytes + 1024u + static_cast<uint32_t>(lane & ~3) * 4u);
            ea[j] = __funnelshift_r(tb.x, tb.y, key[j]);
            eb[j] = __funnelshift_r(tb.z, tb.w, key[j]);
        }
        if (left < 4) {
            const uint32_t keep = (1u << (8 * left)) - 1u;
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                ea[j] = (ea[j] & keep) | (0x7F7F7F7Fu & ~keep);
                eb[j] = (eb[j] & keep) | (0x7F7F7F7Fu & ~keep);
            }
        }
#pragma unroll
        for (int j = 0; j < MT; ++j) mid &= (ea[j] ^ (ea[j] << 1)) & (eb[j] ^ (eb[j] << 1));
        if (plain && !__all_sync(0xFFFFFFFFu, mid == 0x80808080u)) {
            plain = false;
#pragma unroll
            for (int j = 0; j < MT; ++j) to_numbers<NT>(acc[j], t, unit);
        }
        float sa[MT][4], sb[MT][4];
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            e8m0x4(ea[j], sa[j]);
            e8m0x4(eb[j], sb[j]);
        }
        // block b of row g, word t: bits 4 and 5 of the address hold b ^ (g / 2)
        const uint32_t row = slot + static_cast<uint32_t>(g * 64 + ((g >> 1) & 3) * 16 + t * 4);
        if (plain) {
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const uint32_t at = row ^ static_cast<uint32_t>(b * 16);
                uint32_t a[MT][4], c[MT][4];
#pragma unroll
                for (int j = 0; j < MT; ++j) {
                    e2m1x8_f16(lds32(at + j * kStageBytes), a[j]);
                    e2m1x8_f16(lds32(at + j * kStageBytes + 512u), c[j]);
                }
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const uint4 v = x(b, n);
#pragma unroll
                    for (int j = 0; j < MT; ++j) {
                        float d[4];
                        mma_f16_first(d, a[j][0], c[j][0], a[j][1], c[j][1], v.x, v.y);
                        mma_f16(d, a[j][2], c[j][2], a[j][3], c[j][3], v.z, v.w);
                        acc[j][n][0] = __fmaf_rn(d[0], sa[j][b], acc[j][n][0]);
                        acc[j][n][1] = __fmaf_rn(d[1], sa[j][b], acc[j][n][1]);
                        acc[j][n][2] = __fmaf_rn(d[2], sb[j][b], acc[j][n][2]);
                        acc[j][n][3] = __fmaf_rn(d[3], sb[j][b], acc[j][n][3]);
                    }
                }
            }
        } else {
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {
#pragma unroll
                for (int j = 0; j < MT; ++j) {
                    const uint32_t at = (row ^ static_cast<uint32_t>(b * 16)) + j * kStageBytes;
                    uint32_t a[4], c[4];
                    e2m1x8_f16(lds32(at), a);
                    e2m1x8_f16(lds32(at + 512u), c);
                    const float s0 = b == 0 ? sa[j][0] : (b == 1 ? sa[j][1] : (b == 2 ? sa[j][2] : sa[j][3]));
                    const float s1 = b == 0 ? sb[j][0] : (b == 1 ? sb[j][1] : (b == 2 ? sb[j][2] : sb[j][3]));
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        const uint4 v = x(b, n);
                        float d[4];
                        mma_f16_first(d, a[0], c[0], a[1], c[1], v.x, v.y);
                        mma_f16(d, a[2], c[2], a[3], c[3], v.z, v.w);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float u = unit(n * 8 + 2 * t + (i & 1)), s = i < 2 ? s0 : s1;
                            // a large and a small one are exact together; two of a side might leave fp32
                            const bool same = (u >= 1.0f) == (s >= 1.0f);
                            acc[j][n][i] = __fmaf_rn(same ? d[i] * u : d[i], same ? s : s * u, acc[j][n][i]);
                        }
                    }
                }
            }
        }
    }
    template <int NT, int N>
    static __device__ __forceinline__ void consume_shared(const Mat& w, uint32_t slot, int lane, uint32_t key, int step,
                                                          float (&acc)[NT][4], uint32_t x, uint32_t piece_stride,
                                                          const uint32_t (&xo)[NT], bool& plain, const uint32_t* field, int cols) {
        const uint32_t keys[1] = {key};
        consume_tiles<1, NT, N>(
            w, slot, lane, keys, step, reinterpret_cast<float(&)[1][NT][4]>(acc), plain,
            [&](int b, int n) { return lds128(x + static_cast<uint32_t>(b) * piece_stride + xo[n]); }, FieldUnit{field, cols});
    }

    template <int NT, class Unit>
    static __device__ __forceinline__ void to_numbers(float (&acc)[NT][4], int t, Unit unit) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] *= unit(n * 8 + 2 * t + (i & 1));
    }

    static __device__ __forceinline__ uint32_t lds32(uint32_t addr) {
        uint32_t v;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
        return v;
    }
    static __device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t (&d)[4]) {
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
            "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
            "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
            : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
            : "r"(w));
    }
    // four E8M0 bytes -> fp32 (exact; 255 becomes NaN)
    static __device__ __forceinline__ void e8m0x4(uint32_t e, float (&s)[4]) {
        uint32_t lo, hi;
        asm("{\n\t.reg .b16 h0, h1;\n\t"
            "mov.b32 {h0, h1}, %2;\n\t"
            "cvt.rn.bf16x2.ue8m0x2 %0, h0;\n\t"
            "cvt.rn.bf16x2.ue8m0x2 %1, h1;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(e));
        s[0] = __uint_as_float(lo << 16);
        s[1] = __uint_as_float(lo & 0xFFFF0000u);
        s[2] = __uint_as_float(hi << 16);
        s[3] = __uint_as_float(hi & 0xFFFF0000u);
    }
    static __device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                         uint32_t b0, uint32_t b1) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %10, %10, %10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
    }
    static __device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                                   uint32_t b1) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    }
};

// Barrier of the warps that share a tile.
__device__ __forceinline__ void group_sync(int group, int k_warps) {
    if (k_warps == 1) __syncwarp();
    else named_bar_sync(1u + static_cast<uint32_t>(group), static_cast<uint32_t>(k_warps) * 32u);
}

// ---- the phase with shared activations -----------------------------------------------------
// One column group ("segment") of activations in shared memory.
struct XBuffer {
    uint32_t addr;        // pieces
    int bytes;            // room for them
    uint32_t* field;      // kScaled: per column, the largest exponent field so far
    uint32_t* old_field;  // the same before the chunk that was staged last
};

__device__ __forceinline__ uint32_t max_field(const uint4& v) {
    uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
    return max(m & 0xFFFFu, m >> 16) >> 7;
}
__device__ __forceinline__ uint32_t scaled_half2(uint32_t bf16x2, float f) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;"
        : "=r"(d)
        : "f"(__uint_as_float(bf16x2 & 0xFFFF0000u) * f), "f"(__uint_as_float(bf16x2 << 16) * f));
    return d;
}

// Stage the activations of `cols` columns for steps [s0, s0 + n): piece (step,
// i, column, t) of 16 bytes at ((step kPieces + i) cols + column) 64 + 16 t.
// row(c): column c's activations (K of them; zeros behind).  All threads of the
// block; the caller synchronises before (the buffer is free) and after.  A warp
// takes 32 consecutive pieces of a column at a time, four such lots in flight;
// the blocks begin at different lots, since a line that all of them want at once
// is served to one after another.
template <class F, class Row>
__device__ __forceinline__ void stage_columns(const XBuffer& xb, int cols, int s0, int n, int K, Row row) {
    constexpr int kPer = 4 * F::kPieces;  // pieces of a column and step
    constexpr int kLots = 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per_col = n * kPer, lots = (per_col + 31) >> 5, all = cols * lots;
    const int first = static_cast<int>(static_cast<int64_t>(all) * blockIdx.x / gridDim.x);
    const int k0 = s0 * F::kStepCols;
    const uint32_t stride = static_cast<uint32_t>(cols) * 64u;
    if (F::kScaled) {
        for (int c = threadIdx.x; c < cols; c += kStreamThreads) {
            const uint32_t f = s0 == 0 ? 0u : xb.field[c];
            xb.old_field[c] = f;
            xb.field[c] = f;
        }
        __syncthreads();
    }
    auto place = [&](int c, int q) {
        const int step = q / kPer, r = q % kPer;
        return xb.addr + static_cast<uint32_t>(step * F::kPieces + F::piece_index(r)) * stride + static_cast<uint32_t>(c) * 64u +
               F::piece_lane(r) * 16u;
    };
    for (int u0 = warp; u0 < all; u0 += kStreamWarps * kLots) {
        uint4 v[kLots];
        uint32_t at[kLots];
        int col[kLots];
#pragma unroll
        for (int j = 0; j < kLots; ++j) {
            int u = u0 + j * kStreamWarps;
            v[j] = make_uint4(0u, 0u, 0u, 0u);
            col[j] = -1;
            if (u < all) {
                u += first;
                if (u >= all) u -= all;
                const int c = u / lots, q = (u - c * lots) * 32 + lane;
                if (q < per_col) {
                    col[j] = c;
                    at[j] = place(c, q);
                    if (k0 + 8 * q < K) v[j] = ldg128(row(c) + k0 + 8 * q);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kLots; ++j) {
            if (col[j] >= 0)
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at[j]), "r"(v[j].x), "r"(v[j].y), "r"(v[j].z), "r"(v[j].w)
                             : "memory");
            if (F::kScaled) {
                const uint32_t f = __reduce_max_sync(0xFFFFFFFFu, max_field(v[j]));
                if (lane == 0 && f > 0) atomicMax(xb.field + col[j], f);  // f > 0: the lot has pieces, lane 0 one of them
            }
        }
    }
    if (F::kScaled) {
        __syncthreads();
        for (int u1 = warp; u1 < all; u1 += kStreamWarps) {  // the pieces this thread wrote
            const int u = u1 + first < all ? u1 + first : u1 + first - all;
            const int c = u / lots, q = (u - c * lots) * 32 + lane;
            if (q >= per_col) continue;
            const uint32_t at = place(c, q);
            const float f = x_inverse(xb.field[c]);
            const uint4 v = lds128(at);
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(scaled_half2(v.x, f)), "r"(scaled_half2(v.y, f)),
                         "r"(scaled_half2(v.z, f)), "r"(scaled_half2(v.w, f))
                         : "memory");
        }
    }
}

constexpr uint32_t kSharedArea = 2176;  // a warp's partial sums awaiting a join: up to 4 tiles of 16 x 8

// Tiles in segments; the tiles of a segment multiply the same columns.  Job:
//   mat, K, segs; begin(s), end(s): tiles of segment s; cols(s); x_row(s, c);
//   start(feed, tile, lane, step), key(tile, lane): where the lane's rows are;
//   store(s, tile, n, lane, v): sums of column tile n in fragment order.
// All warps of the block call this together.
template <class F, int NT, class Job>
__device__ __forceinline__ void shared_phase(const Job& job, uint32_t ring, uint8_t* areas, const XBuffer& xb) {
    constexpr int kDepth = Ring<NT>::kDepth;
    constexpr uint32_t kRingBytes = Ring<NT>::kBytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int S = (job.K + F::kStepCols - 1) / F::kStepCols;
    auto chunk_steps = [&](int s) { return min(S, xb.bytes / (64 * F::kPieces * job.cols(s))); };

    // How many warps share a tile's K (lane i weighs 2^i): the choice that ends
    // first, counting steps, about two more for joining partial sums and four
    // for a refill of the activations.
    int lw;
    {
        const int i = min(lane, 4), k = 1 << i;
        int cost = 0;
        for (int s = 0; s < job.segs; ++s) {
            const int tiles = job.end(s) - job.begin(s), rounds = (tiles + (kStreamWarps >> i) - 1) >> (4 - i);
            const int cs = chunk_steps(s), chunks = cs == S ? 1 : (S + cs - 1) / cs;
            cost += rounds * (chunks * ((cs + k - 1) >> i) + (i > 0 ? 2 : 0) + (chunks > 1 ? 4 * chunks : 0));
        }
        lw = static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, static_cast<uint32_t>(min(cost, 0x0FFFFFFF)) << 3 | static_cast<uint32_t>(i)) & 7u);
    }
    const int wk = 1 << lw, groups = kStreamWarps >> lw, group = warp >> lw, kw = warp & (wk - 1);

    // producer: segment and tile, in the same order as the consumer below
    int ps = 0, ptile = job.segs ? job.begin(0) + group : 0;
    const int own = kw < S ? (S - kw + wk - 1) >> lw : 0;  // this warp's steps of a tile
    int pleft = 0;
    uint32_t pslot = ring, cslot = ring;
    typename F::Feed feed;
    auto seek = [&]() {  // the next tile of this group at or behind ptile, and its feed
        while (ps < job.segs && ptile >= job.end(ps))
            if (++ps < job.segs) ptile = job.begin(ps) + group;
        pleft = 0;
        if (ps < job.segs) {
            job.start(feed, ptile, lane, kw);
            pleft = own;
        }
    };
    if (own > 0) seek();
    auto issue = [&]() {
        if (pleft > 0) {
            F::issue(job.mat, feed, pslot, lane, wk);
            if (--pleft == 0) {
                ptile += groups;
                seek();
            }
        }
        cp_async_commit();
        pslot = pslot == ring + kRingBytes - kStageBytes ? ring : pslot + kStageBytes;
    };
#pragma unroll 1
    for (int i = 0; i < kDepth - 1; ++i) issue();

    constexpr int kBatch = NT == 1 ? 4 : (NT == 2 ? 2 : 1);  // tiles between two joins
    constexpr int kJoin = NT < 4 ? NT : 4;                   // column tiles of a join
    constexpr int kAreaVecs = kSharedArea / 16;
    static_assert(kBatch * kJoin * 512 <= kSharedArea, "area");
    float4* area = reinterpret_cast<float4*>(areas + warp * kSharedArea);
    const float4* group_area = reinterpret_cast<const float4*>(areas + group * wk * kSharedArea);
    for (int s = 0; s < job.segs; ++s) {
        const int t0 = job.begin(s), t1 = job.end(s), cols = job.cols(s), nt = (cols + 7) / 8;
        const int cs = chunk_steps(s), chunks = (S + cs - 1) / cs;
        const int rounds = (t1 - t0 + groups - 1) / groups;
        const uint32_t piece_stride = static_cast<uint32_t>(cols) * 64u;
        uint32_t xo[NT];  // this lane's piece of column tile n (of some column where the tile has none for it)
#pragma unroll
        for (int n = 0; n < NT; ++n) xo[n] = static_cast<uint32_t>(min(n * 8 + g, cols - 1)) * 64u + static_cast<uint32_t>(t) * 16u;
        auto stage = [&](int c) {
            __syncthreads();  // what was there has been read
            stage_columns<F>(xb, cols, c * cs, min(cs, S - c * cs), job.K, [&](int col) { return job.x_row(s, col); });
            __syncthreads();
        };
        if (chunks == 1) stage(0);
        int pending = 0;  // tiles of this group whose sums wait for a join
        for (int r = 0; r < rounds; ++r) {
            const int tile = t0 + r * groups + group;
            const bool live = tile < t1;
            float acc[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
            const uint32_t key = live ? job.key(tile, lane) : 0u;
            bool plain = true;  // kScaled: sums are in the columns' units
            int step = kw;
            for (int c = 0; c < chunks; ++c) {
                if (chunks > 1) {
                    stage(c);
                    if (F::kScaled && c > 0 && plain) {  // the sums so far, in the columns' new units
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int col = min(n * 8 + 2 * t + i, cols - 1);
                                const int d = static_cast<int>(x_field(xb.old_field[col])) - static_cast<int>(x_field(xb.field[col]));
                                const float f = d < -126 ? 0.f : __uint_as_float(static_cast<uint32_t>(127 + d) << 23);
                                acc[n][i] *= f;
                                acc[n][2 + i] *= f;
                            }
                    }
                }
                if (!live) continue;
                const int end = min((c + 1) * cs, S);
                uint32_t x = xb.addr + static_cast<uint32_t>((step - c * cs) * F::kPieces) * piece_stride;
                const uint32_t x_step = static_cast<uint32_t>(F::kPieces << lw) * piece_stride;
                // N column tiles, a power of two: unused ones repeat the last column
                auto run = [&](auto count) {
                    constexpr int N = decltype(count)::value < NT ? decltype(count)::value : NT;
#pragma unroll 1
                    for (; step < end; step += wk) {
                        cp_async_wait<kDepth - 2>();
                        __syncwarp();  // the copies of all lanes have landed; the slot refilled below is read out
                        issue();
                        F::template consume_shared<NT, N>(job.mat, cslot, lane, key, step, acc, x, piece_stride, xo, plain, xb.field,
                                                          cols);
                        x += x_step;
                        cslot = cslot == ring + kRingBytes - kStageBytes ? ring : cslot + kStageBytes;
                    }
                };
                if (NT == 1 || nt == 1) run(std::integral_constant<int, 1>{});
                else if (NT == 2 || nt == 2) run(std::integral_constant<int, 2>{});
                else if (NT == 4 || nt <= 4) run(std::integral_constant<int, 4>{});
                else run(std::integral_constant<int, 8>{});
            }
            if constexpr (F::kScaled) {
                if (plain) F::template to_numbers<NT>(acc, t, FieldUnit{xb.field, cols});
            }
            if (wk == 1) {
                if (live) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        if (n < nt) job.store(s, tile, n, lane, make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]));
                }
                continue;
            }
#pragma unroll
            for (int n0 = 0; n0 < NT; n0 += kJoin) {
                if (n0 >= nt) break;
                if (live) {
#pragma unroll
                    for (int n = 0; n < kJoin; ++n)
                        area[(pending * kJoin + n) * 32 + lane] =
                            make_float4(acc[n0 + n][0], acc[n0 + n][1], acc[n0 + n][2], acc[n0 + n][3]);
                    ++pending;
                }
                // a group's tiles end together: the same number is pending in all its warps
                const bool last = r + 1 == rounds || tile + groups >= t1;
                if (pending == 0 || (pending < kBatch && !last)) continue;
                group_sync(group, wk);
                const int first = tile - (pending - 1) * groups;
                for (int i = kw * 32 + lane; i < pending * kJoin * 32; i += wk * 32) {
                    const int b = i / (kJoin * 32), n = n0 + (i >> 5) % kJoin;
                    if (n >= nt) continue;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int w = 0; w < wk; ++w) {
                        const float4 q = group_area[w * kAreaVecs + i];
                        v.x += q.x;
                        v.y += q.y;
                        v.z += q.z;
                        v.w += q.w;
                    }
                    job.store(s, first + b * groups, n, i & 31, v);
                }
                group_sync(group, wk);
                pending = 0;
            }
        }
    }
    cp_async_wait<0>();
}

}  // namespace mlxq
