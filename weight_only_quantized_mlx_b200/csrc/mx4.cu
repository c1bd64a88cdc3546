// BF16 -> MX4 and back (the format: mx4_common.cuh).
//
// Quantisation, per block of 32 columns, with m = max |x|:
//   e = clamp(floor(log2 m) - 2, -127, 127)   (2 = exponent of the largest E2M1 binade)
//   scale byte = e + 127;  code = E2M1 value nearest to x 2^-e, ties to the
//   even code, magnitudes above 6 to 6.
// floor(log2 m) is the exponent field of the largest magnitude, and x 2^-e is
// exact in fp32, so the codes are those of exact arithmetic.  A block of zeros
// gets byte 0; a block that holds an infinity or NaN gets byte 255 and codes 0.
//
// Both directions are one pass and HBM-bound: 2 + 17/32 bytes per element (14336 x
// 4096: 24.4 us each way, the copy rate gives 22.7).
// Quantisation: two lanes share a block, each loads 16 BF16 (32 bytes) and
// writes 8 bytes of codes; the maximum crosses one shuffle.  Dequantisation:
// a thread turns 8 bytes of codes into 32 bytes of BF16.
#include "device_common.cuh"
#include "kernels.h"
#include "mx4_common.cuh"

namespace mlxq {
namespace {

constexpr int kMxThreads = 256;

__device__ __forceinline__ void ldg_nc_v8(const void* p, uint32_t (&v)[8]) {
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "l"(p));
}

// Eight fp32 values -> one word of E2M1 codes, the first in the low nibble.
__device__ __forceinline__ uint32_t e2m1x8(const float (&f)[8]) {
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(w)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
    return w;
}

// VEC: x is 32-byte aligned (rows are multiples of 64 bytes, so every half
// block then is); otherwise 2-byte loads.
template <bool VEC>
__global__ void __launch_bounds__(kMxThreads) k_mx4_quantize(const uint16_t* __restrict__ x, int64_t halves,
                                                             uint2* __restrict__ codes, uint8_t* __restrict__ scales) {
    pdl_launch_dependents();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kMxThreads + threadIdx.x;  // half block of 16 columns
    pdl_wait();
    const bool live = i < halves;  // both halves of a block are live or not
    uint32_t v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (live) {
        if (VEC) {
            ldg_nc_v8(x + i * 16, v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t lo = __ldg(x + i * 16 + 2 * j), hi = __ldg(x + i * 16 + 2 * j + 1);
                v[j] = lo | hi << 16;
            }
        }
    }
    uint32_t mx = 0;  // per 16-bit half: the largest magnitude's bits
#pragma unroll
    for (int j = 0; j < 8; ++j) mx = __vmaxu2(mx, v[j] & 0x7FFF7FFFu);
    mx = __vmaxu2(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
    const uint32_t top = max(mx & 0xFFFFu, mx >> 16) >> 7;  // exponent field of the maximum
    const uint32_t byte = top == 255u ? 255u : (top > 2u ? top - 2u : 0u);
    // 2^-e, e = byte - 127: exponent field 254 - byte (1 .. 254)
    const float inv = __uint_as_float((254u - min(byte, 253u)) << 23);
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = __uint_as_float(v[4 * h + j] << 16) * inv;
            f[2 * j + 1] = __uint_as_float(v[4 * h + j] & 0xFFFF0000u) * inv;
        }
        w[h] = byte == 255u ? 0u : e2m1x8(f);
    }
    if (!live) return;
    codes[i] = make_uint2(w[0], w[1]);
    if ((i & 1) == 0) scales[i >> 1] = static_cast<uint8_t>(byte);
}

// A thread writes 16 columns.  VEC: out is 32-byte aligned; otherwise 2-byte stores.
template <bool VEC>
__global__ void __launch_bounds__(kMxThreads) k_mx4_dequant(const uint2* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales, int64_t halves,
                                                            uint16_t* __restrict__ out) {
    pdl_launch_dependents();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kMxThreads + threadIdx.x;
    pdl_wait();
    if (i >= halves) return;
    const uint2 c = __ldg(codes + i);
    const uint32_t sc = e8m0_to_bf16(__ldg(scales + (i >> 1))) * 0x00010001u;
    const uint32_t w[2] = {c.x, c.y};
    uint32_t o[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        // pairs (0, 4), (1, 5), (2, 6), (3, 7); exact products, then columns in order
        const uint32_t p0 = mul_bf16x2(mul_bf16x2(e2m1_pair<0>(w[h]), kTwo126), sc);
        const uint32_t p1 = mul_bf16x2(mul_bf16x2(e2m1_pair<1>(w[h]), kTwo126), sc);
        const uint32_t p2 = mul_bf16x2(mul_bf16x2(e2m1_pair<2>(w[h]), kTwo126), sc);
        const uint32_t p3 = mul_bf16x2(mul_bf16x2(e2m1_pair<3>(w[h]), kTwo126), sc);
        o[4 * h + 0] = __byte_perm(p0, p1, 0x5410);
        o[4 * h + 1] = __byte_perm(p2, p3, 0x5410);
        o[4 * h + 2] = __byte_perm(p0, p1, 0x7632);
        o[4 * h + 3] = __byte_perm(p2, p3, 0x7632);
    }
    if (VEC) {
        stg_cs_v8(out + i * 16, o);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            out[i * 16 + 2 * j] = static_cast<uint16_t>(o[j]);
            out[i * 16 + 2 * j + 1] = static_cast<uint16_t>(o[j] >> 16);
        }
    }
}

cudaError_t blocks_for(int64_t halves, unsigned* blocks) {
    const int64_t b = (halves + kMxThreads - 1) / kMxThreads;
    if (b > 0x7FFFFFFF) return cudaErrorInvalidValue;
    *blocks = static_cast<unsigned>(b);
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_mx4_quantize(const void* x, const Mx4View& dst, cudaStream_t stream) {
    const int64_t halves = dst.rows * dst.cols / 16;
    if (halves == 0) return cudaSuccess;
    unsigned blocks = 0;
    cudaError_t e = blocks_for(halves, &blocks);
    if (e != cudaSuccess) return e;
    auto* codes = reinterpret_cast<uint2*>(const_cast<uint8_t*>(dst.codes));
    auto kern = (reinterpret_cast<uintptr_t>(x) & 31u) == 0 ? k_mx4_quantize<true> : k_mx4_quantize<false>;
    return launch_pdl(kern, dim3(blocks), dim3(kMxThreads), 0, stream, static_cast<const uint16_t*>(x), halves, codes,
                      const_cast<uint8_t*>(dst.scales));
}

cudaError_t launch_mx4_dequant(const Mx4View& w, void* out, cudaStream_t stream) {
    const int64_t halves = w.rows * w.cols / 16;
    if (halves == 0) return cudaSuccess;
    unsigned blocks = 0;
    cudaError_t e = blocks_for(halves, &blocks);
    if (e != cudaSuccess) return e;
    auto kern = (reinterpret_cast<uintptr_t>(out) & 31u) == 0 ? k_mx4_dequant<true> : k_mx4_dequant<false>;
    return launch_pdl(kern, dim3(blocks), dim3(kMxThreads), 0, stream, reinterpret_cast<const uint2*>(w.codes), w.scales,
                      halves, static_cast<uint16_t*>(out));
}

}  // namespace mlxq
