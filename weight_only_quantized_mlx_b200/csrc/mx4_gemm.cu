// Y = X W^T with an MX4 weight and BF16 activations, up to 64 rows of X.
//
// HBM-bound on the weight (17/32 bytes per element): one block per SM streams
// a balanced range of rows of W (stream_tile.cuh), every byte once, and W's
// BF16 values, which are exact, meet all rows of X in tensor-pipe fragments
// with fp32 sums.  One rounding, of the result.
#include "stream_tile.cuh"

namespace mlxq {
namespace {

struct GemmParams {
    Mx4Fmt::Mat w;
    const uint16_t* x;
    uint16_t* y;
    int N, K, m;
};

template <int NT>
__global__ void __launch_bounds__(kStreamThreads, 1) k_mx4_gemm(const __grid_constant__ GemmParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    pdl_launch_dependents();
    const int64_t N = p.N;
    const int lo = static_cast<int>(N * blockIdx.x / gridDim.x), hi = static_cast<int>(N * (blockIdx.x + 1) / gridDim.x);
    pdl_wait();
    const uint32_t ring = smem_u32(smem) + (threadIdx.x >> 5) * kRingBytes;
    stream_rows<Mx4Fmt, NT, false>(p.w, 0, lo, hi, 1, nullptr, Columns{}, p.x, p.K, p.m, p.y, N, ring,
                                   smem + kStreamWarps * kRingBytes, [] { return true; });
}

template <int NT>
cudaError_t launch_nt(const GemmParams& p, cudaStream_t stream) {
    static std::atomic<int> configured[64];
    const size_t smem = kStreamWarps * (kRingBytes + kAreaBytes);
    cudaError_t e = ensure_dynamic_smem(k_mx4_gemm<NT>, smem, configured);
    if (e != cudaSuccess) return e;
    const int sms = device_info().sm_count, tiles = (p.N + 7) / 8;
    return launch_pdl(k_mx4_gemm<NT>, dim3(static_cast<unsigned>(tiles < sms ? tiles : sms)), dim3(kStreamThreads), smem, stream, p);
}

}  // namespace

cudaError_t launch_mx4_gemm(const Mx4View& w, const void* x, void* y, int64_t m, cudaStream_t stream) {
    if (w.cols == 0) return cudaMemsetAsync(y, 0, static_cast<size_t>(m * w.rows * 2), stream);  // empty sums
    const GemmParams p{Mx4Fmt::make(w), static_cast<const uint16_t*>(x), static_cast<uint16_t*>(y), static_cast<int>(w.rows),
                       static_cast<int>(w.cols), static_cast<int>(m)};
    if (m <= 8) return launch_nt<1>(p, stream);
    if (m <= 16) return launch_nt<2>(p, stream);
    if (m <= 32) return launch_nt<4>(p, stream);
    return launch_nt<8>(p, stream);
}

}  // namespace mlxq
