// Y = X W^T with an MX4 weight and BF16 activations, up to 64 rows of X.
//
// HBM-bound on the weight (17/32 bytes per element): one block per SM streams
// a balanced range of rows of W, every byte once (row_stream.cuh), and keeps the
// rows of X in shared memory (in chunks of K where they do not fit).  One
// rounding, of the result.
#include "row_stream.cuh"

namespace mlxq {
namespace {

struct GemmParams {
    Mx4HalfFmt::Mat w;
    const uint16_t* x;
    uint16_t* y;
    int N, K, m;
};

// Rows [lo, hi) of W in tiles of 16, one segment whose columns are the rows of X.
struct GemmJob {
    const GemmParams& p;
    const Mx4HalfFmt::Mat& mat;
    int K, lo, hi, segs;

    __device__ __forceinline__ explicit GemmJob(const GemmParams& p_) : p(p_), mat(p_.w) {
        K = p.K;
        lo = static_cast<int>(static_cast<int64_t>(p.N) * blockIdx.x / gridDim.x);
        hi = static_cast<int>(static_cast<int64_t>(p.N) * (blockIdx.x + 1) / gridDim.x);
        segs = lo < hi ? 1 : 0;
    }
    __device__ __forceinline__ int begin(int) const { return 0; }
    __device__ __forceinline__ int end(int) const { return (hi - lo + 15) / 16; }
    __device__ __forceinline__ int cols(int) const { return p.m; }
    __device__ __forceinline__ const uint16_t* x_row(int, int c) const { return p.x + static_cast<int64_t>(c) * p.K; }
    __device__ __forceinline__ void start(Mx4HalfFmt::Feed& f, int tile, int lane, int step) const {
        const int r = lo + tile * 16 + (lane >> 2);
        Mx4HalfFmt::start(f, p.w, p.w, r, r + 8, r < hi, r + 8 < hi, lane, step);
    }
    __device__ __forceinline__ uint32_t key(int tile, int lane) const {
        return Mx4HalfFmt::row_key(p.w, static_cast<uint32_t>(lo + tile * 16 + (lane >> 2)));
    }
    __device__ __forceinline__ void store(int, int tile, int n, int lane, const float4& v) const {
        const int r = lo + tile * 16 + (lane >> 2), c = n * 8 + 2 * (lane & 3);
        const float s[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (c + i >= p.m) continue;
            uint16_t* y = p.y + static_cast<int64_t>(c + i) * p.N + r;
            const uint32_t b = pack_bf16x2(s[i], s[2 + i]);
            if (r < hi) y[0] = static_cast<uint16_t>(b);
            if (r + 8 < hi) y[8] = static_cast<uint16_t>(b >> 16);
        }
    }
};

constexpr uint32_t kAreas = kStreamWarps * kRingBytes;
constexpr uint32_t kFields = kAreas + kStreamWarps * kSharedArea;
constexpr uint32_t kX = kFields + 2 * kMx4GemmMaxM * 4;
constexpr uint32_t kTotal = 227 * 1024;

template <int NT>
__global__ void __launch_bounds__(kStreamThreads, 1) k_mx4_gemm(const __grid_constant__ GemmParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    pdl_launch_dependents();
    uint32_t* field = reinterpret_cast<uint32_t*>(smem + kFields);
    const uint32_t ring = smem_u32(smem) + (threadIdx.x >> 5) * kRingBytes;
    const XBuffer xb{smem_u32(smem) + kX, static_cast<int>(kTotal - kX), field, field + kMx4GemmMaxM};
    pdl_wait();
    shared_phase<Mx4HalfFmt, NT>(GemmJob(p), ring, smem + kAreas, xb);
}

template <int NT>
cudaError_t launch_nt(const GemmParams& p, cudaStream_t stream) {
    static std::atomic<int> configured[64];
    cudaError_t e = ensure_dynamic_smem(k_mx4_gemm<NT>, kTotal, configured);
    if (e != cudaSuccess) return e;
    const int sms = device_info().sm_count, octets = (p.N + 7) / 8;
    return launch_pdl(k_mx4_gemm<NT>, dim3(static_cast<unsigned>(octets < sms ? octets : sms)), dim3(kStreamThreads), kTotal, stream, p);
}

}  // namespace

cudaError_t launch_mx4_gemm(const Mx4View& w, const void* x, void* y, int64_t m, cudaStream_t stream) {
    if (w.cols == 0) return cudaMemsetAsync(y, 0, static_cast<size_t>(m * w.rows * 2), stream);  // empty sums
    const GemmParams p{Mx4HalfFmt::make(w), static_cast<const uint16_t*>(x), static_cast<uint16_t*>(y), static_cast<int>(w.rows),
                       static_cast<int>(w.cols), static_cast<int>(m)};
    if (m <= 8) return launch_nt<1>(p, stream);
    if (m <= 16) return launch_nt<2>(p, stream);
    if (m <= 32) return launch_nt<4>(p, stream);
    return launch_nt<8>(p, stream);
}

}  // namespace mlxq
