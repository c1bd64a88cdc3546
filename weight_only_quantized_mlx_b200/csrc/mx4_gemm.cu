// Y = X W^T with an MX4 weight and BF16 activations, up to 64 rows of X.
//
// Blocks stream balanced ranges of the weight's rows (17/32 bytes per element), every
// byte once (row_stream.cuh).  One rounding, of the result.
//
// k_mx4_gemm, up to 8 rows of X: a block keeps them in shared memory, converted on
// the way (in chunks of K where they do not fit).  28672 x 8192, one row: 39 us, 3.2
// TB/s of the weight, half of the measured copy rate.  No unit is full (issue slots 64
// %, ALU 51 %, tensor pipe 20 %, DRAM 36 %): three warps a scheduler wait for their own
// instructions' results.  4096 x 4096: 7.3 us, mostly the latencies of one launch,
// of the first loads and of the join.
//
// k_mx4_gemm_async, more rows: every block needs all of X over its columns, and
// fetching and converting them between products took most of the time (4096 x
// 4096, m = 64: 80 us).  So k_mx4_prepare writes X once in the order and units in
// which the products take it, step after step, and bulk copies bring the steps into
// a ring while the warps multiply.  Where rows are few, four blocks of a cluster share
// a range of rows and split K, which divides the copies of X, and add their sums
// through distributed shared memory in rank order.  28672 x 8192: 16 rows 65 us, 32
// rows 92, 64 rows 171; 4096 x 4096: 14, 16, 19.  The products take the time (without
// them 33 us whatever the rows at 28672 x 8192; without the copies of the weight 64,
// 93 and 145), and again no unit is full (64 rows: issue slots 42 %, tensor pipe 38 %,
// DRAM 9 %; two warps a scheduler, which wait for their own results).  The 8-bit gemm of
// this library takes 76, 101 and 120 us there: from 40 rows on it is the faster one.
#include <cooperative_groups.h>

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

constexpr uint32_t kAreas = kStreamWarps * Ring<1>::kBytes;
constexpr uint32_t kFields = kAreas + kStreamWarps * kSharedArea;
constexpr uint32_t kX = kFields + 2 * kMx4GemmMaxM * 4;
constexpr uint32_t kTotal = 227 * 1024;

__global__ void __launch_bounds__(kStreamThreads, 1) k_mx4_gemm(const __grid_constant__ GemmParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    pdl_launch_dependents();
    uint32_t* field = reinterpret_cast<uint32_t*>(smem + kFields);
    const uint32_t ring = smem_u32(smem) + (threadIdx.x >> 5) * Ring<1>::kBytes;
    const XBuffer xb{smem_u32(smem) + kX, static_cast<int>(kTotal - kX), field, field + kMx4GemmMaxM};
    pdl_wait();
    shared_phase<Mx4HalfFmt, 1>(GemmJob(p), ring, smem + kAreas, xb);
}

cudaError_t launch_direct(const GemmParams& p, cudaStream_t stream) {
    static std::atomic<int> configured[64];
    cudaError_t e = ensure_dynamic_smem(k_mx4_gemm, kTotal, configured);
    if (e != cudaSuccess) return e;
    const int sms = device_info().sm_count, octets = (p.N + 7) / 8;
    return launch_pdl(k_mx4_gemm, dim3(static_cast<unsigned>(octets < sms ? octets : sms)), dim3(kStreamThreads), kTotal, stream, p);
}

// ---- more rows ------------------------------------------------------------------------------
struct AsyncParams {
    Mx4HalfFmt::Mat w;
    const uint8_t* xp;      // pieces of X: ((step 4 + block) m + row) 64 + 16 t
    const uint32_t* field;  // [m]
    uint16_t* y;
    int N, K, m, S;
    unsigned int* status;
};

constexpr uint32_t kPartialBytes = 32 * 1024;  // S > 1: fp32 sums of a cluster's rows
constexpr int kMaxXStages = 16;
constexpr int kSplit = 4;  // blocks of a cluster that split K, where they do
constexpr uint32_t kAsyncTotal = 227 * 1024 - 512;

// Shared memory: weight rings | areas | units | sums (S > 1) | steps of X.
template <int NT>
struct AsyncSmem {
    // A warp's tile is MT times 16 rows.  With four column tiles, two: a piece of X is
    // read from shared memory once for both, and eight warps have the registers for
    // their sums (28672 x 8192, 32 rows: 99 -> 91 us; at 16 rows 67 -> 66, but 4096 x
    // 4096 13 -> 14).
    static constexpr int MT = NT <= 2 ? 1 : 2;
    static constexpr int kLogWarps = NT <= 2 ? 4 : 3;
    static constexpr int kWarps = 1 << kLogWarps, kThreads = 32 * kWarps;
    static constexpr int kDepth = 4;
    static constexpr uint32_t kStage = MT * kStageBytes;
    static constexpr uint32_t kRing = kDepth * kStage;
    static constexpr uint32_t kAreas = kWarps * kRing;
    static constexpr uint32_t kFields = kAreas + kWarps * kSharedArea;
    static constexpr uint32_t kX = kFields + kMx4GemmMaxM * 4;
    static_assert(kAsyncTotal - kX - kPartialBytes >= 2u * (NT < 4 ? NT * 8 : kMx4GemmMaxM) * 256, "two steps of X");
};

// Steps of X that fit behind the rest.
template <int NT>
__host__ __device__ int x_room(int S, int m) {
    const int n = static_cast<int>((kAsyncTotal - AsyncSmem<NT>::kX - (S > 1 ? kPartialBytes : 0u)) / (static_cast<uint32_t>(m) * 256u));
    return n < kMaxXStages ? n : kMaxXStages;
}

// The steps that a warp takes where 2^i warps share a unit, `join` counted for each join.
template <int NT>
__host__ __device__ __forceinline__ int warp_steps(int units, int steps, int i, int join) {
    const int groups = AsyncSmem<NT>::kWarps >> i;
    return (units + groups - 1) / groups * (((steps + (1 << i) - 1) >> i) + (i > 0 ? join : 0));
}

// A block per row of X: its unit (the largest exponent), then its pieces.
constexpr int kPrepareThreads = 512;
__global__ void __launch_bounds__(kPrepareThreads) k_mx4_prepare(const uint16_t* __restrict__ x, int K, int m, int steps,
                                                                 uint8_t* __restrict__ xp, uint32_t* __restrict__ fields) {
    __shared__ uint32_t top;
    pdl_launch_dependents();
    if (threadIdx.x == 0) top = 0u;
    __syncthreads();
    pdl_wait();
    const int c = blockIdx.x, pieces = steps * 16;
    const uint4* src = reinterpret_cast<const uint4*>(x + static_cast<int64_t>(c) * K);
    uint32_t f = 0;
    for (int q = threadIdx.x; q < K / 8; q += kPrepareThreads) f = max(f, max_field(__ldg(src + q)));
    f = __reduce_max_sync(0xFFFFFFFFu, f);
    if ((threadIdx.x & 31) == 0) atomicMax(&top, f);
    __syncthreads();
    f = top;
    if (threadIdx.x == 0) fields[c] = f;
    const float inv = x_inverse(f);
    for (int q = threadIdx.x; q < pieces; q += kPrepareThreads) {
        const uint4 v = q < K / 8 ? __ldg(src + q) : make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(xp + (static_cast<int64_t>(q >> 2) * m + c) * 64 + (q & 3) * 16) =
            make_uint4(scaled_half2(v.x, inv), scaled_half2(v.y, inv), scaled_half2(v.z, inv), scaled_half2(v.w, inv));
    }
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr, uint32_t rank) {
    float v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
                 : "=f"(v)
                 : "r"(addr), "r"(rank));
    return v;
}

template <int NT>
__global__ void __launch_bounds__(AsyncSmem<NT>::kThreads, 1) k_mx4_gemm_async(const __grid_constant__ AsyncParams p) {
    using F = Mx4HalfFmt;
    using M = AsyncSmem<NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[2 * kMaxXStages];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    pdl_launch_dependents();
    const int S = p.S, rank = static_cast<int>(blockIdx.x) % S, cl = static_cast<int>(blockIdx.x) / S;
    const int clusters = static_cast<int>(gridDim.x) / S;
    const int lo = static_cast<int>(static_cast<int64_t>(p.N) * cl / clusters);
    const int hi = static_cast<int>(static_cast<int64_t>(p.N) * (cl + 1) / clusters);
    const int all_steps = (p.K + F::kStepCols - 1) / F::kStepCols;
    const int st0 = static_cast<int>(static_cast<int64_t>(all_steps) * rank / S);
    const int steps = static_cast<int>(static_cast<int64_t>(all_steps) * (rank + 1) / S) - st0;
    constexpr int MT = M::MT, kRows = 16 * MT;
    // a unit of work: a tile with one part of up to 8 NT rows of X
    const int parts = (p.m + 8 * NT - 1) / (8 * NT), units = (hi - lo + kRows - 1) / kRows * parts;
    const uint32_t step_bytes = static_cast<uint32_t>(p.m) * 256u;
    const uint32_t partial = smem_u32(smem) + M::kX, x0 = partial + (S > 1 ? kPartialBytes : 0u);
    const int room = x_room<NT>(S, p.m);
    uint32_t* field = reinterpret_cast<uint32_t*>(smem + M::kFields);

    // Warps per unit (lane i weighs 2^i of them): steps, and two for a join.  A
    // stage of X is one step; their number is a multiple of the warps of a unit,
    // so that a warp meets a stage only in its own steps (it could else test the
    // barrier's parity a phase early), and at least twice it.
    int lw;
    {
        const int i = min(lane, M::kLogWarps);
        int cost = warp_steps<NT>(units, steps, i, 2);
        if ((2 << i) > room && i > 0) cost = 0x0FFFFFFF;
        lw = static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, static_cast<uint32_t>(min(cost, 0x0FFFFFFF)) << 3 | static_cast<uint32_t>(i)) & 7u);
    }
    const int wk = 1 << lw, groups = M::kWarps >> lw, stages = room >> lw << lw;
    const int rounds = (units + groups - 1) / groups;
    auto full = [&](int s) { return smem_u32(&bars[s]); };
    auto empty = [&](int s) { return smem_u32(&bars[kMaxXStages + s]); };
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), static_cast<uint32_t>(groups));  // the warp of each group whose step it is
        }
        mbar_fence_init();
    }
    __syncthreads();
    pdl_wait();

    // (A round has a multiple of wk steps, the last ones perhaps without work, so
    // that a warp's steps fall on the same stages in every round.)
    const int padded = (steps + wk - 1) >> lw << lw, total = rounds * padded;
    const uint64_t pol = policy_evict_last();
    auto feed_x = [&](int s, int k) {  // step k of a round into stage s
        mbar_arrive_expect_tx(full(s), step_bytes);
        bulk_g2s(x0 + static_cast<uint32_t>(s) * step_bytes, p.xp + static_cast<int64_t>(st0 + min(k, steps - 1)) * step_bytes, step_bytes,
                 full(s), pol);
    };
    if (threadIdx.x == 0)
        for (int it = 0; it < min(stages, total); ++it) feed_x(it, it % padded);
    __syncwarp();
    {
        const int group = warp >> lw, kw = warp & (wk - 1);
        const uint32_t ring = smem_u32(smem) + warp * M::kRing;
        float4* area = reinterpret_cast<float4*>(smem + M::kAreas + warp * kSharedArea);
        const float4* group_area = reinterpret_cast<const float4*>(smem + M::kAreas + group * wk * kSharedArea);
        constexpr int kAreaVecs = kSharedArea / 16;
        static_assert(NT * 512 <= kSharedArea, "area");

        const int own = kw < steps ? (steps - kw + wk - 1) >> lw : 0;
        int punit = own > 0 ? group : units, pleft = 0;
        uint32_t pslot = ring, cslot = ring;
        F::Feed feed[MT];
        auto seek = [&]() {
            pleft = 0;
            if (punit < units) {
#pragma unroll
                for (int j = 0; j < MT; ++j) {
                    const int r = lo + punit / parts * kRows + 16 * j + g;
                    F::start(feed[j], p.w, p.w, r, r + 8, r < hi, r + 8 < hi, lane, st0 + kw);
                }
                pleft = own;
            }
        };
        seek();
        auto issue = [&]() {
            if (pleft > 0) {
#pragma unroll
                for (int j = 0; j < MT; ++j) F::issue(p.w, feed[j], pslot + j * kStageBytes, lane, wk);
                if (--pleft == 0) {
                    punit += groups;
                    seek();
                }
            }
            cp_async_commit();
            pslot = pslot == ring + M::kRing - M::kStage ? ring : pslot + M::kStage;
        };
#pragma unroll 1
        for (int i = 0; i < M::kDepth - 1; ++i) issue();
        for (int c = threadIdx.x; c < p.m; c += M::kThreads) field[c] = p.field[c];
        __syncthreads();  // the fields are there

        const uint32_t piece_stride = static_cast<uint32_t>(p.m) * 64u;
        auto store = [&](int r0, int c0, int l, const float4& v) {
            const int r = r0 + (l >> 2), c = c0 + 2 * (l & 3), rows = hi - lo;
            const float s[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = r + (i >> 1) * 8, col = c + (i & 1);
                if (col >= p.m || row >= rows) continue;
                if (S > 1)
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(partial + static_cast<uint32_t>(col * rows + row) * 4u), "f"(s[i]) : "memory");
                else
                    p.y[static_cast<int64_t>(col) * p.N + lo + row] = static_cast<uint16_t>(pack_bf16x2(s[i], 0.f));
            }
        };
        bool ok = true;
        int stage = kw;        // of this warp's present step; stages is a multiple of wk
        uint32_t parity = 0;   // of that stage's use
        const int ahead = (stages - wk) % padded;
        for (int r = 0; r < rounds; ++r) {
            const int unit = r * groups + group, tile = unit / parts, c0 = (unit - tile * parts) * 8 * NT;
            const bool live = unit < units;
            const int cols = p.m - c0, nt = (cols + 7) / 8;  // column tiles; the kernel's others repeat the last row of X
            uint32_t xo[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) xo[n] = static_cast<uint32_t>(min(c0 + n * 8 + g, p.m - 1)) * 64u + static_cast<uint32_t>(t) * 16u;
            float acc[MT][NT][4];
            uint32_t key[MT];
#pragma unroll
            for (int j = 0; j < MT; ++j) {
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[j][n][0] = acc[j][n][1] = acc[j][n][2] = acc[j][n][3] = 0.f;
                key[j] = F::row_key(p.w, static_cast<uint32_t>(lo + tile * kRows + 16 * j + g));
            }
            bool plain = true;  // sums are in the columns' units
#pragma unroll 1
            for (int k = kw; k < padded; k += wk) {
                const int it = r * padded + k;
                // The stage of this warp's last step gets its next contents as soon as
                // all groups have read it: one warp of each kw sees to it, the groups
                // taking turns.
                const int next = it + stages - wk;
                if (it >= wk && next < total && ((next >> lw) & (groups - 1)) == group) {
                    const int s = stage >= wk ? stage - wk : stage - wk + stages;
                    if (ok) ok = mbar_wait(empty(s), stage >= wk ? parity : parity ^ 1u, p.status);
                    if (lane == 0 && ok) feed_x(s, k + ahead < padded ? k + ahead : k + ahead - padded);
                    __syncwarp();
                }
                // after a wait has given up there are no more, the control flow goes on
                if (ok) ok = mbar_wait(full(stage), parity, p.status);
                if (live && k < steps) {
                    cp_async_wait<M::kDepth - 2>();
                    __syncwarp();  // the copies of all lanes have landed; the slot refilled below is read out
                    issue();
                    const uint32_t xs = x0 + static_cast<uint32_t>(stage) * step_bytes;
                    auto x = [&](int b, int n) { return lds128(xs + static_cast<uint32_t>(b) * piece_stride + xo[n]); };
                    if (NT == 4 && nt <= 2)
                        F::consume_tiles<MT, NT, (NT + 1) / 2>(p.w, cslot, lane, key, st0 + k, acc, plain, x, FieldUnit{field + c0, cols});
                    else
                        F::consume_tiles<MT, NT, NT>(p.w, cslot, lane, key, st0 + k, acc, plain, x, FieldUnit{field + c0, cols});
                    cslot = cslot == ring + M::kRing - M::kStage ? ring : cslot + M::kStage;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty(stage));
                stage += wk;
                if (stage >= stages) {
                    stage -= stages;
                    parity ^= 1u;
                }
            }
            if (!live) continue;
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                const int r0 = tile * kRows + 16 * j;
                if (plain) F::to_numbers<NT>(acc[j], t, FieldUnit{field + c0, cols});
                if (wk == 1) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        if (n < nt) store(r0, c0 + n * 8, lane, make_float4(acc[j][n][0], acc[j][n][1], acc[j][n][2], acc[j][n][3]));
                    continue;
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) area[n * 32 + lane] = make_float4(acc[j][n][0], acc[j][n][1], acc[j][n][2], acc[j][n][3]);
                group_sync(group, wk);
                for (int i = kw * 32 + lane; i < NT * 32; i += wk * 32) {
                    if (i >> 5 >= nt) continue;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int w = 0; w < wk; ++w) {
                        const float4 q = group_area[w * kAreaVecs + i];
                        v.x += q.x;
                        v.y += q.y;
                        v.z += q.z;
                        v.w += q.w;
                    }
                    store(r0, c0 + (i >> 5) * 8, i & 31, v);
                }
                group_sync(group, wk);
            }
        }
        cp_async_wait<0>();
    }
    if (threadIdx.x == 0)  // every issued copy has landed before the block may exit
        for (int it = total > stages ? total - stages : 0; it < total; ++it)
            if (!mbar_wait(full(it % stages), (it / stages) & 1, p.status)) break;
    __syncwarp();
    if (S > 1) {
        cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
        cluster.sync();  // all sums are there
        const int rows = hi - lo, n = rows * p.m;
        for (int i = rank * static_cast<int>(blockDim.x) + threadIdx.x; i < n; i += S * static_cast<int>(blockDim.x)) {
            float v[kSplit];  // all ranks' sums, in flight together
#pragma unroll
            for (int q = 0; q < kSplit; ++q) v[q] = ld_cluster_f32(partial + static_cast<uint32_t>(i) * 4u, static_cast<uint32_t>(q));
            float s = v[0];
#pragma unroll
            for (int q = 1; q < kSplit; ++q) s += v[q];
            const int c = i / rows, row = i - c * rows;
            p.y[static_cast<int64_t>(c) * p.N + lo + row] = static_cast<uint16_t>(pack_bf16x2(s, 0.f));
        }
        cluster.sync();  // no block leaves while a peer reads its sums
    }
}

// Clusters of kSplit blocks that the device holds at once (asked once per device).
template <int NT>
int resident_clusters(const cudaLaunchConfig_t& cfg) {
    static std::atomic<int> known[64];
    const int dev = device_info().device;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        SetupScope scope;
        if (cudaOccupancyMaxActiveClusters(&n, k_mx4_gemm_async<NT>, &cfg) != cudaSuccess || n < 1) {
            (void)cudaGetLastError();
            n = device_info().sm_count / kSplit / 2 > 0 ? device_info().sm_count / kSplit / 2 : 1;
        }
        known[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

template <int NT>
cudaError_t launch_async(AsyncParams p, cudaStream_t stream) {
    static std::atomic<int> configured[64];
    cudaError_t e = ensure_dynamic_smem(k_mx4_gemm_async<NT>, kAsyncTotal, configured);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(AsyncSmem<NT>::kThreads);
    cfg.dynamicSmemBytes = kAsyncTotal;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;

    // S: 1 or kSplit, the one that ends first by a model in cycles of an SM: the
    // products of its warps (measured at 28672 x 8192) or the weight at its share of
    // HBM; what is not hidden of the copies of X; and the exchange of sums.  Measured
    // with 64 rows at S = 1, 2, 4 and 8: 1024 x 4096 19.0, 16.9, 13.8, 15.1 us; 4096 x
    // 4096 19.4, 21.4, 22.3, -; 8192 x 28672 153, 163, -, - (- : too many sums).
    const int steps = (p.K + Mx4HalfFmt::kStepCols - 1) / Mx4HalfFmt::kStepCols;
    const int per_step = NT == 1 ? 81 : (NT == 2 ? 107 : 300);
    int64_t best = INT64_MAX;
    unsigned grid = 1;
    for (int S = 1; S <= kSplit && S <= steps; S *= kSplit) {
        cfg.gridDim = dim3(static_cast<unsigned>(S));
        attr[0].val.clusterDim.x = static_cast<unsigned>(S);
        cfg.numAttrs = 1;
        int clusters = S == 1 ? device_info().sm_count : resident_clusters<NT>(cfg);
        if (clusters > (p.N + 7) / 8) clusters = (p.N + 7) / 8;
        const int64_t rows = (p.N + clusters - 1) / clusters;
        if (S > 1 && (rows + 1) * p.m * 4 > kPartialBytes) continue;
        constexpr int kRows = 16 * AsyncSmem<NT>::MT;
        const int64_t own = (steps + S - 1) / S, units = (rows + kRows - 1) / kRows * ((p.m + 8 * NT - 1) / (8 * NT));
        int64_t cost = INT64_MAX;
        for (int i = 0; i <= AsyncSmem<NT>::kLogWarps && (i == 0 || (2 << i) <= x_room<NT>(S, p.m)); ++i) {
            const int64_t c = static_cast<int64_t>(warp_steps<NT>(static_cast<int>(units), static_cast<int>(own), i, 1)) *
                              AsyncSmem<NT>::kWarps * per_step;
            if (c < cost) cost = c;
        }
        if (rows * own * 3 > cost) cost = rows * own * 3;
        cost += p.m * own * 3 / 2;
        if (S > 1) cost += cost / 32 + 4000 + rows * p.m;
        if (cost < best) {
            best = cost;
            p.S = S;
            grid = static_cast<unsigned>(clusters * S);
        }
    }
    cfg.gridDim = dim3(grid);
    attr[0].val.clusterDim.x = static_cast<unsigned>(p.S);
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_mx4_gemm_async<NT>, p);
}

cudaError_t launch_prepared(const Mx4View& w, const void* x, void* y, int m, cudaStream_t stream) {
    const DeviceInfo& dev = device_info();
    AsyncParams p{};
    p.w = Mx4HalfFmt::make(w);
    p.y = static_cast<uint16_t*>(y);
    p.N = static_cast<int>(w.rows);
    p.K = static_cast<int>(w.cols);
    p.m = m;
    p.status = device_status_ptr();
    const int steps = (p.K + Mx4HalfFmt::kStepCols - 1) / Mx4HalfFmt::kStepCols;
    const size_t pieces = static_cast<size_t>(steps) * m * 256;
    cudaMemPool_t pool;
    cudaError_t e = scratch_pool(dev.device, &pool);
    if (e != cudaSuccess) return e;
    void* ws = nullptr;
    e = cudaMallocFromPoolAsync(&ws, pieces + kMx4GemmMaxM * 4, pool, stream);
    if (e != cudaSuccess) return e;
    uint8_t* xp = static_cast<uint8_t*>(ws);
    uint32_t* field = reinterpret_cast<uint32_t*>(xp + pieces);
    p.xp = xp;
    p.field = field;
    e = launch_pdl(k_mx4_prepare, dim3(static_cast<unsigned>(m)), dim3(kPrepareThreads), 0, stream, static_cast<const uint16_t*>(x), p.K, m,
                   steps, xp, field);
    if (e == cudaSuccess)
        e = m <= 8 ? launch_async<1>(p, stream)
                   : (m <= 16 ? launch_async<2>(p, stream) : launch_async<4>(p, stream));
    const cudaError_t ef = cudaFreeAsync(ws, stream);
    return e != cudaSuccess ? e : ef;
}

// Preparing costs a launch and a pass over X, about 4 us; without it a block
// refills its copy of X for every round of tiles.  Measured at 8 rows: 10.7
// against 12.0 us at 4096 x 4096 and 48 against 54 at 28672 x 8192 without it, but
// 72 against 54 at 8192 x 28672; at 16 rows 18 against 13 and 74 against 67.
constexpr int kDirectRows = 8;
constexpr int64_t kDirectBytes = 160 * 1024;

}  // namespace

cudaError_t launch_mx4_gemm(const Mx4View& w, const void* x, void* y, int64_t m, cudaStream_t stream) {
    if (w.cols == 0) return cudaMemsetAsync(y, 0, static_cast<size_t>(m * w.rows * 2), stream);  // empty sums
    if (m > kDirectRows || m * w.cols * 2 > kDirectBytes) return launch_prepared(w, x, y, static_cast<int>(m), stream);
    const GemmParams p{Mx4HalfFmt::make(w), static_cast<const uint16_t*>(x), static_cast<uint16_t*>(y), static_cast<int>(w.rows),
                       static_cast<int>(w.cols), static_cast<int>(m)};
    return launch_direct(p, stream);
}

}  // namespace mlxq
