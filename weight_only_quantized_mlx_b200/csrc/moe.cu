// A mixture-of-experts layer for a few tokens, in two kernels:
//   logits = x R^T;  S = the top_k largest of each token (ties: lowest index);
//   p = softmax over S (or over all experts);
//   h[t,j] = p silu(Wg_e x) * (Wu_e x), e = S[t][j];  y[t] = sum_j Wd_e h[t,j].
//
// k_moe_router: a cluster of 8 blocks per token (or 2 or 4 tokens), each block
// an eighth of the experts; logits meet in the first block's shared memory,
// whose warps pick the experts, a token each.
//
// k_moe_experts: one persistent block per SM (cooperative launch).  Each block
// builds the lists of tokens per expert, then streams its share of the hit
// experts' gate and up rows (stream_tile.cuh; the 16 rows of a tile are 8 gate
// rows and the same 8 up rows, so silu(gate) * up is a lane's own business),
// writes h, crosses a grid barrier, and streams its share of the down rows over
// all experts at once.  HBM-bound on the experts hit; each weight byte is read
// once whatever the number of tokens.  The ring is filled with down rows
// before the barrier, so the barrier's wait overlaps their copies.
//
// Rounding: h is rounded to BF16 once (with p in it), the operand type of the
// tensor pipe; sums, silu and p are fp32.
#include <cooperative_groups.h>

#include <utility>

#include "stream_tile.cuh"

namespace mlxq {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxExperts = kMoeMaxExperts;
constexpr int kRouterCluster = 8;
constexpr int kRouterWarps = 8;

// Workspace (see moe_workspace_bytes): 256 bytes holding the barrier count,
// ids [slots], shares [slots], h [slots][inter].
struct MoeWorkspace {
    unsigned int* barrier;
    int* ids;
    float* share;
    uint16_t* h;
};

int64_t align256(int64_t v) { return (v + 255) & ~int64_t{255}; }

MoeWorkspace carve(void* ws, int64_t slots) {
    uint8_t* b = static_cast<uint8_t*>(ws);
    MoeWorkspace r;
    r.barrier = reinterpret_cast<unsigned int*>(b);
    r.ids = reinterpret_cast<int*>(b + 256);
    r.share = reinterpret_cast<float*>(b + 256 + align256(slots * 4));
    r.h = reinterpret_cast<uint16_t*>(b + 256 + 2 * align256(slots * 4));
    return r;
}

// ---- router ------------------------------------------------------------------------------
struct RouterParams {
    const uint16_t* router;  // [E, H]
    const uint16_t* x;       // [m, H]
    int E, H, m, top_k, softmax_all;
    MoeWorkspace ws;
};

// fp32 -> unsigned with the same order; NaN above everything, 0 left free
__device__ __forceinline__ uint32_t order_key(float f) {
    if (f != f) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(f == 0.f ? 0.f : f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float dot8(const uint4& a, const uint4& b, float s) {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s = __fmaf_rn(__uint_as_float(u[i] << 16), __uint_as_float(v[i] << 16), s);
        s = __fmaf_rn(__uint_as_float(u[i] & 0xFFFF0000u), __uint_as_float(v[i] & 0xFFFF0000u), s);
    }
    return s;
}

template <int TB>
__global__ void __cluster_dims__(kRouterCluster, 1, 1) __launch_bounds__(kRouterWarps * 32)
    k_moe_router(const __grid_constant__ RouterParams p) {
    __shared__ float logits[TB][kMaxExperts];          // rank 0: all experts of the cluster's tokens
    __shared__ float part[kRouterWarps][kMaxExperts / kRouterCluster][TB];
    pdl_launch_dependents();
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank());
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = (blockIdx.x / kRouterCluster) * TB;
    auto started = cluster.barrier_arrive();  // waited for before the first write to the root's memory
    pdl_wait();
    // experts rank, rank + 8, ...; with fewer of them than warps, several warps share one's H
    const int mine = p.E > rank ? (p.E - rank - 1) / kRouterCluster + 1 : 0;
    const int split = mine > 4 ? 1 : (mine > 2 ? 2 : (mine > 1 ? 4 : 8));
    const int sub = warp % split, chunks = p.H / 8;
    for (int i = warp / split; i < mine; i += kRouterWarps / split) {
        const uint4* r = reinterpret_cast<const uint4*>(p.router + static_cast<int64_t>(rank + kRouterCluster * i) * p.H);
        float s[TB];
#pragma unroll
        for (int j = 0; j < TB; ++j) s[j] = 0.f;
#pragma unroll 4
        for (int c = sub * 32 + lane; c < chunks; c += 32 * split) {
            const uint4 w = __ldg(r + c);
#pragma unroll
            for (int j = 0; j < TB; ++j)
                if (t0 + j < p.m) s[j] = dot8(w, __ldg(reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(t0 + j) * p.H) + c), s[j]);
        }
#pragma unroll
        for (int j = 0; j < TB; ++j) {
            for (int o = 16; o > 0; o >>= 1) s[j] += __shfl_xor_sync(0xFFFFFFFFu, s[j], o);
            if (lane == 0) part[sub][i][j] = s[j];
        }
    }
    __syncthreads();
    cluster.barrier_wait(std::move(started));
    float* root = cluster.map_shared_rank(&logits[0][0], 0);
    for (int i = threadIdx.x; i < mine * TB; i += kRouterWarps * 32) {
        const int e = i / TB, j = i - e * TB;
        float s = 0.f;
        for (int v = 0; v < split; ++v) s += part[v][e][j];
        root[j * kMaxExperts + rank + kRouterCluster * e] = s;
    }
    cluster.sync();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.ws.barrier = 0u;  // the experts kernel's barrier starts at zero
    if (rank != 0 || warp >= TB || t0 + warp >= p.m) return;
    uint32_t key[kMaxExperts / 32];
#pragma unroll
    for (int i = 0; i < kMaxExperts / 32; ++i) {
        const int e = lane + 32 * i;
        key[i] = e < p.E ? order_key(logits[warp][e]) : 0u;
    }
    float first = 0.f, mine_v = 0.f;  // the largest logit; this lane's pick
    int mine_e = 0;
    for (int j = 0; j < p.top_k; ++j) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < kMaxExperts / 32; ++i) best = max(best, key[i]);
        best = __reduce_max_sync(0xFFFFFFFFu, best);
        uint32_t at = 0xFFFFFFFFu;
#pragma unroll
        for (int i = kMaxExperts / 32 - 1; i >= 0; --i)
            if (key[i] == best) at = static_cast<uint32_t>(lane + 32 * i);
        at = __reduce_min_sync(0xFFFFFFFFu, at);
#pragma unroll
        for (int i = 0; i < kMaxExperts / 32; ++i)
            if (static_cast<uint32_t>(lane + 32 * i) == at) key[i] = 0u;  // taken
        const float v = logits[warp][at];
        if (j == 0) first = v;
        if (lane == j) {
            mine_v = v;
            mine_e = static_cast<int>(at);
        }
    }
    float sum = 0.f;
    if (p.softmax_all) {
        for (int e = lane; e < p.E; e += 32) sum += expf(logits[warp][e] - first);
    } else if (lane < p.top_k) {
        sum = expf(mine_v - first);
    }
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane < p.top_k) {
        const int s = (t0 + warp) * p.top_k + lane;
        p.ws.ids[s] = mine_e;
        p.ws.share[s] = __fdiv_rn(expf(mine_v - first), sum);
    }
}

// ---- experts ------------------------------------------------------------------------------
template <class F>
struct ExpertParams {
    typename F::Mat gate, up, down;
    const uint16_t* x;
    uint16_t* y;
    int E, H, I, m, top_k;
    MoeWorkspace ws;
    unsigned int* status;
};

constexpr int kMaxSlots = kMoeMaxTokens * kMoeMaxTopK;
constexpr int kMaxCols = kMaxSlots + 7 * kMaxExperts;  // lists padded to multiples of 8

struct ExpertLists {
    int count[kMaxExperts];   // tokens of expert e
    int place[kMaxExperts];   // NT > 1: next free entry of expert e's list
    int16_t index[kMaxExperts];  // active index of expert e
    int16_t act[kMaxExperts];    // expert of active index a
    int16_t off[kMaxExperts];
    int16_t cnt[kMaxExperts];
    int16_t cols[kMaxCols];
    int experts;
    int stop;
};

// All threads of the block.  The order of a list's entries has no effect on
// results (MMA columns are independent); the experts are in ascending order.
template <int NT>
__device__ __forceinline__ void build_lists(ExpertLists& L, const int* ids, int slots, int top_k, int E) {
    const int tid = threadIdx.x, lane = tid & 31;
    for (int e = tid; e < kMaxExperts; e += kStreamThreads) L.count[e] = 0;
    for (int c = tid; c < kMaxCols; c += kStreamThreads) L.cols[c] = -1;
    __syncthreads();
    for (int s = tid; s < slots; s += kStreamThreads) atomicAdd(&L.count[ids[s]], 1);
    __syncthreads();
    if (tid < 32) {  // exclusive sums over the experts: active index and list start
        int a = 0, o = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const int n = e < E ? L.count[e] : 0;
            const unsigned hit = __ballot_sync(0xFFFFFFFFu, n > 0);
            int len = n > 0 ? (NT == 1 ? 8 : (n + 7) / 8 * 8) : 0, sum = len;
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, sum, d);
                if (lane >= d) sum += v;
            }
            if (n > 0) {
                const int i = a + __popc(hit & ((1u << lane) - 1u));
                L.index[e] = static_cast<int16_t>(i);
                L.act[i] = static_cast<int16_t>(e);
                L.off[i] = static_cast<int16_t>(o + sum - len);
                L.cnt[i] = static_cast<int16_t>(n);
                L.place[e] = o + sum - len;
            }
            a += __popc(hit);
            o += __shfl_sync(0xFFFFFFFFu, sum, 31);
        }
        if (lane == 0) L.experts = a;
    }
    __syncthreads();
    for (int s = tid; s < slots; s += kStreamThreads) {
        const int e = ids[s];
        const int c = NT == 1 ? L.off[L.index[e]] + s / top_k : atomicAdd(&L.place[e], 1);
        L.cols[c] = static_cast<int16_t>(s);
    }
    __syncthreads();
}

// Every block has passed its writes of h.  Bounded: false (and a status bit)
// when the others do not arrive.
__device__ __forceinline__ bool grid_barrier(unsigned int* count, unsigned int* status, int* stop) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        atomicAdd(count, 1u);
        int gave_up = 0;
        const unsigned long long t0 = globaltimer_ns();
        for (uint32_t it = 1;; ++it) {
            unsigned int v;
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(count) : "memory");
            if (v >= gridDim.x) break;
            if ((it & 63u) == 0u && globaltimer_ns() - t0 > kWaitLimitNs) {
                atomicOr(status, MLXQ_STATUS_TIMEOUT);
                gave_up = 1;
                break;
            }
        }
        __threadfence();
        *stop = gave_up;
    }
    __syncthreads();
    return *stop == 0;
}

template <class F, int NT>
__global__ void __launch_bounds__(kStreamThreads, 1) k_moe_experts(const __grid_constant__ ExpertParams<F> p) {
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* areas = smem + kStreamWarps * kRingBytes;
    ExpertLists& L = *reinterpret_cast<ExpertLists*>(areas + kStreamWarps * kAreaBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * kRingBytes;
    pdl_wait();
    build_lists<NT>(L, p.ws.ids, p.m * p.top_k, p.top_k, p.E);
    const Columns cm{L.cols, L.off, L.cnt, p.top_k};
    const int A = L.experts;

    // ---- gate and up: flattened rows [lo, hi) of A x I, in octets (I % 8 == 0) ----
    {
        const int64_t rows = static_cast<int64_t>(A) * p.I;
        const int64_t lo = rows * blockIdx.x / gridDim.x, hi = rows * (blockIdx.x + 1) / gridDim.x;
        const int64_t o0 = lo >> 3;
        const int octets = hi > lo ? static_cast<int>(((hi - 1) >> 3) - o0) + 1 : 0;
        const int per = p.I >> 3;  // octets of an expert
        const Share sh(octets, (p.H + F::kStepCols - 1) / F::kStepCols, 1, warp);
        float4* area = reinterpret_cast<float4*>(areas + warp * kAreaBytes);
        const float4* group_area = reinterpret_cast<const float4*>(areas + sh.group * sh.k_warps * kAreaBytes);
        constexpr int kAreaVecs = kAreaBytes / 16;
        constexpr int kBatch = 8 / NT;  // tiles between two joins
        Cursor pc(sh);
        uint32_t pslot = 0, cslot = 0;
        auto issue = [&]() {
            if (pc.tile < sh.tiles) {
                const int64_t o = o0 + pc.tile;
                const int a = static_cast<int>(o / per);
                const int64_t row = static_cast<int64_t>(L.act[a]) * p.I + (o - static_cast<int64_t>(a) * per) * 8 + g;
                const bool live = 8 * o + g >= lo && 8 * o + g < hi;
                const StepRows r{row, row, live, live};
                F::issue(p.gate, p.up, ring + pslot * kStageBytes, lane, r, pc.step);
                pc.next(sh);
            }
            cp_async_commit();
            pslot = (pslot + 1) % kDepth;
        };
#pragma unroll 1
        for (int i = 0; i < kDepth - 1; ++i) issue();
        const int own = sh.own_steps();
        for (int tile0 = sh.group; tile0 < sh.tiles; tile0 += sh.groups * kBatch) {
            int batch = 0;
            for (; batch < kBatch; ++batch) {
                const int tile = tile0 + batch * sh.groups;
                if (tile >= sh.tiles) break;
                const int64_t o = o0 + tile;
                const int a = static_cast<int>(o / per);
                const uint32_t low = static_cast<uint32_t>(L.act[a]) * static_cast<uint32_t>(p.I) +
                                     static_cast<uint32_t>((o - static_cast<int64_t>(a) * per) * 8 + g);
                const int nt = NT == 1 ? 1 : (L.cnt[a] + 7) / 8;
                float acc[NT][4];
                const uint16_t* xp[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
                    const int s = n < nt ? cm.slot(a, n * 8 + g) : -1;
                    xp[n] = s >= 0 ? p.x + static_cast<int64_t>(s / p.top_k) * p.H : nullptr;
                }
                int step = sh.kw;
                for (int it = 0; it < own; ++it) {
                    cp_async_wait<kDepth - 2>();
                    __syncwarp();  // the quad's scales have landed; the slot refilled below is read out
                    issue();
                    F::template consume<NT>(p.gate, ring + cslot * kStageBytes, lane, low, step, xp, nt, acc);
                    cslot = (cslot + 1) % kDepth;
                    step += sh.k_warps;
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    if (n < nt) area[(batch * NT + n) * 32 + lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
            }
            group_sync(sh.group, sh.k_warps);
            for (int i = sh.kw * 32 + lane; i < batch * NT * 32; i += sh.k_warps * 32) {
                const int b = i / (NT * 32), n = (i >> 5) % NT, l = i & 31;
                const int64_t o = o0 + tile0 + b * sh.groups;
                const int a = static_cast<int>(o / per);
                if (NT > 1 && n >= (L.cnt[a] + 7) / 8) continue;
                float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int v = 0; v < sh.k_warps; ++v) {
                    const float4 q = group_area[v * kAreaVecs + i];
                    s.x += q.x;
                    s.y += q.y;
                    s.z += q.z;
                    s.w += q.w;
                }
                const int64_t flat = 8 * o + (l >> 2);
                if (flat < lo || flat >= hi) continue;
                const int64_t row = (o - static_cast<int64_t>(a) * per) * 8 + (l >> 2);
                const float gate[2] = {s.x, s.y}, up[2] = {s.z, s.w};
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int slot = cm.slot(a, n * 8 + 2 * (l & 3) + c);
                    if (slot < 0) continue;
                    const float v = p.ws.share[slot] * (__fdiv_rn(gate[c], 1.0f + expf(-gate[c])) * up[c]);
                    p.ws.h[static_cast<int64_t>(slot) * p.I + row] = static_cast<uint16_t>(pack_bf16x2(v, 0.f));
                }
            }
            group_sync(sh.group, sh.k_warps);
        }
        cp_async_wait<0>();
        __syncthreads();  // the groups of the next phase are others: areas are free
    }
    (void)t;

    // ---- down: rows [lo, hi) of y ----
    const int lo = static_cast<int>(static_cast<int64_t>(p.H) * blockIdx.x / gridDim.x);
    const int hi = static_cast<int>(static_cast<int64_t>(p.H) * (blockIdx.x + 1) / gridDim.x);
    stream_rows<F, NT, true>(p.down, p.H, lo, hi, A, L.act, cm, p.ws.h, p.I, p.m, p.y, p.H, ring, areas,
                             [&] { return grid_barrier(p.ws.barrier, p.status, &L.stop); });
}

constexpr size_t kExpertSmem = kStreamWarps * (kRingBytes + kAreaBytes) + sizeof(ExpertLists);
static_assert(kExpertSmem <= 227 * 1024, "shared memory of a block");

template <int TB>
cudaError_t launch_router(const RouterParams& r, cudaStream_t stream) {
    const unsigned clusters = static_cast<unsigned>((r.m + TB - 1) / TB);
    return launch_pdl(k_moe_router<TB>, dim3(clusters * kRouterCluster), dim3(kRouterWarps * 32), 0, stream, r);
}

template <class F, int NT>
cudaError_t launch_experts(const ExpertParams<F>& p, cudaStream_t stream) {
    static std::atomic<int> configured[64];
    cudaError_t e = ensure_dynamic_smem(k_moe_experts<F, NT>, kExpertSmem, configured);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(device_info().sm_count));
    cfg.blockDim = dim3(kStreamThreads);
    cfg.dynamicSmemBytes = kExpertSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;  // the grid barrier needs every block resident
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_moe_experts<F, NT>, p);
}

template <class F, class View>
cudaError_t launch_moe_any(const MoeCall& c, const View& gate, const View& up, const View& down, cudaStream_t stream) {
    const MoeWorkspace ws = carve(c.workspace, static_cast<int64_t>(c.m) * c.top_k);
    const RouterParams r{static_cast<const uint16_t*>(c.router), static_cast<const uint16_t*>(c.x), c.experts, c.hidden, c.m,
                         c.top_k, c.softmax_all, ws};
    // few tokens: a cluster each; more: several tokens share a pass over the
    // router's weights, so that the clusters still fit the SMs at once
    cudaError_t e = c.m <= 16 ? launch_router<1>(r, stream) : (c.m <= 32 ? launch_router<2>(r, stream) : launch_router<4>(r, stream));
    if (e != cudaSuccess) return e;
    const ExpertParams<F> p{F::make(gate), F::make(up), F::make(down), static_cast<const uint16_t*>(c.x),
                            static_cast<uint16_t*>(c.y), c.experts, c.hidden, c.inter, c.m, c.top_k, ws, device_status_ptr()};
    if (c.m <= 8) return launch_experts<F, 1>(p, stream);
    if (c.m <= 16) return launch_experts<F, 2>(p, stream);
    if (c.m <= 32) return launch_experts<F, 4>(p, stream);
    return launch_experts<F, 8>(p, stream);
}

}  // namespace

size_t moe_workspace_bytes(int64_t inter, int64_t slots) {
    return static_cast<size_t>(256 + 2 * align256(slots * 4) + align256(slots * inter * 2));
}

cudaError_t launch_moe(const MoeCall& c, const WeightView& gate, const WeightView& up, const WeightView& down,
                       cudaStream_t stream) {
    return launch_moe_any<Q8Fmt>(c, gate, up, down, stream);
}

cudaError_t launch_mx4_moe(const MoeCall& c, const Mx4View& gate, const Mx4View& up, const Mx4View& down,
                           cudaStream_t stream) {
    return launch_moe_any<Mx4Fmt>(c, gate, up, down, stream);
}

}  // namespace mlxq
