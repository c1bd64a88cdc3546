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
// experts' gate and up rows (row_stream.cuh; the 16 rows of a tile are 8 gate
// rows and the same 8 up rows, so silu(gate) * up is a lane's own business),
// writes h, crosses a grid barrier (two, with a conversion of h between them, in one
// form: see Rounding), and streams its share of the down rows over all experts at
// once.  Each weight byte of a hit expert is read once (again for every 8 NT tokens
// more of one expert).  The ring is filled with down rows before the barrier, so the
// barrier's wait overlaps their copies.
//
// Measured: one token, two of 8 experts of 4096 x 14336, 8 bits: 108 us (the
// weights' copy time is 57); 64 tokens, 128 experts of 4128 x 1504, MX4: 465 us
// (190).  Neither fills a unit (issue slots 63 and 59 %, ALU 62 and 52 %, DRAM 43 and
// 36 %): the four warps of a scheduler mostly wait for their own instructions' results
// and for one another, most of the instructions turning codes into operands.  One
// token, 8 of 64 experts of 2048 x 1024, MX4: 25 us (4), a chain of latencies: router
// 5 us, lists 1.4, first copies and activations 2.3, gate and up 5, barrier 3.5, down
// 4.2.
//
// Rounding: the tensor pipe takes 16-bit operands, and one BF16 value for h (with p in
// it) showed in y (relative error 2.4e-3 against 1.7e-3 of y's own rounding).  So h is
// held as the sum of two BF16 values, a column of the down product each, to 2^-16 of
// itself; or, for MX4 and more than four tokens, as FP16 in units of the slot's
// largest power of two, to 2^-11 (and to 2^-39 of the largest), for which the blocks
// write fp32, cross a barrier and convert a share each: half the products, and the
// codes need no BF16 form (64 tokens, 128 experts of 4128 x 1504: 480 us against 535 with
// two parts; 8 tokens, 64 experts of 2048 x 1024: 63 against 72; 64 tokens, 8 of 32 experts: 128
// against 142).  With BF16 weights FP16 is not open.  Sums, silu and p are fp32.
#include <cooperative_groups.h>

#include <utility>

#include "row_stream.cuh"

namespace mlxq {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxExperts = kMoeMaxExperts;
constexpr int kRouterCluster = 8;
constexpr int kRouterWarps = 16;

// Workspace (see moe_workspace_bytes): 256 bytes holding the barrier count,
// ids [slots], shares [slots], largest exponents [slots], h.  Where h is the sum of two
// BF16 parts: h [slots][F::h_row(inter)], in the order in which the down phase reads it
// (F::place); else raw [slots][inter] fp32 and h [slots][inter] FP16, made of raw.
constexpr int kHStep = 128;  // F::h_row is at most 2 inter rounded up to it
struct MoeWorkspace {
    unsigned int* barrier;
    int* ids;
    float* share;
    uint32_t* top;
    float* raw;
    uint16_t* h;
};

int64_t align256(int64_t v) { return (v + 255) & ~int64_t{255}; }

int64_t raw_bytes(int64_t inter, int64_t slots) { return align256(slots * ((inter + kHStep - 1) / kHStep * kHStep) * 4); }

MoeWorkspace carve(void* ws, int64_t inter, int64_t slots, bool pair) {
    uint8_t* b = static_cast<uint8_t*>(ws);
    const int64_t per_slot = align256(slots * 4);
    MoeWorkspace r;
    r.barrier = reinterpret_cast<unsigned int*>(b);
    r.ids = reinterpret_cast<int*>(b + 256);
    r.share = reinterpret_cast<float*>(b + 256 + per_slot);
    r.top = reinterpret_cast<uint32_t*>(b + 256 + 2 * per_slot);
    b += 256 + 3 * per_slot;
    r.raw = reinterpret_cast<float*>(b);
    r.h = reinterpret_cast<uint16_t*>(pair ? b : b + raw_bytes(inter, slots));
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
    // experts rank, rank + 8, ...; with fewer of them than warps, several warps share one's H.
    // As many for every expert of the call: equal rows have equal sums, whose block's they are.
    const int mine = p.E > rank ? (p.E - rank - 1) / kRouterCluster + 1 : 0;
    const int most = (p.E + kRouterCluster - 1) / kRouterCluster;
    const int split = most > 8 ? 1 : (most > 4 ? 2 : (most > 2 ? 4 : (most > 1 ? 8 : 16)));
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
        p.ws.top[s] = 0u;
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

// The hit experts with their tokens, as entries of up to 8 NT columns (an expert
// with more tokens takes several entries: its weights are then streamed once for
// each).  A slot is token * top_k + choice.  Up to 8 tokens (NT == 1):
// column = token, eight columns per entry, -1 where the token did not choose the
// expert.  Otherwise an entry's slots one after another, padded with -1 to a
// multiple of 8.
constexpr int kMaxSlots = kMoeMaxTokens * kMoeMaxTopK;
constexpr int kMaxEntries = kMaxExperts + kMaxSlots / 16;
constexpr int kMaxListed = kMaxSlots + 7 * kMaxExperts;  // lists padded to multiples of 8

struct ExpertLists {
    int count[kMaxExperts];      // tokens of expert e
    int place[kMaxExperts];      // first column of expert e, then its next free one
    int16_t act[kMaxEntries];    // expert of entry a
    int16_t off[kMaxEntries];    // its first column
    int16_t cnt[kMaxEntries];    // its columns
    int16_t cols[kMaxListed];    // slots
    uint8_t field[kMaxListed];   // their largest exponent fields, where h is FP16
    long long before[kMaxEntries + 1];  // NT > 1: weight of all gate and up rows before entry a's
    int entries;
    int columns;                 // places of `cols` in use
    int stop;

    // What a row of entry a costs: some fixed work, and the products of its column
    // tiles (measured 132, 165 and 243 cycles a step at one, two and four).
    __device__ __forceinline__ int weight(int a) const { return cnt[a] <= 8 ? 4 : (cnt[a] <= 16 ? 5 : 7); }
};

struct Columns {
    const int16_t* cols;
    const int16_t* off;
    const int16_t* cnt;
    int top_k;
    __device__ __forceinline__ int slot(int a, int c) const { return cols[off[a] + c]; }
};

// All threads of the block.  Entries are in ascending order of experts.  The
// order of an entry's columns has no effect on results (MMA columns are
// independent), so they are placed by atomics; which entry of several a token
// falls into could change the order of sums, so there a slot's place is its rank.
__device__ __forceinline__ void clear_lists(ExpertLists& L, int E) {
    for (int e = threadIdx.x; e < E; e += kStreamThreads) L.count[e] = 0;
    for (int c = threadIdx.x; c < kMaxListed; c += kStreamThreads) L.cols[c] = -1;
    __syncthreads();
}

template <int NT>
__device__ __forceinline__ void build_lists(ExpertLists& L, const int* ids, int slots, int top_k, int E, int I) {
    constexpr int kMaxCols = 8 * NT;
    const int tid = threadIdx.x, lane = tid & 31;
    for (int s = tid; s < slots; s += kStreamThreads) atomicAdd(&L.count[ids[s]], 1);
    __syncthreads();
    if (tid < 32) {  // exclusive sums over the experts: first entry and first column
        int a = 0, o = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const int n = e < E ? L.count[e] : 0;
            const int own = (n + kMaxCols - 1) / kMaxCols, len = n > 0 ? (NT == 1 ? 8 : (n + 7) / 8 * 8) : 0;
            int sum = len << 16 | own;  // both at once; columns < 2^15, entries < 2^16
            const int mine = sum;
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, sum, d);
                if (lane >= d) sum += v;
            }
            const int i = a + ((sum - mine) & 0xFFFF), c = o + ((sum - mine) >> 16);
            for (int j = 0; j < own; ++j) {
                L.act[i + j] = static_cast<int16_t>(e);
                L.off[i + j] = static_cast<int16_t>(c + j * kMaxCols);
                L.cnt[i + j] = static_cast<int16_t>(min(n - j * kMaxCols, kMaxCols));
            }
            if (n > 0) L.place[e] = c;
            const int total = __shfl_sync(0xFFFFFFFFu, sum, 31);
            a += total & 0xFFFF;
            o += total >> 16;
        }
        if (lane == 0) {
            L.entries = a;
            L.columns = o;
        }
    }
    __syncthreads();
    for (int s = tid; s < slots; s += kStreamThreads) {
        const int e = ids[s];
        int c;
        if (NT == 1) {
            c = L.place[e] + s / top_k;
        } else if (L.count[e] <= kMaxCols) {
            c = atomicAdd(&L.place[e], 1);
        } else {
            c = L.place[e];
            for (int q = 0; q < s; ++q) c += ids[q] == e;
        }
        L.cols[c] = static_cast<int16_t>(s);
    }
    if (NT > 1 && tid < 32) {  // exclusive sums of the entries' weights
        long long sum = 0;
        for (int a0 = 0; a0 < L.entries; a0 += 32) {
            const int a = a0 + lane;
            long long v = a < L.entries ? static_cast<long long>(I) * L.weight(a) : 0;
            const long long mine = v;
            for (int d = 1; d < 32; d <<= 1) {
                const long long u = __shfl_up_sync(0xFFFFFFFFu, v, d);
                if (lane >= d) v += u;
            }
            if (a < L.entries) L.before[a] = sum + v - mine;
            sum += __shfl_sync(0xFFFFFFFFu, v, 31);
        }
        if (lane == 0) L.before[L.entries] = sum;
    }
    __syncthreads();
}

// Every block has come here `times` times, its writes before are seen.  Bounded:
// false (and a status bit) when the others do not arrive.
__device__ __forceinline__ bool grid_barrier(unsigned int* count, unsigned int times, unsigned int* status, int* stop) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        atomicAdd(count, 1u);
        int gave_up = 0;
        const unsigned long long t0 = globaltimer_ns();
        for (uint32_t it = 1;; ++it) {
            unsigned int v;
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(count) : "memory");
            if (v >= times * gridDim.x) break;
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

// ---- the streaming phases --------------------------------------------------------------------
// Shared memory: rings | lists | gate and up: areas, column exponents, activations
//                              | down: areas.
template <int NT>
struct Smem {
    static constexpr int kTokens = NT == 1 ? 8 : kMoeMaxTokens;  // most tokens of a call
    static constexpr uint32_t kDownArea = NT == 1 ? 2048 : 16 * (kTokens + 4) * 4;  // a warp's sums of the down phase
    static constexpr uint32_t kLists = kStreamWarps * Ring<NT>::kBytes;
    static constexpr uint32_t kAreas = (kLists + sizeof(ExpertLists) + 127) / 128 * 128;
    static constexpr uint32_t kFields = kAreas + kStreamWarps * kSharedArea;
    static constexpr uint32_t kX = kFields + 2 * kMoeMaxTokens * 4;
    static constexpr uint32_t kTotal = 227 * 1024;
    static constexpr uint32_t kXBytes = kTotal - kX;
    static_assert(kX % 16 == 0 && kX + 16 * 1024 <= kTotal, "room for one step of 64 columns");
    static_assert(kAreas + kStreamWarps * kDownArea <= kTotal && kDownArea % 16 == 0, "areas of the down phase");
};

// h as two parts that BF16 takes: its top half, cut (so that it is finite where h is), and the
// rest, which the caller rounds (to 2^-9 of 2^-7 of h).  Neither is zero where h is
// not, since an infinite weight times zero would be NaN: an h that BF16 holds whole
// comes as two halves, and so do infinities and NaN.  (Next to BF16's subnormals a half
// would lose a bit: there the rest is zero.)
__device__ __forceinline__ float2 two_parts(float h) {
    const float top = __uint_as_float(__float_as_uint(h) & 0xFFFF0000u), rest = h - top;
    if (fabsf(rest) > 0.f || fabsf(h) < 0x1p-100f) return make_float2(top, rest);
    return make_float2(0.5f * h, 0.5f * h);
}

// gate and up, then h = p silu(gate) up, for the flattened rows [lo, hi) of
// (hit experts) x I, in octets (I % 8 == 0): a tile is 8 gate rows and the
// same 8 up rows, so the lane that holds a gate sum holds its up sum.  With up
// to 8 tokens all tiles are one segment (column = token), else a segment is an
// expert (columns = its tokens).
template <class F, class FD, int NT>
struct GateUpJob {
    const ExpertParams<F>& p;
    const typename F::Mat& mat;
    const ExpertLists& L;
    Columns cm;
    int64_t lo, hi;
    int K, per, o0, octets, a_first, segs;  // per: octets of an expert; o0: the first octet (A I / 8 < 2^26)

    __device__ __forceinline__ GateUpJob(const ExpertParams<F>& p_, const ExpertLists& L_, const Columns& cm_)
        : p(p_), mat(p_.gate), L(L_), cm(cm_) {
        lo = first_row(blockIdx.x);
        hi = first_row(blockIdx.x + 1);
        K = p.H;
        per = p.I >> 3;
        o0 = static_cast<int>(lo >> 3);
        octets = lo < hi ? static_cast<int>((hi - 1) >> 3) - o0 + 1 : 0;
        a_first = o0 / per;
        segs = octets == 0 ? 0 : (NT == 1 ? 1 : (o0 + octets - 1) / per - a_first + 1);
    }
    // The first of the rows that block b takes: shares of equal weight.
    __device__ __forceinline__ int64_t first_row(unsigned b) const {
        if (NT == 1) return static_cast<int64_t>(L.entries) * p.I * b / gridDim.x;
        const long long at = L.before[L.entries] * b / gridDim.x;
        int a = 0, n = L.entries;  // the last entry that begins at or before `at`
        while (n > 1) {
            const int half = n >> 1;
            if (L.before[a + half] <= at) a += half;
            n -= half;
        }
        const int64_t row = static_cast<int64_t>(a) * p.I + (at - L.before[a]) / L.weight(a);
        return row;
    }
    __device__ __forceinline__ int begin(int s) const { return NT == 1 ? 0 : max((a_first + s) * per - o0, 0); }
    __device__ __forceinline__ int end(int s) const { return NT == 1 ? octets : min((a_first + s + 1) * per - o0, octets); }
    __device__ __forceinline__ int cols(int s) const { return NT == 1 ? p.m : static_cast<int>(L.cnt[a_first + s]); }
    __device__ __forceinline__ const uint16_t* x_row(int s, int c) const {
        const int token = NT == 1 ? c : cm.slot(a_first + s, c) / p.top_k;
        return p.x + static_cast<int64_t>(token) * p.H;
    }
    __device__ __forceinline__ void start(typename F::Feed& f, int tile, int lane, int step) const {
        const int o = o0 + tile, a = o / per, g = lane >> 2;
        const int64_t row = static_cast<int64_t>(L.act[a]) * p.I + (o - a * per) * 8 + g;
        const int64_t flat = 8 * static_cast<int64_t>(o) + g;
        const bool live = flat >= lo && flat < hi;
        F::start(f, p.gate, p.up, row, row, live, live, lane, step);
    }
    __device__ __forceinline__ uint32_t key(int tile, int lane) const {
        const int o = o0 + tile, a = o / per;
        return F::row_key(p.gate, static_cast<uint32_t>(L.act[a]) * static_cast<uint32_t>(p.I) +
                                      static_cast<uint32_t>((o - a * per) * 8 + (lane >> 2)));
    }
    // (all lanes of a warp, for one tile)
    __device__ __forceinline__ void store(int s, int tile, int n, int lane, const float4& v) const {
        const int o = o0 + tile, a = o / per, g = lane >> 2;
        const int64_t flat = 8 * static_cast<int64_t>(o) + g;
        const bool live = flat >= lo && flat < hi;
        const int row = (o - a * per) * 8 + g;
        const float gate[2] = {v.x, v.y}, up[2] = {v.z, v.w};
        uint32_t field = 0;  // both columns' exponent fields, 16 bits each
        int slot[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = n * 8 + 2 * (lane & 3) + i;
            slot[i] = c < cols(s) ? cm.slot(a, c) : -1;
            if (slot[i] < 0 || !live) continue;
            const float h = p.ws.share[slot[i]] * (__fdiv_rn(gate[i], 1.0f + expf(-gate[i])) * up[i]);
            if constexpr (FD::kPair) {
                uint16_t* at = p.ws.h + static_cast<int64_t>(slot[i]) * FD::h_row(p.I) + FD::place(row);
                const float2 parts = two_parts(h);
                at[0] = static_cast<uint16_t>(__float_as_uint(parts.x) >> 16);
                at[32] = static_cast<uint16_t>(pack_bf16x2(parts.y, 0.f));
            } else {
                p.ws.raw[static_cast<int64_t>(slot[i]) * p.I + row] = h;
                field |= (__float_as_uint(h) >> 23 & 255u) << (16 * i);
            }
        }
        if constexpr (!FD::kPair) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) field = __vmaxu2(field, __shfl_xor_sync(0xFFFFFFFFu, field, d));
            if (g == 0) {  // the same columns' eight rows: one lane tells
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (slot[i] >= 0) atomicMax(p.ws.top + slot[i], field >> (16 * i) & 0xFFFFu);
            }
        }
    }
};

// raw -> h, the grid's blocks a share each; and the list's exponent fields.
template <class Params>
__device__ __forceinline__ void convert_h(const Params& p, ExpertLists& L, int listed) {
    const int per = p.I >> 3, pieces = p.m * p.top_k * per;  // (1024 slots of 2^17 pieces at most)
    for (int i = blockIdx.x * kStreamThreads + threadIdx.x; i < pieces; i += gridDim.x * kStreamThreads) {
        const float f = x_inverse(p.ws.top[i / per]);
        const float4* from = reinterpret_cast<const float4*>(p.ws.raw) + 2 * static_cast<int64_t>(i);
        const float4 a = from[0], b = from[1];
        uint4 v;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(v.x) : "f"(a.y * f), "f"(a.x * f));
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(v.y) : "f"(a.w * f), "f"(a.z * f));
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(v.z) : "f"(b.y * f), "f"(b.x * f));
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(v.w) : "f"(b.w * f), "f"(b.z * f));
        reinterpret_cast<uint4*>(p.ws.h)[i] = v;
    }
    for (int c = threadIdx.x; c < listed; c += kStreamThreads) {
        const int s = L.cols[c];
        L.field[c] = static_cast<uint8_t>(s >= 0 ? p.ws.top[s] : 0u);
    }
}

// y[token][row] = sum over hit experts a and columns k of Wd_a[row, k] h[slot][k]
// for the block's rows [lo, hi).  Tiles are 16 rows; every expert's slice of a
// tile goes into one accumulator, so the sum over experts needs no second pass
// and no atomics: with up to 8 tokens column = token and each expert's fragment is
// added, where the token chose the expert, else each warp adds an expert's columns to
// its own [16][tokens] sums in shared memory.  The warps that share a tile join in
// warp order, so results do not depend on timing.  Where h has two parts (F::kPair)
// a column tile holds four slots, both parts of each side by side, so that one lane
// gets both parts' sums; else eight.  h is read once or twice per block, so it is not
// staged: a lane loads the next step's first column tile before it multiplies the
// present one.  `ready` runs once the ring has been filled (weights only) and before h
// is read; false ends the phase.
template <class F, int NT, class Params, class Ready>
__device__ __forceinline__ void down_phase(const Params& p, const ExpertLists& L, const Columns& cm, uint32_t ring,
                                           uint8_t* areas, Ready ready) {
    constexpr int kDepth = Ring<NT>::kDepth;
    constexpr uint32_t kRingBytes = Ring<NT>::kBytes;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int lo = static_cast<int>(static_cast<int64_t>(p.H) * blockIdx.x / gridDim.x);
    const int hi = static_cast<int>(static_cast<int64_t>(p.H) * (blockIdx.x + 1) / gridDim.x);
    const int tiles = (hi - lo + 15) / 16, S = (p.I + F::kStepCols - 1) / F::kStepCols, A = L.entries;
    // The warps of a tile (2^lw) split the experts into contiguous ranges and,
    // 2^ls of them together, the steps of an expert in turns: turns bring
    // neighbouring 64-byte pieces of a row at about the same time (four or more
    // warps: whole DRAM bursts; copies alone measured 6 TB/s, against 2.9 with one
    // warp walking a row), ranges change expert seldom.  Lane i weighs one pair:
    // steps, about one for a change of expert, two for a join, and an eighth more
    // below four turns.
    int lw, ls;
    {
        const int i = min(lane, 14), w = i < 1 ? 0 : (i < 3 ? 1 : (i < 6 ? 2 : (i < 10 ? 3 : 4))), d = i - w * (w + 1) / 2;
        const int rounds = (tiles + (kStreamWarps >> w) - 1) >> (4 - w), ranges = 1 << (w - d);
        int cost = rounds * (((A + ranges - 1) >> (w - d)) * (((S + (1 << d) - 1) >> d) + 1) + (w > 0 ? 2 : 0));
        if (d < 2) cost += cost / 8;
        const uint32_t best = __reduce_min_sync(0xFFFFFFFFu, static_cast<uint32_t>(min(cost, 0x07FFFFFF)) << 4 | static_cast<uint32_t>(i)) & 15u;
        lw = __shfl_sync(0xFFFFFFFFu, w, static_cast<int>(best));
        ls = __shfl_sync(0xFFFFFFFFu, d, static_cast<int>(best));
    }
    const int wk = 1 << lw, groups = kStreamWarps >> lw, group = warp >> lw, kw = warp & (wk - 1);
    const int turns = 1 << ls, s0 = kw & (turns - 1);
    const int a0 = A * (kw >> ls) >> (lw - ls), a1 = A * ((kw >> ls) + 1) >> (lw - ls);  // this warp's experts
    const bool idle = a0 >= a1 || s0 >= S;
    constexpr int kBatch = NT == 1 ? 4 : 1;           // tiles between two joins
    constexpr int kAreaFloats = Smem<NT>::kDownArea / 4;
    constexpr int kStride = Smem<NT>::kTokens + 1;    // NT > 1: floats per row of the area
    constexpr int kSlots = F::kPair ? 4 : 8;          // slots of a column tile
    constexpr int DT = 8 * NT / kSlots;               // column tiles of an entry
    // The first tile's h is loaded a step ahead, except with four tiles of MX4, whose registers
    // do not reach (64 tokens, 8 of 32 experts of 2048 x 1024: 132 us with it, 128 without).
    constexpr bool kAhead = F::kPieces == 2 || NT < 4;
    float* area = reinterpret_cast<float*>(areas + warp * Smem<NT>::kDownArea);
    const float* group_area = reinterpret_cast<const float*>(areas + group * wk * Smem<NT>::kDownArea);

    int ptile = idle ? tiles : group, pa = a0, pstep = s0;
    uint32_t pslot = ring, cslot = ring;
    typename F::Feed feed;
    auto restart = [&]() {
        if (ptile >= tiles) return;
        const int r = lo + ptile * 16 + g;
        const int64_t row = static_cast<int64_t>(L.act[pa]) * p.H + r;
        F::start(feed, p.down, p.down, row, row + 8, r < hi, r + 8 < hi, lane, s0);
    };
    restart();
    auto issue = [&]() {
        if (ptile < tiles) {
            F::issue(p.down, feed, pslot, lane, turns);
            pstep += turns;
            if (pstep >= S) {
                pstep = s0;
                if (++pa == a1) {
                    pa = a0;
                    ptile += groups;
                }
                restart();
            }
        }
        cp_async_commit();
        pslot = pslot == ring + kRingBytes - kStageBytes ? ring : pslot + kStageBytes;
    };
#pragma unroll 1
    for (int i = 0; i < kDepth - 1; ++i) issue();
    if (!ready()) {
        cp_async_wait<0>();
        return;
    }

    for (int tile0 = group; tile0 < tiles; tile0 += groups * kBatch) {
        int batch = 0;
        for (; batch < kBatch; ++batch) {
            const int tile = tile0 + batch * groups;
            if (tile >= tiles) break;
            float acc[DT][4];
            float sum[4] = {0.f, 0.f, 0.f, 0.f};  // NT == 1: over the experts; rows g and g + 8 of one slot, then of another
            int xp[DT];  // this lane's rows of h, at its place in a step, in units of 8 values; -1: none
#pragma unroll
            for (int n = 0; n < DT; ++n) {
                acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
                xp[n] = -1;
            }
            if (NT > 1) {
                for (int i = lane; i < 16 * kStride; i += 32) area[i] = 0.f;
                __syncwarp();
            }
            auto scatter = [&](int a, int nt) {
#pragma unroll
                for (int n = 0; n < DT; ++n) {
                    if (n >= nt) break;
                    if constexpr (F::kPair) {
                        const int s = cm.slot(a, n * 4 + t);
                        if (s >= 0) {
                            const int token = s / cm.top_k;
                            area[g * kStride + token] += F::kUnit * (acc[n][0] + acc[n][1]);
                            area[(g + 8) * kStride + token] += F::kUnit * (acc[n][2] + acc[n][3]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int s = cm.slot(a, n * 8 + 2 * t + i);
                            if (s >= 0) {
                                const int token = s / cm.top_k;
                                area[g * kStride + token] += acc[n][i];
                                area[(g + 8) * kStride + token] += acc[n][2 + i];
                            }
                        }
                    }
                }
                // all tiles: an unused one that was multiplied holds zeros times weights, NaN where they are infinite
#pragma unroll
                for (int n = 0; n < DT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
                __syncwarp();
            };
            auto column = [&](int a, int n) {
                const int s = cm.slot(a, F::kPair ? n * 4 + (g >> 1) : n * 8 + g);
                if (s < 0) return -1;
                if constexpr (F::kPair) return s * (F::h_row(p.I) >> 3) + (g & 1) * 4 + t;  // (< 2^28)
                else return s * (p.I >> 3) + t;
            };
            // piece i of the lane's row of h for a step; zeros where there is none
            auto piece = [&](int row, int step, int i) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                const bool in = F::kPair ? step * F::kStepCols + t * (8 * F::kPieces) < p.I : step * F::kStepCols + 32 * i < p.I;
                if (row >= 0 && in)
                    v = ldg128(reinterpret_cast<const uint4*>(p.ws.h) + row +
                               (F::kPair ? (step * F::kPieces + i) * 8 : step * (F::kStepCols / 8) + 4 * i));
                return v;
            };
            auto fetch = [&](uint4 (&v)[F::kPieces], int row, int step) {
#pragma unroll
                for (int i = 0; i < F::kPieces; ++i) v[i] = piece(row, step, i);
            };
            uint4 x0[F::kPieces];
            int row0 = -1;  // h of column tile 0
            if (!idle) {
                row0 = column(a0, 0);
                if (kAhead) fetch(x0, row0, s0);
            }
            for (int a = a0; a < a1 && !idle; ++a) {
                const int nt = ((NT == 1 ? p.m : cm.cnt[a]) + kSlots - 1) / kSlots;
#pragma unroll
                for (int n = 1; n < DT; ++n) xp[n] = n < nt ? column(a, n) : -1;
                const uint32_t key = F::row_key(p.down, static_cast<uint32_t>(L.act[a]) * static_cast<uint32_t>(p.H) +
                                                            static_cast<uint32_t>(lo + tile * 16 + g));
                const int next0 = a + 1 < a1 ? column(a + 1, 0) : -1;
                [[maybe_unused]] bool plain = true;  // sums are in the columns' units (FP16)
                [[maybe_unused]] auto unit = [&](int c) { return x_unit(L.field[cm.off[a] + min(c, nt * 8 - 1)]); };
                // N column tiles, a power of two: unused ones are zeros
                auto run = [&](auto count) {
                    constexpr int N = decltype(count)::value < DT ? decltype(count)::value : DT;
#pragma unroll 1
                    for (int step = s0; step < S; step += turns) {
                        const bool turn = step + turns >= S;
                        uint4 x1[F::kPieces];
                        if (kAhead) fetch(x1, turn ? next0 : row0, turn ? s0 : step + turns);
                        cp_async_wait<kDepth - 2>();
                        __syncwarp();  // the copies of all lanes have landed; the slot refilled below is read out
                        issue();
                        auto x = [&](int i, int n) {
                            if (n > 0 || !kAhead) return piece(n > 0 ? xp[n] : row0, step, i);
                            uint4 v = x0[0];  // (not indexed: a loop over i may stay one, and x0 has to stay in registers)
#pragma unroll
                            for (int j = 1; j < F::kPieces; ++j)
                                if (i == j) v = x0[j];
                            return v;
                        };
                        if constexpr (F::kPair) {
                            F::template consume<DT, N>(p.down, cslot, lane, key, step, acc, x);
                        } else {
                            const uint32_t keys[1] = {key};
                            F::template consume_tiles<1, DT, N>(p.down, cslot, lane, keys, step, reinterpret_cast<float(&)[1][DT][4]>(acc), plain,
                                                                x, unit);
                        }
                        cslot = cslot == ring + kRingBytes - kStageBytes ? ring : cslot + kStageBytes;
#pragma unroll
                        for (int i = 0; i < F::kPieces && kAhead; ++i) x0[i] = x1[i];
                    }
                };
                if (DT == 1 || nt == 1) run(std::integral_constant<int, 1>{});
                else if (DT == 2 || nt == 2) run(std::integral_constant<int, 2>{});
                else if (DT == 4 || nt <= 4) run(std::integral_constant<int, 4>{});
                else run(std::integral_constant<int, 8>{});
                row0 = next0;
                if constexpr (!F::kPair) {
                    if (plain) F::template to_numbers<DT>(acc, t, unit);
                }
                if (NT > 1) {
                    scatter(a, nt);
                } else {
                    // a token that did not choose the expert gets nothing of it: zeros
                    // times an infinite or NaN weight would not be zero
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int n = F::kPair ? i : 0;
                        if (cm.slot(a, F::kPair ? 4 * i + t : 2 * t + i) < 0) continue;
                        sum[2 * i] += F::kPair ? F::kUnit * (acc[n][0] + acc[n][1]) : acc[n][i];
                        sum[2 * i + 1] += F::kPair ? F::kUnit * (acc[n][2] + acc[n][3]) : acc[n][2 + i];
                    }
#pragma unroll
                    for (int n = 0; n < DT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
                }
            }
            if (NT == 1) reinterpret_cast<float4*>(area)[batch * 32 + lane] = make_float4(sum[0], sum[1], sum[2], sum[3]);
        }
        group_sync(group, wk);
        const int me = kw * 32 + lane, threads = wk * 32;
        if (NT == 1) {
            for (int i = me; i < batch * 32; i += threads) {
                float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int v = 0; v < wk; ++v) {
                    const float4 q = reinterpret_cast<const float4*>(group_area + v * kAreaFloats)[i];
                    s.x += q.x;
                    s.y += q.y;
                    s.z += q.z;
                    s.w += q.w;
                }
                const int r = lo + (tile0 + (i >> 5) * groups) * 16 + ((i & 31) >> 2), q = i & 3;
                const uint32_t b0 = pack_bf16x2(s.x, s.y), b1 = pack_bf16x2(s.z, s.w);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int c = F::kPair ? 4 * j + q : 2 * q + j;
                    uint16_t* y = p.y + static_cast<int64_t>(c) * p.H + r;
                    const uint32_t b = j == 0 ? b0 : b1;
                    if (c < p.m && r < hi) y[0] = static_cast<uint16_t>(b);
                    if (c < p.m && r + 8 < hi) y[8] = static_cast<uint16_t>(b >> 16);
                }
            }
        } else {
            const int r0 = lo + tile0 * 16;
            for (int i = me; i < 16 * p.m; i += threads) {
                const int r = i & 15, c = i >> 4;
                float s = 0.f;
                for (int v = 0; v < wk; ++v) s += group_area[v * kAreaFloats + r * kStride + c];
                if (r0 + r < hi) p.y[static_cast<int64_t>(c) * p.H + r0 + r] = static_cast<uint16_t>(pack_bf16x2(s, 0.f));
            }
        }
        group_sync(group, wk);
    }
    cp_async_wait<0>();
}

// FG: the format's form for shared activations (gate and up), FD: for the down phase.
template <class FG, class FD, int NT>
__global__ void __launch_bounds__(kStreamThreads, 1) k_moe_experts(const __grid_constant__ ExpertParams<FG> p) {
    extern __shared__ __align__(128) uint8_t smem[];
    using M = Smem<NT>;
    ExpertLists& L = *reinterpret_cast<ExpertLists*>(smem + M::kLists);
    uint32_t* field = reinterpret_cast<uint32_t*>(smem + M::kFields);
    const uint32_t ring = smem_u32(smem) + (threadIdx.x >> 5) * Ring<NT>::kBytes;
    clear_lists(L, p.E);
    pdl_wait();
    build_lists<NT>(L, p.ws.ids, p.m * p.top_k, p.top_k, p.E, p.I);
    const Columns cm{L.cols, L.off, L.cnt, p.top_k};
    const XBuffer xb{smem_u32(smem) + M::kX, static_cast<int>(M::kXBytes), field, field + kMoeMaxTokens};
    shared_phase<FG, NT>(GateUpJob<FG, FD, NT>(p, L, cm), ring, smem + M::kAreas, xb);
    __syncthreads();  // the groups of the next phase are others, and its areas lie over the activations
    down_phase<FD, NT>(p, L, cm, ring, smem + M::kAreas, [&] {
        if (!grid_barrier(p.ws.barrier, 1u, p.status, &L.stop)) return false;
        if constexpr (FD::kPair) return true;
        convert_h(p, L, L.columns);
        return grid_barrier(p.ws.barrier, 2u, p.status, &L.stop);
    });
}

template <int TB>
cudaError_t launch_router(const RouterParams& r, cudaStream_t stream) {
    const unsigned clusters = static_cast<unsigned>((r.m + TB - 1) / TB);
    return launch_pdl(k_moe_router<TB>, dim3(clusters * kRouterCluster), dim3(kRouterWarps * 32), 0, stream, r);
}

template <class FG, class FD, int NT>
cudaError_t launch_experts(const ExpertParams<FG>& p, cudaStream_t stream) {
    static std::atomic<int> configured[64];
    cudaError_t e = ensure_dynamic_smem(k_moe_experts<FG, FD, NT>, Smem<NT>::kTotal, configured);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(device_info().sm_count));
    cfg.blockDim = dim3(kStreamThreads);
    cfg.dynamicSmemBytes = Smem<NT>::kTotal;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeCooperative;  // the grid barrier needs every block resident
    attr[0].val.cooperative = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_moe_experts<FG, FD, NT>, p);
}

template <class FG, class FD, int NT, class View>
cudaError_t launch_both(const MoeCall& c, const View& gate, const View& up, const View& down, cudaStream_t stream) {
    const MoeWorkspace ws = carve(c.workspace, c.inter, static_cast<int64_t>(c.m) * c.top_k, FD::kPair);
    const RouterParams r{static_cast<const uint16_t*>(c.router), static_cast<const uint16_t*>(c.x), c.experts, c.hidden, c.m,
                         c.top_k, c.softmax_all, ws};
    // few tokens: a cluster each; more: several tokens share a pass over the
    // router's weights, so that the clusters still fit the SMs at once
    cudaError_t e = c.m <= 16 ? launch_router<1>(r, stream) : (c.m <= 32 ? launch_router<2>(r, stream) : launch_router<4>(r, stream));
    if (e != cudaSuccess) return e;
    const ExpertParams<FG> p{FG::make(gate), FG::make(up), FD::make(down), static_cast<const uint16_t*>(c.x),
                            static_cast<uint16_t*>(c.y), c.experts, c.hidden, c.inter, c.m, c.top_k, ws, device_status_ptr()};
    return launch_experts<FG, FD, NT>(p, stream);
}

template <class FG, class FD, class View>
cudaError_t launch_moe_any(const MoeCall& c, const View& gate, const View& up, const View& down, cudaStream_t stream) {
    if (c.m <= 8) return launch_both<FG, FD, 1>(c, gate, up, down, stream);
    // Two column tiles where experts have up to 8 tokens on average: fewer registers,
    // and the few experts with more than 16 are streamed again.
    if (c.m <= 16 || c.m * c.top_k <= 8 * c.experts) return launch_both<FG, FD, 2>(c, gate, up, down, stream);
    return launch_both<FG, FD, 4>(c, gate, up, down, stream);
}

}  // namespace

size_t moe_workspace_bytes(int64_t inter, int64_t slots) {
    return static_cast<size_t>(256 + 3 * align256(slots * 4) + raw_bytes(inter, slots) + align256(slots * inter * 2));
}

cudaError_t launch_moe(const MoeCall& c, const WeightView& gate, const WeightView& up, const WeightView& down,
                       cudaStream_t stream) {
    return launch_moe_any<Q8Fmt, Q8Fmt>(c, gate, up, down, stream);
}

cudaError_t launch_mx4_moe(const MoeCall& c, const Mx4View& gate, const Mx4View& up, const Mx4View& down,
                           cudaStream_t stream) {
    // Up to four tokens fit a column tile with both parts of h, which needs no second
    // barrier and no pass over h in between: 24.9 against 26.6 us at one token (8 of 64
    // experts of 2048 x 1024), 47.2 against 47.3 at four; at eight 72 against 63.
    if (c.m <= 4) return launch_both<Mx4HalfFmt, Mx4Fmt, 1>(c, gate, up, down, stream);
    return launch_moe_any<Mx4HalfFmt, Mx4HalfFmt>(c, gate, up, down, stream);
}

}  // namespace mlxq
