// logprobs.cu -- log probability, entropy and top alternatives of rows of
// logits, in one pass over them.
//
// With a reference m near the maximum, d = (z - m) log2(e), S = sum 2^d and T =
// sum d 2^d: log p_t = (z_t - m) - ln S and the entropy is ln S - ln 2 T / S.
// The bytes of the logits bound it; the exponential (16 lanes a clock and SM)
// is next at bf16, so the other work of an element is kept to paired fp32
// instructions.
//
// The logits come in by bulk copies through a ring in shared memory, so that a
// thread spends no instructions on addresses and no registers on prefetches.
// A row is cut into C pieces, one CTA each, and the C CTAs are one
// thread-block cluster: the others leave their sums and candidates in the
// leader's shared memory, so no workspace, no counters and no second launch
// are needed.
//
// 128 rows of 248320 fp32 logits: 24.8 us, 5.1 TB/s; 144 rows of 262144 bf16
// logits: 17.4 us (4.3 TB/s), 24.6 with one alternative, 28.9 with twenty
// (the bound on the K-th and the ranking at the end are chains of barriers that
// two CTAs an SM cannot hide); 4 rows with five alternatives: 8.0 us, all
// latency.
#include "logprobs.cuh"

#include <cooperative_groups.h>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace mtp {

namespace {

constexpr int kLpThreads = 512, kLpWarps = kLpThreads / 32;
constexpr int kLpRing = 8 * kLpThreads;           // 16-byte vectors in shared memory: 64 KB; two CTAs share an SM
constexpr int kLpStagesMax = 4;
constexpr int kLpCap = 4096;                      // candidates of a piece (a first slab of ties fits: 512 threads x 8)
constexpr int kLpMaxC = 16;                       // pieces of a row
constexpr float kL2E = 1.44269504f, kLn2 = 0.693147181f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// the largest 64-bit key of a warp, by its halves
__device__ __forceinline__ unsigned long long warp_max_u32x2(unsigned long long v) {
    const unsigned hi = __reduce_max_sync(0xffffffffu, (unsigned)(v >> 32));
    const unsigned lo = __reduce_max_sync(0xffffffffu, (unsigned)(v >> 32) == hi ? (unsigned)v : 0u);
    return (unsigned long long)hi << 32 | lo;
}
// wait of at most ns (a copy takes a few microseconds); after one of the CTA gave
// up every other does too
__device__ __forceinline__ bool mbar_wait_bounded(unsigned long long* bar, unsigned parity, volatile int* lost, unsigned long long ns) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (*lost) return false;
        if (global_ns() - t0 > ns) {
            *lost = 1;
            return false;
        }
    }
    return true;
}
// the cluster's barrier (whole warps; orders shared memory of all its CTAs)
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ float neg_inf() { return -__int_as_float(0x7F800000); }

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(uint16_t x) { return bf16_to_f32(x); }
template <typename T> struct Vec;
template <> struct Vec<uint16_t> {
    static constexpr int n = 8;
    static __device__ __forceinline__ float get(const uint4& v, int i) {
        const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
        return i & 1 ? bf16_hi(w) : bf16_lo(w);
    }
};
template <> struct Vec<float> {
    static constexpr int n = 4;
    static __device__ __forceinline__ float get(const uint4& v, int i) {
        return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
    }
};
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {   // a NaN loses
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// largest of a 16-byte vector, NaN left out (NaN if there is nothing else)
__device__ __forceinline__ float vec_max(const uint4& v, uint16_t) {
    const uint32_t m = max_bf16x2(max_bf16x2(v.x, v.y), max_bf16x2(v.z, v.w));
    return fmaxf(bf16_lo(m), bf16_hi(m));
}
__device__ __forceinline__ float vec_max(const uint4& v, float) {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
}

// two fp32 values in a register pair
__device__ __forceinline__ unsigned long long pair(float a, float b) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void split(unsigned long long v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Sums of one thread relative to its own reference m (a logit): the maximum of
// its first block, moved only when a value is more than 27 above it.
struct Sums { float m, S, T; };

__device__ __forceinline__ void move_ref(Sums& s, float m) {
    const float d = (s.m - m) * kL2E, f = ex2(d);
    s.T = f == 0.f ? 0.f : f * fmaf(s.S, d, s.T);
    s.S = f == 0.f ? 0.f : f * s.S;
    s.m = m;
}
// one value, any value: -inf and NaN add nothing
__device__ __forceinline__ void add_one(Sums& s, float z) {
    if (!(z > neg_inf())) return;
    const float d = (z - s.m) * kL2E, e = ex2(d);
    if (e == 0.f) return;
    s.S += e;
    s.T = fmaf(e, d, s.T);
}
// A block's values far below the reference add nothing: they are lifted to 200
// below it (e^-200 is 0 in fp32), which also takes -inf and NaN out of the
// products.  Next to a reference so large that a bf16 step there is more than
// that, to 1/64 of it below.
__device__ __forceinline__ float lifted(float m) { return m - fmaxf(200.f, fabsf(m) * (1.f / 64.f)); }
// Two logits; nm: twice -m log2(e) as rounded, S2, T2: the block's sums of even
// and odd elements (what nm's rounding left out is put back for the block).
__device__ __forceinline__ void add_pair(float a, float b, unsigned long long nm, unsigned long long& S2, unsigned long long& T2) {
    const unsigned long long d = fma2(pair(a, b), pair(kL2E, kL2E), nm);
    float d0, d1;
    split(d, d0, d1);
    const unsigned long long e = pair(ex2(d0), ex2(d1));
    S2 = add2(S2, e);
    T2 = fma2(e, d, T2);
}
__device__ __forceinline__ void add_vec(const uint4& v, float lo, unsigned long long nm, unsigned long long& S2,
                                        unsigned long long& T2, uint16_t) {
    uint32_t l;
    asm("cvt.rn.bf16x2.f32 %0, %1, %1;" : "=r"(l) : "f"(lo));
    const uint32_t w[4] = {max_bf16x2(v.x, l), max_bf16x2(v.y, l), max_bf16x2(v.z, l), max_bf16x2(v.w, l)};
#pragma unroll
    for (int i = 0; i < 4; ++i) add_pair(bf16_lo(w[i]), bf16_hi(w[i]), nm, S2, T2);
}
__device__ __forceinline__ void add_vec(const uint4& v, float lo, unsigned long long nm, unsigned long long& S2,
                                        unsigned long long& T2, float) {
    add_pair(fmaxf(__uint_as_float(v.x), lo), fmaxf(__uint_as_float(v.y), lo), nm, S2, T2);
    add_pair(fmaxf(__uint_as_float(v.z), lo), fmaxf(__uint_as_float(v.w), lo), nm, S2, T2);
}

struct LpShared {
    uint4 ring[kLpRing];
    unsigned long long buf[kLpCap];           // candidates, in no order
    unsigned long long sel[kLpThreads];       // those still above the bound at the end
    unsigned long long top[MTP_MAX_TOP];      // the K best of select_top, descending
    unsigned long long wkey[64];              // the largest thread maxima of the warps
    unsigned long long full[kLpStagesMax], empty[kLpStagesMax];
    unsigned long long bound;
    Sums wsum[kLpWarps];
    int count, nsel;                          // candidates; entries of sel
    volatile int lost;                        // a wait gave up
    // the leader's: what the pieces' CTAs leave here
    unsigned long long tops[kLpMaxC * MTP_MAX_TOP];   // [C][K], descending
    Sums pieces[kLpMaxC];
    int piece_lost[kLpMaxC];
    float m, ls;                              // the row's reference, and ln of its sum
    int nmerge;                               // entries of buf that the leader ranks
};

// The code below a block's sums runs a few times a CTA, and what it costs is
// mostly the fetching of its instructions: it is kept in functions that the
// several places share.

// The K largest of n <= 512 distinct keys into out[], descending: every key
// counts the larger ones, with as many threads as there are.  (Barriers are
// the caller's.)
__device__ __noinline__ void rank_keys(const unsigned long long* key, int n, int K, unsigned long long* out) {
    int glog = 0;
    while (glog < 5 && n << (glog + 1) <= kLpThreads) ++glog;
    const int g = 1 << glog, which = (int)threadIdx.x >> glog;
    const unsigned long long mine = which < n ? key[which] : ~0ull;
    int r = 0;
#pragma unroll 4
    for (int i = (int)threadIdx.x & (g - 1); i < n; i += g) r += key[i] > mine;
#pragma unroll 1
    for (int o = g >> 1; o > 0; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
    if (which < n && r < K) out[r] = mine;
}
// the K-th largest of n <= 64 distinct keys in shared memory, by one warp (0 is
// no key; 0 if there are fewer)
__device__ __noinline__ unsigned long long kth_of(const unsigned long long* keys, int n, int K) {
    const int lane = threadIdx.x & 31;
    const unsigned long long a = lane < n ? keys[lane] : 0ull, b = lane + 32 < n ? keys[lane + 32] : 0ull;
    int ca = 0, cb = 0;
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
        const unsigned long long x = keys[i];
        ca += x > a;
        cb += x > b;
    }
    const bool ha = a != 0ull && ca == K - 1, hb = b != 0ull && cb == K - 1;
    const unsigned hit = __ballot_sync(0xffffffffu, ha || hb);
    return hit ? __shfl_sync(0xffffffffu, ha ? a : b, __ffs(hit) - 1) : 0ull;
}
// A key that K of the CTA's elements are at or above (0: not known): the K-th of
// the largest few `best` of each of the first W warps, one element of each thread (0: none).
__device__ __noinline__ unsigned long long bound_of(LpShared& sh, unsigned long long best, int W, int K) {
    const int lane = threadIdx.x & 31, warp = (int)threadIdx.x >> 5;
    const int R = (3 * K / 2 + W) / W, n = R * W;   // half as many again as K, 64 in all at most
    if (warp < W) {
#pragma unroll 1
        for (int r = 0; r < R; ++r) {
            const unsigned long long w = warp_max_u32x2(best);
            if (lane == 0) sh.wkey[r * W + warp] = w;
            if (best == w) best = 0ull;
        }
    }
    __syncthreads();
    if (warp == 0) {
        const unsigned long long b = kth_of(sh.wkey, n, K);
        if (lane == 0) sh.bound = b;
    }
    __syncthreads();
    return sh.bound;
}
// sums of a warp's lanes (m = -inf: none), relative to the largest reference
__device__ __noinline__ Sums join_warp(Sums w) {
    const float M = warp_max(w.m);
    if (M > neg_inf()) {
        if (w.m > neg_inf()) move_ref(w, M);
        else w = {M, 0.f, 0.f};
    }
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) {
        w.S += __shfl_xor_sync(0xffffffffu, w.S, o);
        w.T += __shfl_xor_sync(0xffffffffu, w.T, o);
    }
    w.m = M;
    return w;
}

// the K largest of buf[0, n) into top[], descending (0: none)
__device__ __noinline__ void select_top(LpShared& sh, int n, int K) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned long long mine[kLpCap / kLpThreads];
#pragma unroll
    for (int i = 0; i < kLpCap / kLpThreads; ++i) mine[i] = tid + i * kLpThreads < n ? sh.buf[tid + i * kLpThreads] : 0ull;
    for (int k = 0; k < K; ++k) {
        unsigned long long m = 0ull;
#pragma unroll
        for (int i = 0; i < kLpCap / kLpThreads; ++i) m = mine[i] > m ? mine[i] : m;
        m = warp_max_u64(m);
        __syncthreads();
        if (lane == 0) sh.wkey[warp] = m;
        __syncthreads();
        for (int w = 0; w < kLpWarps; ++w) m = sh.wkey[w] > m ? sh.wkey[w] : m;
#pragma unroll
        for (int i = 0; i < kLpCap / kLpThreads; ++i)
            if (mine[i] == m) mine[i] = 0ull;   // keys are distinct: they hold the index
        if (tid == 0) sh.top[k] = m;
    }
    __syncthreads();
}

// A piece whose candidates overflowed (ascending rows): its elements again,
// 512 at a time, keeping the K best whenever the buffer is nearly full.
template <typename T>
__device__ __noinline__ void select_slowly(LpShared& sh, const T* rowp, long long e0, long long e1, int K) {
    const int tid = threadIdx.x;
    __syncthreads();
    if (tid == 0) sh.count = 0;
    __syncthreads();
    unsigned long long kth = 0ull;
    for (long long e = e0; e < e1; e += kLpThreads) {
        if (sh.count > kLpCap - kLpThreads) {   // nobody adds before the barrier below
            select_top(sh, sh.count, K);
            if (tid < K) sh.buf[tid] = sh.top[tid];
            kth = sh.top[K - 1];
            if (tid == 0) sh.count = K;
        }
        __syncthreads();
        const float z = e + tid < e1 ? ld_elem<T>(rowp, e + tid) : neg_inf();
        const unsigned long long key = pack_argmax(z, (uint32_t)(e + tid));
        if (z > neg_inf() && key > kth) sh.buf[atomicAdd(&sh.count, 1)] = key;
        __syncthreads();
    }
}

__device__ __forceinline__ float key_value(unsigned long long key) {
    const uint32_t u = (uint32_t)(key >> 32);
    return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kLpThreads, 2) logprob_kernel(const __grid_constant__ LogprobArgs a) {
    extern __shared__ __align__(128) unsigned char smem_raw[];
    LpShared& sh = *reinterpret_cast<LpShared*>(smem_raw);
    // 16-byte vectors of a block that a thread takes, all of a block's, blocks in shared memory
    constexpr int kLpVec = VEC, kLpBlock = kLpThreads * VEC, kLpStages = kLpRing / kLpBlock;
    static_assert(kLpStages <= kLpStagesMax, "barriers");
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const long long row = blockIdx.x / C;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long tok = -1;
    if (a.tokens) {
        tok = a.tokens[row];
        if (tok < 0 || tok >= a.V) return;   // the whole cluster: nothing of the row is read or written
    }
    constexpr int EPV = Vec<T>::n;
    const T* rowp = reinterpret_cast<const T*>(a.logits) + row * a.stride;
    // the row in 16-byte vectors from the boundary at or before its start:
    // vector v holds elements [v * EPV - h, v * EPV - h + EPV); this piece's
    // whole vectors are [vs, ve), a row's ends that fill none are `loose`
    const int h = (int)((reinterpret_cast<uintptr_t>(rowp) & 15) / sizeof(T));
    const long long nv = (a.V + h + EPV - 1) / EPV, per = (nv + C - 1) / C;
    const long long v0 = per * rank < nv ? per * rank : nv, v1 = v0 + per < nv ? v0 + per : nv;
    const long long whole = (a.V + h) / EPV;
    const long long vs = h > 0 && v0 == 0 ? 1 : v0, ve = whole < v1 ? whole : v1;
    const int nvec = ve > vs ? (int)(ve - vs) : 0, blocks = (nvec + kLpBlock - 1) / kLpBlock;
    const T* first = rowp - h + vs * EPV;
    auto fetch = [&](int blk) {   // one thread
        const int n = nvec - blk * kLpBlock < kLpBlock ? nvec - blk * kLpBlock : kLpBlock;
        unsigned long long* bar = &sh.full[blk % kLpStages];
        mbar_arrive_expect_tx(bar, (unsigned)n * 16u);
        bulk_g2s(sh.ring + blk % kLpStages * kLpBlock, first + (long long)blk * kLpBlock * EPV, (unsigned)n * 16u, bar);
    };
    if (tid == 0) {
        for (int i = 0; i < kLpStages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], kLpWarps);
        }
        mbar_fence_init();
        for (int i = 0; i < kLpStages && i < blocks; ++i) fetch(i);
        sh.count = 0;
        sh.nsel = 0;
        sh.nmerge = 0;
        sh.lost = 0;
    }
    if (C > 1) cluster_arrive_relaxed();   // waited for before the leader's memory is written: it has started by then
    float zt = neg_inf();
    if (tid == 0 && rank == 0 && tok >= 0) zt = ld_elem<T>(rowp, tok);
    // a loose element of this thread
    float loose = neg_inf();
    long long loose_at = 0;
    {
        const int head = h > 0 && v0 == 0 ? (EPV - h < a.V ? EPV - h : (int)a.V) : 0;
        const int tail = v1 == nv && v0 < nv && whole < nv && !(head && whole == 0) ? (int)(a.V + h - whole * EPV) : 0;
        if (tid < head) loose_at = tid;
        else if (tid < head + tail) loose_at = whole * EPV - h + (tid - head);
        if (tid < head + tail) loose = ld_elem<T>(rowp, loose_at);
    }
    __syncthreads();
    Sums s = {neg_inf(), 0.f, 0.f};
    float lo = 0.f, nm1 = 0.f, left = 0.f, f = 1.f;   // of the reference: what far values are lifted to, -m log2(e),
                                                      // what its rounding left out, 2^-that
    auto refer = [&](float m) {
        if (s.m > neg_inf()) move_ref(s, m);
        s.m = m;
        lo = lifted(m);
        nm1 = -(m * kL2E);
        left = fmaf(m, kL2E, nm1);
        f = ex2(-left);
    };
    unsigned long long bound = 0ull;          // K keys of the piece are at or above it
    float tau = neg_inf();                    // its value
    float run = neg_inf();                    // this thread's largest element so far,
    uint32_t run_at = 0u;                     // and the last index that it can have (not above its own key)
    int check = 0;                            // the block at which the bound is next taken
    const int warps = nvec < kLpThreads ? (nvec + 31) / 32 : kLpWarps;   // that hold elements
    bool lost = false;                        // a wait of this thread gave up
    int fetched = blocks < kLpStages ? blocks : kLpStages;   // (thread 0)
    for (int it = 0; it < blocks; ++it) {
        const int stage = it % kLpStages;
        lost = !mbar_wait_bounded(&sh.full[stage], (unsigned)(it / kLpStages) & 1u, &sh.lost, a.timeout_ns) || lost;
        if (tid == 0 && !lost && it > 0 && it - 1 + kLpStages < blocks) {
            // refill the stage before this one, which the other warps leave about now
            const int prev = (it - 1) % kLpStages;
            lost = !mbar_wait_bounded(&sh.empty[prev], (unsigned)((it - 1) / kLpStages) & 1u, &sh.lost, a.timeout_ns);
            if (!lost) {
                fence_proxy_async_smem();
                fetch(it - 1 + kLpStages);
                ++fetched;
            }
        }
        const int n = nvec - it * kLpBlock;
        uint4 cur[kLpVec];
        float vm[kLpVec], bm = neg_inf();
#pragma unroll
        for (int k = 0; k < kLpVec; ++k) {
            const uint32_t none = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;   // -inf
            cur[k] = k * kLpThreads + tid < n ? sh.ring[stage * kLpBlock + k * kLpThreads + tid] : make_uint4(none, none, none, none);
        }
#pragma unroll
        for (int k = 0; k < kLpVec; ++k) {
            vm[k] = vec_max(cur[k], T());
            bm = fmaxf(bm, vm[k]);
        }
        if (bm > neg_inf()) {
            if (!(s.m > neg_inf()) || bm > s.m + 27.f) refer(bm);
            if (fabsf(s.m) < 1e5f) {
                const unsigned long long nm = pair(nm1, nm1);
                unsigned long long S2 = 0ull, T2 = 0ull;
#pragma unroll
                for (int k = 0; k < kLpVec; ++k) add_vec(cur[k], lo, nm, S2, T2, T());
                float x, y, u, v;
                split(S2, x, y);
                split(T2, u, v);
                x += y;
                s.S = fmaf(f, x, s.S);
                s.T = fmaf(f, fmaf(-left, x, u + v), s.T);
            } else {   // a reference whose products round by whole bits (masks of the type's lowest value), an infinity
#pragma unroll 1
                for (int i = 0; i < kLpVec * EPV; ++i) {
                    const int v = i / EPV * kLpThreads + tid;
                    if (v < n) add_one(s, to_float(reinterpret_cast<const T*>(sh.ring + stage * kLpBlock)[v * EPV + i % EPV]));
                }
            }
        }
        if (a.K > 0) {
            // Candidates: the keys at or above a lower bound of the K-th.
            const long long at = (vs + (long long)it * kLpBlock) * EPV - h;   // element 0 of the block
            if (bm > run) {
                int k = 0;
#pragma unroll
                for (int i = VEC - 1; i >= 0; --i)
                    if (vm[i] == bm) k = i;
                run = bm;
                run_at = (uint32_t)(at + (k * kLpThreads + tid) * EPV + EPV - 1);
            }
            // At blocks 0, 3, 12, 39, ..: the K best mostly lie in different
            // threads.
            if (it == check) {
                bound = bound_of(sh, run > neg_inf() ? pack_argmax(run, run_at) : 0ull, warps, a.K);
                tau = bound ? key_value(bound) : neg_inf();
                check = 3 * check + 3;
            }
            int mask = 0;   // this lane's vectors that hold a candidate
#pragma unroll
            for (int k = 0; k < kLpVec; ++k) mask |= vm[k] >= tau && vm[k] > neg_inf() ? 1 << k : 0;
#pragma unroll 1
            while (__any_sync(0xffffffffu, mask != 0)) {
                const int v = (__ffs(mask) - 1) * kLpThreads + tid;
                if (mask) {
                    const uint4 x = sh.ring[stage * kLpBlock + v];
#pragma unroll
                    for (int i = 0; i < EPV; ++i) {
                        const float z = Vec<T>::get(x, i);
                        if (z >= tau && z > neg_inf()) {
                            const unsigned long long key = pack_argmax(z, (uint32_t)(at + v * EPV + i));
                            const int pos = key >= bound ? atomicAdd(&sh.count, 1) : kLpCap;
                            if (pos < kLpCap) sh.buf[pos] = key;
                        }
                    }
                }
                mask &= mask - 1;
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[stage]);
    }
    if (loose > neg_inf()) {
        if (!(s.m > neg_inf()) || loose > s.m + 27.f) refer(loose);
        add_one(s, loose);
        const unsigned long long key = pack_argmax(loose, (uint32_t)loose_at);
        if (a.K > 0 && key >= bound) {
            const int pos = atomicAdd(&sh.count, 1);
            if (pos < kLpCap) sh.buf[pos] = key;
        }
    }
    if (tid == 0 && lost) {   // gave up: the copies in flight end before the CTA does
        const unsigned long long t0 = global_ns();
        for (int i = fetched > kLpStages ? fetched - kLpStages : 0; i < fetched; ++i)
            while (!mbar_try_wait(&sh.full[i % kLpStages], (unsigned)(i / kLpStages) & 1u) && global_ns() - t0 < a.timeout_ns) {}
    }
    // the piece's sums
    s = join_warp(s);
    if (lane == 0) sh.wsum[warp] = s;
    __syncthreads();
    if (warp == 0) {
        s = join_warp(lane < kLpWarps ? sh.wsum[lane] : Sums{neg_inf(), 0.f, 0.f});
        if (C > 1) cluster_wait();
        if (lane == 0) {
            *cluster.map_shared_rank(&sh.pieces[rank], 0) = s;
            *cluster.map_shared_rank(&sh.piece_lost[rank], 0) = sh.lost;
        }
    } else if (C > 1) {
        cluster_wait();
    }
    if (a.K > 0) {
        int n = sh.count;
        if (n > kLpCap) {
            const long long e0 = v0 * EPV - h, e1 = v1 * EPV - h;
            select_slowly<T>(sh, rowp, e0 > 0 ? e0 : 0, e1 < a.V ? e1 : a.V, a.K);
            n = sh.count;
        }
        const unsigned long long* from = sh.buf;
        if (n > kLpThreads) {   // a bound from the candidates themselves: every thread's largest of its share
            unsigned long long best = 0ull;
            for (int i = tid; i < n; i += kLpThreads) best = sh.buf[i] > best ? sh.buf[i] : best;
            const unsigned long long b = bound_of(sh, best, kLpWarps, a.K);
            bound = b > bound ? b : bound;
            for (int i = tid; i < n; i += kLpThreads) {
                const unsigned long long key = sh.buf[i];
                if (key >= bound) {   // (what is below it by now cannot be among the K)
                    const int pos = atomicAdd(&sh.nsel, 1);
                    if (pos < kLpThreads) sh.sel[pos] = key;
                }
            }
            __syncthreads();
            from = sh.sel;
        }
        const int m = n > kLpThreads ? sh.nsel : n;
        unsigned long long* out = cluster.map_shared_rank(sh.tops, 0) + rank * a.K;
        if (m <= kLpThreads) {
            rank_keys(from, m, a.K, out);
            if (tid >= m && tid < a.K) out[tid] = 0ull;
        } else {
            select_top(sh, n, a.K);
            if (tid < a.K) out[tid] = sh.top[tid];
        }
    }
    if (C > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (rank != 0) return;
    if (warp == 0) {
        const Sums w = join_warp(lane < C ? sh.pieces[lane] : Sums{neg_inf(), 0.f, 0.f});
        // a piece whose copies never came: no answer rather than a wrong one
        const bool none = __any_sync(0xffffffffu, lane < C && sh.piece_lost[lane] != 0);
        if (lane == 0) {
            const float ls = none ? __uint_as_float(0x7FC00000u) : logf(w.S);
            sh.lost = none;
            sh.m = w.m;
            sh.ls = ls;
            if (a.logprob) a.logprob[row] = ((zt == zt ? zt : neg_inf()) - w.m) - ls;
            if (a.entropy) a.entropy[row] = ls - kLn2 * (w.T / w.S);
        }
    }
    if (a.K > 0) {
        int real = a.K;
        const unsigned long long* best = sh.tops;   // one piece: its own
        if (C > 1) {
            // the K-th of the pieces' first few bounds the K-th of all, so most
            // are dropped before the ranking
            const int n = C * a.K;   // at most 16 pieces x 32 keys: one a thread
            const unsigned long long mine = tid < n ? sh.tops[tid] : 0ull;
            const int p = lane & (C - 1), q = lane / C;   // C is a power of two
            if (warp == 0) {
                sh.wkey[lane] = q < a.K ? sh.tops[p * a.K + q] : 0ull;
                __syncwarp();
                const unsigned long long b = kth_of(sh.wkey, 32, a.K);
                if (lane == 0) sh.bound = b;
            }
            __syncthreads();
            if (mine != 0ull && mine >= sh.bound) sh.buf[atomicAdd(&sh.nmerge, 1)] = mine;
            __syncthreads();
            real = sh.nmerge;
            rank_keys(sh.buf, real, a.K, sh.sel);
            best = sh.sel;
        }
        __syncthreads();
        if (tid < a.K) {
            const unsigned long long key = tid < real && !sh.lost ? best[tid] : 0ull;   // 0: fewer logits above -inf than K
            if (a.top_ids) a.top_ids[row * a.K + tid] = key ? (int32_t)unpack_index(key) : -1;
            if (a.top_logprobs) a.top_logprobs[row * a.K + tid] = key ? (key_value(key) - sh.m) - sh.ls : sh.lost ? sh.ls : neg_inf();
        }
    }
}

constexpr int kMaxDev = 64;
template <typename T, int VEC>
cudaError_t launch(const LogprobArgs& a, int sms, cudaStream_t s) {
    static bool ready[kMaxDev] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDev || !ready[dev]) {   // clusters of 16 are opt-in
        e = cudaFuncSetAttribute(logprob_kernel<T, VEC>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        e = cudaFuncSetAttribute(logprob_kernel<T, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(LpShared));
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < kMaxDev) ready[dev] = true;
    }
    // Pieces a row: the fewest waves of bytes (an SM's share of the bandwidth is
    // about 45 bytes a ns, which takes two CTAs), against some 2500 ns that each
    // wave of two CTAs an SM costs in first loads, joins and cluster barriers;
    // none below 16 KB.
    int C = 1;
    double best = 1e30;
    for (int c = 1; c <= kLpMaxC; c *= 2) {
        if (c > 1 && a.V / c < 4ll * kLpThreads * Vec<T>::n / 2) break;
        const long long ctas = a.rows * c, deep = (ctas + sms - 1) / sms;
        const double rate = deep >= 2 ? 45.0 : 30.0;
        const double ns = (double)a.V * sizeof(T) / rate * (double)deep / c + 2500.0 * (double)((deep + 1) / 2);
        if (ns < best) {
            best = ns;
            C = c;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.rows * C));
    cfg.blockDim = dim3(kLpThreads);
    cfg.dynamicSmemBytes = sizeof(LpShared);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)C;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, logprob_kernel<T, VEC>, a);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs& a, int ldtype, int sms, cudaStream_t s) {
    // Blocks of 32 KB; of 16 KB for fp32 logits without alternatives (128 rows of
    // 248320: 24.1 us, 26.5 with 32 KB; with one alternative 36.1 against 34.4,
    // because the first block bounds less; 144 rows of 262144 bf16 logits without
    // alternatives 18.3 against 17.7).
    if (ldtype == MTP_DTYPE_BF16) return launch<uint16_t, 4>(a, sms, s);
    return a.K > 0 ? launch<float, 4>(a, sms, s) : launch<float, 2>(a, sms, s);
}

}  // namespace mtp
