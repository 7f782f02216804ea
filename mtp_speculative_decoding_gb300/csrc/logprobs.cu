// logprobs.cu -- log probability, entropy and top alternatives of rows of
// logits, in one pass over them.
//
// With a reference m near the maximum, d = (z - m) log2(e), S = sum 2^d and T =
// sum d 2^d: log p_t = (z_t - m) - ln S and the entropy is ln S - ln 2 T / S.  The bytes of the logits bound it; the
// exponential (16 lanes a clock and SM) is next at bf16, so the other work of
// an element is kept to paired fp32 instructions.
//
// A row is cut into C pieces, one CTA each, and the C CTAs are one
// thread-block cluster: the leader reads the others' sums and candidates
// from their shared memory, so no workspace, no counters and no second launch
// are needed.
#include "logprobs.cuh"

#include <cooperative_groups.h>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace mtp {

namespace {

constexpr int kLpThreads = 512, kLpWarps = kLpThreads / 32;
constexpr int kLpVec = 4;            // 16-byte loads a thread has in flight
constexpr int kLpCap = 2048;         // candidates of a piece
constexpr float kL2E = 1.44269504f, kLn2 = 0.693147181f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float neg_inf() { return -__int_as_float(0x7F800000); }

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
    unsigned long long buf[kLpCap];           // candidates, in no order
    unsigned long long top[MTP_MAX_TOP];      // the piece's best, descending
    unsigned long long all[16 * MTP_MAX_TOP]; // the cluster's (leader)
    unsigned long long wkey[kLpWarps];
    float wmax[kLpWarps];
    Sums wsum[kLpWarps];
    Sums piece;
    int count;
};

// the K largest of buf[0, count) into top[], descending (0: none)
__device__ void select_top(LpShared& sh, int n, int K) {
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

__device__ __forceinline__ float key_value(unsigned long long key) {
    const uint32_t u = (uint32_t)(key >> 32);
    return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads, 2) logprob_kernel(const __grid_constant__ LogprobArgs a) {
    __shared__ LpShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const long long row = blockIdx.x / C;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long tok = -1;
    if (a.tokens) {
        tok = a.tokens[row];
        if (tok < 0 || tok >= a.V) return;   // the whole cluster: nothing of the row is read or written
    }
    constexpr int EPV = Vec<T>::n, BLK = kLpThreads * kLpVec;
    const T* rowp = reinterpret_cast<const T*>(a.logits) + row * a.stride;
    float zt = neg_inf();
    if (tid == 0 && rank == 0 && tok >= 0) zt = ld_elem<T>(rowp, tok);
    // the row in 16-byte vectors from the boundary at or before its start:
    // vector v holds elements [v * EPV - h, v * EPV - h + EPV)
    const long long h = (long long)((reinterpret_cast<uintptr_t>(rowp) & 15) / sizeof(T));
    const long long nv = (a.V + h + EPV - 1) / EPV, per = (nv + C - 1) / C;
    const long long v0 = per * rank, v1 = v0 + per < nv ? v0 + per : nv;
    // vectors [vs, ve) lie inside the row as well as inside the piece: no test
    const long long vs = h && v0 == 0 ? 1 : v0, ve = (a.V + h) / EPV < v1 ? (a.V + h) / EPV : v1;
    const T* origin = rowp - h;
    auto load_edge = [&](long long v) -> uint4 {
        const long long e0 = v * EPV - h;
        if (v < v1 && e0 >= 0 && e0 + EPV <= a.V) return ld_stream16(rowp + e0);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;   // -inf
        if (v < v1)   // a row's first or last vector: element by element
            for (int i = 0; i < EPV; ++i) {
                const long long e = e0 + i;
                if (e < 0 || e >= a.V) continue;
                if (sizeof(T) == 2) {
                    const uint32_t x = reinterpret_cast<const uint16_t*>(rowp)[e];
                    const uint32_t old = i < 2 ? w[0] : i < 4 ? w[1] : i < 6 ? w[2] : w[3];
                    const uint32_t nw = i & 1 ? (old & 0xFFFFu) | (x << 16) : (old & 0xFFFF0000u) | x;
                    if (i < 2) w[0] = nw; else if (i < 4) w[1] = nw; else if (i < 6) w[2] = nw; else w[3] = nw;
                } else {
                    const uint32_t x = reinterpret_cast<const uint32_t*>(rowp)[e];
                    if (i == 0) w[0] = x; else if (i == 1) w[1] = x; else if (i == 2) w[2] = x; else w[3] = x;
                }
            }
        return make_uint4(w[0], w[1], w[2], w[3]);
    };
    if (tid == 0) sh.count = 0;
    __syncthreads();
    Sums s = {neg_inf(), 0.f, 0.f};
    float lo = 0.f, nm1 = 0.f, left = 0.f, f = 1.f;   // of the reference: what far values are lifted to, -m log2(e),
                                                      // what its rounding left out, 2^-that
    float tmax = neg_inf();                   // this thread's largest so far
    float tau = neg_inf();                    // K values at or above it lie in earlier blocks
    unsigned long long kth = 0ull;            // set once a compaction knew the K-th key
    int have = 0, seen = 0;                   // candidates before this block; when the bound was last taken from them
    auto load_block = [&](long long base, uint4 (&x)[kLpVec]) {
        if (base >= vs && base + BLK <= ve) {
            const T* p = origin + (base + tid) * EPV;
#pragma unroll
            for (int k = 0; k < kLpVec; ++k) x[k] = ld_stream16(p + k * kLpThreads * EPV);
        } else {
#pragma unroll
            for (int k = 0; k < kLpVec; ++k) x[k] = load_edge(base + k * kLpThreads + tid);
        }
    };
    uint4 cur[kLpVec], nxt[kLpVec];
    load_block(v0, cur);
    int it = 0;
    for (long long base = v0; base < v1; base += BLK, ++it) {
        const bool more = base + BLK < v1;
        if (more) load_block(base + BLK, nxt);
        float vm[kLpVec], bm = neg_inf();
#pragma unroll
        for (int k = 0; k < kLpVec; ++k) {
            vm[k] = vec_max(cur[k], T());
            bm = fmaxf(bm, vm[k]);
        }
        if (bm > neg_inf()) {
            if (!(s.m > neg_inf()) || bm > s.m + 27.f) {
                if (s.m > neg_inf()) move_ref(s, bm);
                s.m = bm;
                lo = lifted(bm);
                nm1 = -(bm * kL2E);
                left = fmaf(bm, kL2E, nm1);
                f = ex2(-left);
            }
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
#pragma unroll
                for (int k = 0; k < kLpVec; ++k)
#pragma unroll
                    for (int i = 0; i < EPV; ++i) add_one(s, Vec<T>::get(cur[k], i));
            }
        }
        if (a.K > 0) {
            auto push = [&](bool at_least) {
                if (!(at_least ? bm >= tau : bm > tau)) return;
#pragma unroll
                for (int k = 0; k < kLpVec; ++k) {
                    if (!(at_least ? vm[k] >= tau : vm[k] > tau)) continue;
#pragma unroll
                    for (int i = 0; i < EPV; ++i) {
                        const float z = Vec<T>::get(cur[k], i);
                        if ((at_least ? z >= tau : z > tau) && z > neg_inf()) {
                            const int pos = atomicAdd(&sh.count, 1);
                            if (pos < kLpCap)
                                sh.buf[pos] = pack_argmax(z, (uint32_t)((base + k * kLpThreads + tid) * EPV - h + i));
                        }
                    }
                }
            };
            if (it > 0) push(false);
            tmax = fmaxf(tmax, bm);
            // a lower bound of the K-th largest so far: every warp vouches for
            // its ceil(K / 16) largest thread maxima, the smallest of those counts
            float wm = warp_max(tmax);
            if (a.K > kLpWarps) {
                const unsigned at = __ballot_sync(0xffffffffu, tmax == wm);
                wm = warp_max(at && lane == __ffs(at) - 1 ? neg_inf() : tmax);
            }
            if (lane == 0) sh.wmax[warp] = wm;
            __syncthreads();
            float t = sh.wmax[0];
#pragma unroll
            for (int w = 1; w < kLpWarps; ++w) t = fminf(t, sh.wmax[w]);
            if (it == 0) {
                tau = t;
                push(true);
                __syncthreads();
            }
            tau = fmaxf(tau, t);
            int cnt = sh.count;
            __syncthreads();   // every thread has the count before the next block adds to it
            if (cnt > kLpCap) {
                // more than the buffer holds (long ties, ascending rows): take this
                // block again, one value per thread at a time, keeping the K best
                // whenever the buffer is nearly full
                if (tid == 0) sh.count = have;
                __syncthreads();
#pragma unroll 1
                for (int e = 0; e < kLpVec * EPV; ++e) {
                    if (sh.count > kLpCap - kLpThreads) {
                        select_top(sh, sh.count, a.K);
                        if (tid < a.K) sh.buf[tid] = sh.top[tid];
                        kth = sh.top[a.K - 1];
                        if (tid == 0) sh.count = a.K;
                    }
                    __syncthreads();
                    float z = neg_inf();
#pragma unroll
                    for (int k = 0; k < kLpVec; ++k)
#pragma unroll
                        for (int i = 0; i < EPV; ++i)
                            if (k * EPV + i == e) z = Vec<T>::get(cur[k], i);
                    const unsigned long long key =
                        pack_argmax(z, (uint32_t)((base + (e / EPV) * kLpThreads + tid) * EPV - h + e % EPV));
                    if (z > neg_inf() && key > kth) sh.buf[atomicAdd(&sh.count, 1)] = key;
                    __syncthreads();
                }
                if (kth) tau = fmaxf(tau, key_value(kth));
                cnt = sh.count;
                __syncthreads();
            } else if (more && cnt >= a.K && cnt >= seen + a.K && cnt <= kLpThreads) {
                // the K-th of the candidates themselves bounds better: every
                // candidate counts the larger ones, the K-th tells the others
                // (again once as many more have come in)
                const unsigned long long mine = tid < cnt ? sh.buf[tid] : ~0ull;
                int r = 0;
                if (tid < cnt)
                    for (int i = 0; i < cnt; ++i) r += sh.buf[i] > mine;
                if (tid < cnt && r == a.K - 1) sh.wkey[0] = mine;
                __syncthreads();
                tau = fmaxf(tau, key_value(sh.wkey[0]));
                seen = cnt;
            }
            have = cnt;
        }
        if (more)
#pragma unroll
            for (int k = 0; k < kLpVec; ++k) cur[k] = nxt[k];
    }
    // the piece's sums
    float M = warp_max(s.m);
    {
        Sums w = s;
        if (M > neg_inf()) {
            if (w.m > neg_inf()) move_ref(w, M);
            else w = {M, 0.f, 0.f};
        }
        w.S = warp_sum(w.S);
        w.T = warp_sum(w.T);
        w.m = M;
        if (lane == 0) sh.wsum[warp] = w;
    }
    __syncthreads();
    if (warp == 0) {
        Sums w = lane < kLpWarps ? sh.wsum[lane] : Sums{neg_inf(), 0.f, 0.f};
        M = warp_max(w.m);
        if (M > neg_inf()) {
            if (w.m > neg_inf()) move_ref(w, M);
            else w = {M, 0.f, 0.f};
        }
        w.S = warp_sum(w.S);
        w.T = warp_sum(w.T);
        if (lane == 0) sh.piece = {M, w.S, w.T};
    }
    if (a.K > 0) {
        const int n = sh.count;
        if (n <= kLpThreads) {   // every candidate counts the larger ones
            const unsigned long long mine = tid < n ? sh.buf[tid] : 0ull;
            if (tid < a.K) sh.top[tid] = 0ull;
            int r = 0;
            if (tid < n)
                for (int i = 0; i < n; ++i) r += sh.buf[i] > mine;
            __syncthreads();
            if (tid < n && r < a.K) sh.top[r] = mine;
        } else {
            select_top(sh, n, a.K);
        }
    }
    __syncthreads();
    if (C > 1) cluster.sync();
    if (rank == 0) {
        if (warp == 0) {
            Sums w = lane < C ? *cluster.map_shared_rank(&sh.piece, lane < C ? lane : 0) : Sums{neg_inf(), 0.f, 0.f};
            M = warp_max(w.m);
            if (M > neg_inf()) {
                if (w.m > neg_inf()) move_ref(w, M);
                else w = {M, 0.f, 0.f};
            }
            w.S = warp_sum(w.S);
            w.T = warp_sum(w.T);
            w.m = M;
            if (lane == 0) {
                sh.wsum[0] = w;
                const float ls = logf(w.S);
                if (a.logprob) a.logprob[row] = ((zt == zt ? zt : neg_inf()) - M) - ls;
                if (a.entropy) a.entropy[row] = ls - kLn2 * (w.T / w.S);
            }
        }
        if (a.K > 0) {
            const int n = C * a.K;
            unsigned long long mine = 0ull;
            if (tid < n) {
                mine = cluster.map_shared_rank(sh.top, tid / a.K)[tid % a.K];
                sh.all[tid] = mine;
            }
            __syncthreads();
            int r = 0, real = 0;
            if (tid < n)
                for (int i = 0; i < n; ++i) {
                    r += sh.all[i] > mine;
                    real += sh.all[i] != 0ull;
                }
            const float m = sh.wsum[0].m, ls = logf(sh.wsum[0].S);
            const bool put = mine != 0ull && r < a.K;
            if (put && a.top_ids) a.top_ids[row * a.K + r] = (int32_t)unpack_index(mine);
            if (put && a.top_logprobs) a.top_logprobs[row * a.K + r] = (key_value(mine) - m) - ls;
            if (tid < a.K && tid >= real) {   // fewer logits above -inf than K
                if (a.top_ids) a.top_ids[row * a.K + tid] = -1;
                if (a.top_logprobs) a.top_logprobs[row * a.K + tid] = neg_inf();
            }
        }
    }
    if (C > 1) cluster.sync();   // the leader has read this CTA's shared memory
}

constexpr int kMaxDev = 64;
template <typename T>
cudaError_t launch(const LogprobArgs& a, int sms, cudaStream_t s) {
    static bool ready[kMaxDev] = {false};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDev || !ready[dev]) {   // clusters of 16 are opt-in
        e = cudaFuncSetAttribute(logprob_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < kMaxDev) ready[dev] = true;
    }
    // Pieces a row: the fewest waves of bytes (an SM's share of the bandwidth is
    // about 45 bytes a ns), against some 2500 ns that each wave of two CTAs an SM
    // costs in first loads, joins and cluster barriers; none below half a block
    // of loads.
    int C = 1;
    double best = 1e30;
    for (int c = 1; c <= 16; c *= 2) {
        const long long ctas = a.rows * c;
        const double rate = ctas > sms ? 45.0 : 30.0;   // one CTA an SM has too few loads in flight
        const double ns = (double)a.V * sizeof(T) / rate * (double)((ctas + sms - 1) / sms) / c +
                          2500.0 * (double)((ctas + 2 * sms - 1) / (2 * sms));
        if (c > 1 && a.V / c < (long long)kLpThreads * kLpVec * Vec<T>::n / 2) break;
        if (ns < best) {
            best = ns;
            C = c;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.rows * C));
    cfg.blockDim = dim3(kLpThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)C;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, logprob_kernel<T>, a);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs& a, int ldtype, int sms, cudaStream_t s) {
    return ldtype == MTP_DTYPE_BF16 ? launch<uint16_t>(a, sms, s) : launch<float>(a, sms, s);
}

}  // namespace mtp
