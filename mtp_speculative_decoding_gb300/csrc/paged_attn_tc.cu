// paged_attn_tc.cu -- attention of a verify step's rows over the paged cache
// on tcgen05 tensor cores.
//
// The rows of one KV head (new rows x query heads of the group, 1 to a few
// hundred) are few against the positions, so the positions take the MMA's M
// side: S^T [128 positions, RT rows] = K Q^T with K's tile as it lies in the
// page (K-major), and O^T [128 dimensions, RT rows] += V^T P^T with V's tile as
// it lies in the page (its dimensions contiguous: the M-major operand).  K and
// V go from the pages to the tensor core by TMA alone; an e4m3 cache is
// multiplied as e4m3, exactly, so its bytes are the only traffic.  What would
// lose bits is split instead: against bf16, a query row and a probability into
// two bf16 parts each (2^-16); against e4m3, a query row into three e4m3 parts
// under a power of two of its own (2^-12) and a probability into three e5m2
// parts (2^-9; e5m2 for its range: a weight keeps all 9 bits down to 2^-19 of the
// largest and counts down to 2^-28).
//
// Softmax: a thread is one position of the tile and holds its RT scores.  The
// reference m of a row (the running maximum) moves only when a score exceeds
// it by more than 2^kSlack, so most tiles need no reduction at all: one vote,
// then exponentials.  A page's value scale is a power of two and joins the
// score's exponent; the sum l takes it out again.
//
// Warps 0-7: softmax and epilogue, half of the rows for each of two
// warpgroups; warp 8: TMA producer; warp 9: MMA issue.
//
// The bytes of K and V bound it where batches are large: 64 sequences x 3 rows
// over 4096 positions, e4m3, 16 heads over 4 KV heads of 256 (537 MB): 98 us
// with the merge, 5.5 TB/s (a copy's rate would take 79); the same heads over
// windows of 1024 in bf16 (193 MB): 43 us; 16 sequences x up to 5 rows over 2k
// to 32k positions, e4m3 (558 MB): 100 us, where the rows take RT = 32 and the
// issue of small MMAs (40 to 80 ns each) comes up to the bytes.  One sequence
// is a chain of latencies: 4 rows over 8192 positions 14.7 us, 1 row over 999
// 10.9 us (4 to 5 us to the first MMA: lengths, pages, TMA, the queries' norm and
// rotation; 3 us in the merge).
#include "paged_attn_tc.cuh"

namespace mtp {

namespace {

// ---- tensor-core helpers of this kernel ----
// D[tmem] (+)= A B^T with the descriptors' low words given and their high words
// fixed: the unrolled issue loops then cost two additions an MMA
template <bool F8>
__device__ __forceinline__ void umma(unsigned int d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                     uint32_t acc) {
    if (F8)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, p;\n\t}" ::"r"(d),
            "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
            "setp.ne.b32 p, %6, 0;\n\t"
            "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d),
            "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc)
            : "memory");
}
__device__ __forceinline__ void tmem_ld8(unsigned int taddr, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(unsigned int taddr, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ bool elect_one() {
    unsigned int p;
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tma_load_4d(void* dst, const void* tmap, int x, int y, int z, int w, unsigned long long* bar,
                                            unsigned long long pol) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, "
        "%4, %5}], [%6], %7;" ::"r"(smem_addr(dst)),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar)), "l"(pol)
        : "memory");
}
// Shared-memory matrix descriptors, as (low, high) words; low: address / 16 plus
// the leading offset (an address below 256 KB leaves it alone when added to).
// Tiles of 128- or 64-byte swizzled rows of ROWB bytes, 8-row groups following
// one another; lead: bytes between the ROWB-wide blocks of an M-major operand
// (0: the same block again, for rows of 64 dimensions under an M of 128 -- the
// upper half of the accumulator repeats the lower and is not read)
__host__ __device__ constexpr uint32_t desc_lead(uint32_t lead) { return (lead >> 4) << 16; }
template <int ROWB>
__host__ __device__ constexpr uint32_t desc_rows_hi() {
    return ((8 * ROWB) >> 4) | 1u << 14 | (ROWB == 128 ? 2u : 4u) << 29;
}
// P: its rows (N) are contiguous, 16 bytes of them a position, no swizzle; 8
// positions are a 128-byte core, positions follow densely, 16-byte row blocks
// are 2048 bytes apart
constexpr uint32_t kDescPHi = (2048 >> 4) | 1u << 14;
// fp32 accumulator, M x N; types 0 / 1: e4m3 / e5m2 (kind f8f6f4), 1: bf16 (kind f16)
// (mn: both operands M- / N-major)
__host__ __device__ constexpr uint32_t instr(int ta, int tb, bool mn, int M, int N) {
    return (1u << 4) | ((uint32_t)ta << 7) | ((uint32_t)tb << 10) | (mn ? 3u << 15 : 0u) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}
// 16-byte chunk `ch` of row r under the swizzle
template <int ROWB>
__device__ __forceinline__ int swz(int r, int ch) {
    return r * ROWB + ((ROWB == 128 ? ch ^ (r & 7) : ch ^ ((r >> 1) & 3)) << 4);
}
// barriers of a softmax warpgroup (id 1 + wg) and of both (id 3)
__device__ __forceinline__ bool vote_or(int wg, bool p) {
    unsigned int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %2, 0;\n\t"
        "barrier.cta.red.or.aligned.pred q, %1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(1 + wg), "r"((unsigned)p)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void wg_sync(int wg) { asm volatile("barrier.cta.sync.aligned %0, 128;" ::"r"(1 + wg) : "memory"); }
__device__ __forceinline__ void both_sync() { asm volatile("barrier.cta.sync.aligned 3, 256;" ::: "memory"); }
// N rows' sums or maxima over a warp's lanes: at each step a lane hands half of
// its rows over, so that N - 1 exchanges (and a few for N below 32) do what 5 N
// would.  Lane i ends with row i / (32 / N).
template <bool MAX, int N>
__device__ __forceinline__ float rows_reduce(const float (&x)[N], int lane) {
    auto op = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
    float v[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const float keep = lane & 16 ? x[i + N / 2] : x[i], give = lane & 16 ? x[i] : x[i + N / 2];
        v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, 16));
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        const int n = N * o / 32;   // rows that stay
        if (n > 0) {
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float keep = lane & o ? v[i + n] : v[i], give = lane & o ? v[i] : v[i + n];
                v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, o));
            }
        } else {
            v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], o));
        }
    }
    return v[0];
}
__device__ __forceinline__ float fexp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <bool E4M3, int HD, int RT>
struct Shape {
    static constexpr int ESZ = E4M3 ? 1 : 2;
    static constexpr int ROWB = HD * ESZ < 128 ? HD * ESZ : 128;   // bytes of a box row
    static constexpr int DB = HD < 128 ? HD : 128;                 // dimensions of a ring slot
    static constexpr int D = HD / DB;                              // slots of a K or V tile
    static constexpr int NBOX = DB * ESZ / ROWB;                   // boxes side by side in a slot
    static constexpr int BOXB = kTcTile * ROWB;
    static constexpr int SLOTB = NBOX * BOXB;
    static constexpr int NQ = E4M3 ? 3 : 2;                        // parts of Q
    static constexpr int QBOX = HD * ESZ / ROWB;                   // boxes of a Q row
    static constexpr int QB = NQ * QBOX * RT * ROWB;
    static constexpr int NP = E4M3 ? 3 : 2;                        // parts of P
    static constexpr int PBUF = tc_p_bufs(E4M3, HD, RT);               // tiles of P
    static constexpr int PB = NP * RT * ESZ * kTcTile;
    // The parts of an operand lie side by side in N where tensor memory has the
    // columns (one MMA instead of NQ or NP: an MMA takes about 40 ns here
    // whatever its N), and are summed when they are read; else they accumulate.
    static constexpr int SCOLS = NQ * RT;                          // scores, two tiles
    static constexpr bool ON = 2 * SCOLS + D * NP * RT <= 512;     // outputs side by side too
    static constexpr int NO = ON ? NP : 1;
    static constexpr int O0 = 2 * SCOLS, COLS0 = O0 + D * NO * RT;
    static constexpr int COLS = COLS0 <= 32 ? 32 : COLS0 <= 64 ? 64 : COLS0 <= 128 ? 128 : COLS0 <= 256 ? 256 : 512;
    static_assert(COLS0 <= 512, "tensor memory");
    static constexpr int RW = RT / 2;                              // rows of a softmax warpgroup
    // a score's exponent relative to its row's reference: at most kSlack; P
    // against e4m3 lies in e5m2's range [2^-16, 2^15] with it and 2^kBias
    static constexpr float kSlack = E4M3 ? 4.f : 8.f, kBias = E4M3 ? 11.f : 0.f;
};

// A segment's dimensions tok, tok + 128, .. where the product left a result that
// is not finite.  An attended infinity is a NaN there (the second part of its weight is
// often 0, or negative), so such a row takes its answer from the attended values
// that are not finite: one pass over the segment's values, by the thread that
// wrote the result.  Rows whose sum is a NaN stay as they are, and so does what
// overflowed without such a value.
template <int RW>
__device__ __noinline__ void infinite_values(const PagedAttnArgs* pa, Plan plan, long long x, int tok, const int* pos,
                                             const int* row, const float* inv, float* part, int rows) {
    const PagedAttnArgs& a = *pa;
    const int hd = a.hd;
    const Segment s = segment_at(a, plan, x, share_lo(plan.pre[a.B], blockIdx.x + 1, a.grid), blockIdx.x);
    constexpr int LK = 8, PER = kTcTile / LK;   // values in flight: slots of one page
#pragma unroll 1
    for (int d = tok; d < hd; d += 128) {
        float acc[RW];
        uint32_t odd = 0u, found = 0u;
#pragma unroll 1
        for (int r = 0; r < RW && r < rows; ++r) {
            const float o = part ? part[r * hd + d] : bf16_to_f32(reinterpret_cast<const uint16_t*>(a.out)[(long long)row[r] * hd + d]);
            if (o - o != 0.f && inv[r] == inv[r]) odd |= 1u << r;
        }
        if (odd == 0u) continue;
#pragma unroll 1
        for (int i = 0; i < s.n * PER; ++i) {
            const int t = tile_at(s.map, s.t0 + i / PER) * kTcTile + i % PER * LK;
            if (t >= s.len + s.n_new) continue;
            const int pg = a.c.table[(long long)s.b * a.c.max_pages + (t >> a.c.ps_log2)];
            if ((unsigned)pg >= (unsigned)a.c.n_pages) continue;
            const uint16_t* v = reinterpret_cast<const uint16_t*>(a.c.v) + pg * a.c.sp + s.g * a.c.sh +
                                (t & ((1 << a.c.ps_log2) - 1)) * a.c.st + d;
            uint16_t x[LK];
            bool any = false;
#pragma unroll
            for (int e = 0; e < LK; ++e) x[e] = v[e * a.c.st];
#pragma unroll
            for (int e = 0; e < LK; ++e) any = any || (x[e] & 0x7F80u) == 0x7F80u;
            if (!any) continue;
#pragma unroll 1
            for (int e = 0; e < LK; ++e) {
                const float val = bf16_to_f32(v[e * a.c.st]);
                if (val - val == 0.f) continue;
#pragma unroll 1
                for (int r = 0; r < RW; ++r)
                    if (odd >> r & 1u && attends(a.c, t + e, pos[r])) {
                        acc[r] = found >> r & 1u ? acc[r] + val : val;
                        found |= 1u << r;
                    }
            }
        }
#pragma unroll 1
        for (int r = 0; r < RW; ++r) {
            if (!(found >> r & 1u)) continue;
            if (part) part[r * hd + d] = acc[r];
            else reinterpret_cast<uint16_t*>(a.out)[(long long)row[r] * hd + d] = (uint16_t)pack_bf16(acc[r], 0.f);
        }
    }
}

constexpr int kTcThreads = 320;

template <bool E4M3, int HD, int RT>
__global__ void __launch_bounds__(kTcThreads, 1) paged_attn_tc_kernel(const __grid_constant__ PagedTcArgs pa) {
    using S = Shape<E4M3, HD, RT>;
    constexpr int RW = S::RW;
    const PagedAttnArgs& a = pa.a;
    extern __shared__ unsigned char raw[];
    unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int NS = pa.slots;
    unsigned char* ring = base;
    unsigned char* sQ = ring + (size_t)NS * S::SLOTB;
    unsigned char* sP = sQ + S::QB;
    float* s_hi = reinterpret_cast<float*>(sP + S::PBUF * S::PB);   // [HD/2], [HD/2]: rotation table
    float* s_lo = s_hi + HD / 2;
    float* m_ks = s_lo + HD / 2;                               // [kTcMeta][8] key scale (0: page not loaded or not used)
    float* m_vs = m_ks + kTcMeta * 8;                          // [kTcMeta][8] exponent of the value scale
    float* s_inv = m_vs + kTcMeta * 8;                         // [RT] one over the row's sum
    float* s_f = s_inv + RT;                                   // [RT] rescale factor
    float* s_c = s_f + RT;                                     // [RT] scale of the query row
    float* s_red = s_c + RT;                                   // [RT][4]: a row's sum or maximum of every warp
    int* s_pos2 = reinterpret_cast<int*>(s_red + 4 * RT);      // [2][RT] position of the row
    int* s_row2 = s_pos2 + 2 * RT;                             // [2][RT] output row
    int* s_fix2 = s_row2 + 2 * RT;                             // [2][kTcFix]
    int* m_all = s_fix2 + 2 * kTcFix;                          // [kTcMeta] every page of the tile is used
    unsigned long long* bars = reinterpret_cast<unsigned long long*>(m_all + kTcMeta);
    unsigned long long *full = bars, *empty = full + kTcSlotsMax, *meta_full = empty + kTcSlotsMax, *s_full = meta_full + kTcMeta,
                       *s_free = s_full + 2, *p_full = s_free + 2, *pv_done = p_full + 2, *q_full = pv_done + 2, *end_bar = q_full + 1;
    long long* tmp = reinterpret_cast<long long*>(end_bar + 1);
    Plan plan;
    plan.pre = tmp + kPlanTmp;
    plan.len = reinterpret_cast<int2*>(plan.pre + a.B + 1);
    __shared__ unsigned int s_tmem;
    __shared__ int s_nfix[2], s_bad;
    __shared__ volatile int s_abort;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    // one thread each: the ring's, the scales', and the ten others' counts
    if (tid < 2 * kTcSlotsMax + kTcMeta) mbar_init(bars + tid, 1);
    else if (tid < 2 * kTcSlotsMax + kTcMeta + 10) {
        const int i = tid - (2 * kTcSlotsMax + kTcMeta);   // s_full, s_free, p_full, pv_done (two each), q_full, end_bar
        mbar_init(bars + tid, i == 2 || i == 3 ? 8 : i == 4 || i == 5 || i == 8 ? 256 : 1);
    }
    mbar_fence_init();
    if (tid == 0) {
        s_nfix[0] = s_nfix[1] = 0;
        s_bad = 0;
        s_abort = 0;
    }
    if (warp == 9) {
        tmem_alloc(&s_tmem, S::COLS);
        tmem_relinquish();
    }
    if (a.rope.on)
        for (int i = tid; i < HD / 2; i += kTcThreads) {
            s_hi[i] = a.rope.hi[i];
            s_lo[i] = a.rope.lo[i];
        }
    asm volatile("griddepcontrol.wait;" ::: "memory");      // what ran before has written its rows
    const bool good = schedule<kTcThreads>(a, plan, tmp);   // meets in CTA barriers
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
    if (blockIdx.x == 0 && !good) s_bad = 1;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const long long T = plan.pre[a.B];
    const long long x0 = share_lo(T, blockIdx.x, a.grid), xe = share_lo(T, blockIdx.x + 1, a.grid);
    // bounded wait; after one gave up every other does too
    auto wait = [&](unsigned long long* bar, unsigned int parity) -> bool {
        if (mbar_try_wait(bar, parity)) return true;
        const unsigned long long t0 = global_ns();
        while (!mbar_try_wait(bar, parity)) {
            if (s_abort) return false;
            if (global_ns() - t0 > a.timeout_ns) {
                s_abort = 1;
                return false;
            }
        }
        return true;
    };
    const int ps = 1 << a.c.ps_log2, box_log2 = a.c.ps_log2 < kTcTileLog2 ? a.c.ps_log2 : kTcTileLog2, box_rows = 1 << box_log2,
              np = kTcTile >> box_log2, np_log2 = kTcTileLog2 - box_log2;

    if (warp == 8) {
        // ------------------------------------------------------------------
        // producer: K tile k, then V tile k - 1, in the order the MMAs take
        // them; lane i of a batch of 32 / np tiles holds page i % np of tile
        // i / np
        // ------------------------------------------------------------------
        const unsigned long long pol = l2_evict_first();
        unsigned int slot = 0, phase = 0, ti = 0;
        bool ok = true, bad = false;
        int4 split = make_int4(0, 0, 0, -1);
        const int per_batch = 32 >> np_log2;
        long long x = x0;
        while (x < xe && ok) {
            const Segment s = segment_at(a, plan, x, xe, blockIdx.x);
            if (s.n <= 0) break;
            const int end = s.len + s.n_new;
            const int lo = a.c.window > 0 && s.len + 1 > a.c.window ? s.len + 1 - a.c.window : 0;
            const int hi = a.c.window > 0 && end > a.c.window ? end - a.c.window : 0;
            const int sink = a.c.sink < hi ? a.c.sink : hi;
            const int* tab = a.c.table + (long long)s.b * a.c.max_pages;
            auto entry = [&](int k, int& y) -> int {   // page of this lane for tile s.t0 + k; below 0: not loaded
                y = 0;
                if (k >= s.n) return -2;
                const int p0 = tile_at(s.map, s.t0 + k) * kTcTile + ((lane & (np - 1)) << box_log2);
                y = p0 & (ps - 1);
                if (p0 >= end || (p0 + box_rows <= lo && p0 >= sink)) return -2;   // attended by no row
                const int pg = tab[p0 >> a.c.ps_log2];
                if ((unsigned)pg < (unsigned)a.c.n_pages) return pg;
                bad = true;
                return -1;
            };
            int pg = -2, y = 0, pv_pg = -2, pv_y = 0, ny = 0;
            int npg = entry(lane >> np_log2, ny);
            for (int k = 0; k <= s.n && ok; ++k) {
                int kp = -2, ky = 0;
                if (k < s.n) {
                    const int in = k & (per_batch - 1);
                    if (in == 0) {   // this batch's pages; the next one's are on their way meanwhile
                        pg = npg;
                        y = ny;
                        npg = entry(k + per_batch + (lane >> np_log2), ny);
                    }
                    kp = __shfl_sync(0xffffffffu, pg, (in << np_log2) + (lane & (np - 1)));
                    ky = __shfl_sync(0xffffffffu, y, (in << np_log2) + (lane & (np - 1)));
                }
#pragma unroll 1
                for (int which = 0; which < 2 && ok; ++which) {
                    const bool key = which == 0;
                    if (key ? k == s.n : k == 0) continue;
                    const int p = key ? kp : pv_pg, yy = key ? ky : pv_y;
                    const unsigned cnt = __popc(__ballot_sync(0xffffffffu, lane < np && p >= 0));
                    for (int d = 0; d < S::D && ok; ++d) {
                        ok = wait(empty + slot, phase ^ 1);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        if (lane == 0) mbar_arrive_expect_tx(full + slot, cnt * (unsigned)(box_rows * S::ROWB * S::NBOX));
                        __syncwarp();
                        if (lane < np && p >= 0) {
                            unsigned char* dst = ring + (size_t)slot * S::SLOTB + lane * box_rows * S::ROWB;
#pragma unroll
                            for (int nb = 0; nb < S::NBOX; ++nb)
                                tma_load_4d(dst + nb * S::BOXB, key ? &pa.tk : &pa.tv, d * S::DB + nb * (S::ROWB / S::ESZ), yy, s.g, p,
                                            full + slot, pol);
                        }
                        if (++slot == (unsigned)NS) {
                            slot = 0;
                            phase ^= 1;
                        }
                    }
                    if (key) {   // the tile's scales, while its keys are on their way
                        float ks = kp >= 0 ? 1.f : 0.f;   // 0: masked
                        if (lane < np) {
                            float vs = 0.f;
                            if (E4M3 && kp >= 0) {
                                const long long o = (long long)kp * a.c.Hkv + s.g;
                                const float kss = a.c.ks[o], vss = a.c.vs[o];
                                const bool fits = scale_ok(kss) && scale_ok(vss);   // else the page counts as absent
                                bad = bad || !fits;
                                ks = fits ? kss : 0.f;
                                vs = (float)((int)(__float_as_uint(fits ? vss : 1.f) >> 23) - 127);
                            }
                            m_ks[(ti % kTcMeta) * 8 + lane] = ks;
                            m_vs[(ti % kTcMeta) * 8 + lane] = vs;
                        }
                        const bool all = __all_sync(0xffffffffu, lane >= np || ks != 0.f);
                        if (lane == 0) m_all[ti % kTcMeta] = all;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(meta_full + ti % kTcMeta);
                        ++ti;
                    }
                }
                pv_pg = kp;
                pv_y = ky;
            }
            if (lane == 0) note_split(a, s, T, blockIdx.x, split);
            x = s.next;
        }
        if (lane == 0 && !a.by_item) a.split[blockIdx.x] = split;
        if (__any_sync(0xffffffffu, bad) && lane == 0) s_bad = 1;
        if (!ok) {   // gave up: this warp's copies in flight end before the CTA does
            const unsigned long long t0 = global_ns();
            for (int i = 0; i < NS; ++i) {
                // slot i's last fill: of this lap below the cursor, of the lap before from it on
                const unsigned int ph = i < (int)slot ? phase : phase ^ 1;
                while (!mbar_try_wait(full + i, ph) && global_ns() - t0 < a.timeout_ns) {}
            }
        }
    } else if (warp == 9) {
        // ------------------------------------------------------------------
        // MMA issue: the whole warp walks (descriptors stay in uniform
        // registers), one elected lane issues
        // ------------------------------------------------------------------
        constexpr uint32_t idS = E4M3 ? instr(0, 0, false, 128, S::SCOLS) : instr(1, 1, false, 128, S::SCOLS);
        constexpr uint32_t idO = E4M3 ? instr(0, 1, true, 128, S::NO * RT) : instr(1, 1, true, 128, S::NO * RT);
        constexpr uint32_t hiR = desc_rows_hi<S::ROWB>();
        const uint32_t q0 = (smem_addr(sQ) >> 4) + desc_lead(16), p0 = (smem_addr(sP) >> 4) + desc_lead(128), r0 = smem_addr(ring) >> 4;
        constexpr int KT = E4M3 ? 32 : 16;   // positions of an MMA over V
        unsigned int slot = 0, phase = 0, ti = 0, seg = 0;
        bool ok = true;
        auto next = [&] {
            if (++slot == (unsigned)NS) {
                slot = 0;
                phase ^= 1;
            }
        };
        auto hold = [&](unsigned long long* bar, unsigned int parity) {
            ok = __all_sync(0xffffffffu, wait(bar, parity));
            tc_fence_after();
        };
        long long x = x0;
        while (x < xe && ok) {
            const Segment s = segment_at(a, plan, x, xe, blockIdx.x);
            if (s.n <= 0) break;
            hold(q_full, seg & 1);
            ++seg;
            for (int k = 0; k <= s.n && ok; ++k) {
                if (k < s.n) {   // S^T of tile k
                    const unsigned int t = ti + k, buf = t & 1;
                    hold(s_free + buf, ((t >> 1) & 1) ^ 1);
                    for (int d = 0; d < S::D && ok; ++d) {
                        hold(full + slot, phase);
                        if (!ok) break;
                        const uint32_t al = r0 + slot * (S::SLOTB >> 4) + desc_lead(16), bl = q0 + d * (S::NBOX * S::NQ * RT * S::ROWB >> 4);
                        if (elect_one()) {
#pragma unroll
                            for (int nb = 0; nb < S::NBOX; ++nb)
#pragma unroll
                                for (int ks = 0; ks < S::ROWB / 32; ++ks)
                                    umma<E4M3>(tmem + buf * S::SCOLS, al + (nb * S::BOXB + ks * 32 >> 4), hiR,
                                               bl + (nb * S::NQ * RT * S::ROWB + ks * 32 >> 4), hiR, idS, d > 0 || nb > 0 || ks > 0);
                            umma_commit(empty + slot);
                        }
                        __syncwarp();
                        next();
                    }
                    if (ok && elect_one()) umma_commit(s_full + buf);
                    __syncwarp();
                }
                if (k > 0 && ok) {   // O^T of tile k - 1
                    const unsigned int t = ti + k - 1, buf = t & 1;
                    hold(p_full + buf, (t >> 1) & 1);
                    for (int d = 0; d < S::D && ok; ++d) {
                        hold(full + slot, phase);
                        if (!ok) break;
                        const uint32_t al = r0 + slot * (S::SLOTB >> 4) + desc_lead(S::NBOX == 2 ? S::BOXB : 0), bl = p0 + (t % S::PBUF) * (S::PB >> 4);
                        if (elect_one()) {
#pragma unroll
                            for (int ks = 0; ks < kTcTile / KT; ++ks)
#pragma unroll
                                for (int part = 0; part < S::NP / S::NO; ++part)
                                    umma<E4M3>(tmem + S::O0 + d * S::NO * RT, al + (ks * KT * S::ROWB >> 4), hiR,
                                               bl + (part * (RT * S::ESZ / 16) * 2048 + ks * KT * 16 >> 4), kDescPHi, idO,
                                               k > 1 || ks > 0 || part > 0);
                            umma_commit(empty + slot);
                        }
                        __syncwarp();
                        next();
                    }
                    if (ok && elect_one()) umma_commit(pv_done + buf);
                    __syncwarp();
                }
            }
            ti += s.n;
            x = s.next;
        }
        if (elect_one()) umma_commit(end_bar);   // whatever was issued has ended before the CTA frees its memory
        const unsigned long long t0 = global_ns();
        while (!mbar_try_wait(end_bar, 0) && global_ns() - t0 < a.timeout_ns) {}
        __syncwarp();
    } else {
        // ------------------------------------------------------------------
        // softmax and epilogue: thread = position of the tile, then dimension;
        // warpgroup wg has the rows [wg RW, wg RW + RW).
        // A wait that gave up ends the other warps' work; these go on to the
        // end with whatever is there, because they meet in barriers.
        // ------------------------------------------------------------------
        const int wg = warp >> 2, tok = tid & 127, w4 = warp & 3, rw = wg * RW;
        const uint32_t my = tmem + ((uint32_t)(w4 * 32) << 16);
        unsigned int ti = 0, g0 = 0;   // tiles and ring slots before this segment
        int par0 = 1;                  // row tables of this segment
        long long x = x0;
        Segment s = {}, nx = {};
        bool have = false;
        constexpr int U = HD / 16, RP = 256 / U;   // threads of a query row, rows of a pass
        const int qc = tid % U, qr = tid / U;
        uint4 raw0 = make_uint4(0, 0, 0, 0), raw1 = raw0;
        // this thread's unit of row r of segment nx, as loaded
        auto load_q = [&](int r, uint4& v0, uint4& v1, int& j) {
            const int at = nx.rt * RT + r;
            j = (int)udiv((unsigned)at, (unsigned)a.G);
            const uint16_t* src =
                reinterpret_cast<const uint16_t*>(a.q) + nx.b * a.sb + j * a.sm + (nx.g * a.G + at - j * a.G) * a.sh + 8 * qc;
            v0 = ld_stream16(src);
            v1 = ld_stream16(src + HD / 2);
        };
        // the segment at x, and its first rows on their way
        int raw_j = 0;
        auto open_next = [&](long long at) {
            nx = segment_at(a, plan, at, xe, blockIdx.x);
            if (qr < nx.rows) load_q(qr, raw0, raw1, raw_j);
        };
        if (x < xe) open_next(x);
        if (nx.n <= 0) x = xe;
        int4 split = make_int4(0, 0, 0, -1);
        float l[RW], m[RW], c[RW];
        // A turn prepares the next segment's queries (its scores' MMAs start
        // on them), writes this segment's output, and goes through the next
        // one's tiles.
        for (;;) {
            const bool more = x < xe;
            if (more) {
                const int pn = par0 ^ 1;
                const int r0 = nx.rt * RT;
                // ---- queries: norm, rotation, scale, parts ----
                {
                    const int c = qc;
#pragma unroll 1
                    for (int rb = 0; rb < RT; rb += RP) {
                        const int r = rb + qr;
                        if (RP > RT && r >= RT) break;   // whole warps
                        const bool in = r < nx.rows;
                        float p[8], q[8];
                        bool fin = true;
                        float amax = 0.f;
                        if (__any_sync(0xffffffffu, in)) {
                            int j = raw_j;
                            if (rb > 0) {
                                j = 0;
                                if (in) load_q(r, raw0, raw1, j);
                            }
                            open_unit(raw0, p);
                            open_unit(raw1, q);
                            float cs[8], sn[8];
                            if (a.rope.on) unit_angles<true>((long long)nx.len + j, s_hi + 8 * c, s_lo + 8 * c, cs, sn);
                            if (a.q_norm) unit_norm(p, q, a.q_norm, c, HD, a.eps);
                            if (a.rope.on) unit_rotate(p, q, cs, sn);
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                p[e] = in ? p[e] * a.scale : 0.f;
                                q[e] = in ? q[e] * a.scale : 0.f;
                                amax = fmaxf(amax, fmaxf(fabsf(p[e]), fabsf(q[e])));
                                fin = fin && p[e] - p[e] == 0.f && q[e] - q[e] == 0.f;
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e) p[e] = q[e] = 0.f;
                        }
                        if (E4M3) {
                            for (int o = U / 2; o > 0; o >>= 1) {
                                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                                fin = __shfl_xor_sync(0xffffffffu, (int)fin, o) && fin;
                            }
                            int k = (int)(__float_as_uint(amax) >> 23) - 127 - 7;   // the largest over 2^k in [128, 256)
                            if (amax == 0.f || k < -100) k = -100;
                            if (k > 100) k = 100;
                            const float inv = __uint_as_float((uint32_t)(127 - k) << 23);
                            if (c == 0) s_c[r] = fin ? __uint_as_float((uint32_t)(127 + k) << 23) : __uint_as_float(0x7FC00000u);
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                p[e] *= inv;
                                q[e] *= inv;
                            }
#pragma unroll
                            for (int part = 0; part < 3; ++part) {
                                uint32_t w[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    float* v = i < 2 ? p + 4 * i : q + 4 * (i - 2);
                                    uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE, __NV_E4M3);
                                    uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2], v[3]), __NV_SATFINITE, __NV_E4M3);
                                    w[i] = lo | (hi << 16);
                                    const float2 a0 = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)lo, __NV_E4M3)));
                                    const float2 a1 = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)hi, __NV_E4M3)));
                                    v[0] -= a0.x;
                                    v[1] -= a0.y;
                                    v[2] -= a1.x;
                                    v[3] -= a1.y;
                                }
#pragma unroll
                                for (int half = 0; half < 2; ++half) {
                                    const int byte = half * (HD / 2) + 8 * c, box = byte / S::ROWB, in_row = byte % S::ROWB;
                                    unsigned char* d = sQ + (box * S::NQ + part) * RT * S::ROWB + swz<S::ROWB>(r, in_row >> 4) + (in_row & 8);
                                    *reinterpret_cast<uint2*>(d) = make_uint2(w[2 * half], w[2 * half + 1]);
                                }
                            }
                        } else {
#pragma unroll
                            for (int part = 0; part < 2; ++part) {
                                uint32_t w[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    float* v = i < 4 ? p + 2 * i : q + 2 * (i - 4);
                                    w[i] = pack_bf16(v[0], v[1]);
                                    v[0] -= bf16_lo(w[i]);
                                    v[1] -= bf16_hi(w[i]);
                                }
#pragma unroll
                                for (int half = 0; half < 2; ++half) {
                                    const int byte = half * HD + 16 * c, box = byte / S::ROWB;
                                    *reinterpret_cast<uint4*>(sQ + (box * S::NQ + part) * RT * S::ROWB +
                                                              swz<S::ROWB>(r, (byte % S::ROWB) >> 4)) =
                                        make_uint4(w[4 * half], w[4 * half + 1], w[4 * half + 2], w[4 * half + 3]);
                                }
                            }
                        }
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive(q_full);
                if (tid < RT) {
                    const int r = tid < nx.rows ? tid : nx.rows - 1;
                    const int j = (int)udiv((unsigned)(r0 + r), (unsigned)a.G);
                    s_pos2[pn * RT + tid] = nx.len + j;
                    s_row2[pn * RT + tid] = (nx.b * a.M + j) * a.Hq + nx.g * a.G + r0 + r - j * a.G;
                }
                if (tid == 0) s_nfix[pn] = 0;
            }
            if (have) {
                // ---- epilogue: the row sums, then the accumulator ----
                const unsigned int last = ti - 1;
                const int pe = par0;
                wg_sync(wg);   // the last tile's column maxima are read
                {
                    const float v = rows_reduce<false, RW>(l, lane);
                    if (lane % (32 / RW) == 0) s_red[(rw + lane / (32 / RW)) * 4 + w4] = v;
                }
                float* part = s.slot >= 0 ? a.part + s.slot * part_floats(RT, HD) : nullptr;
                if (part) {
#pragma unroll
                    for (int r = 0; r < RW; ++r)
                        if (tok == r) part[RT * HD + rw + r] = m[r];
                }
                wg_sync(wg);
                if (tok < RW) {
                    const float4 q = *reinterpret_cast<const float4*>(s_red + (rw + tok) * 4);
                    const float v = (q.x + q.y) + (q.z + q.w);
                    s_inv[rw + tok] = v == 0.f ? 0.f : 1.f / v;
                    if (part) part[RT * (HD + 1) + rw + tok] = v;
                }
                both_sync();
                const int nfix = s_nfix[pe] < kTcFix ? s_nfix[pe] : kTcFix;
                wait(pv_done + (last & 1), (last >> 1) & 1);
                tc_fence_after();
                float odd = 0.f;   // NaN: the product left something that is not finite
#pragma unroll 1
                for (int d0 = 0; d0 < S::D; ++d0) {
                    uint32_t v[S::NO][RW];
#pragma unroll
                    for (int o = 0; o < S::NO; ++o)
#pragma unroll
                        for (int i = 0; i < RW; i += 8) tmem_ld8(my + S::O0 + (d0 * S::NO + o) * RT + rw + i, v[o] + i);
                    tmem_ld_wait();
                    const int d = d0 * 128 + tok;
                    if (HD < 128 && tok >= HD) continue;   // whole warps
                    float o[RW];
#pragma unroll
                    for (int r = 0; r < RW; ++r) {
                        o[r] = __uint_as_float(v[0][r]);
#pragma unroll
                        for (int part = 1; part < S::NO; ++part) o[r] += __uint_as_float(v[part][r]);
                    }
                    if (!E4M3)
#pragma unroll
                        for (int r = 0; r < RW; ++r) odd = fmaf(o[r], 0.f, odd);
                    for (int f = 0; f < nfix; ++f) {   // values that are not finite, to the rows that attend them
                        const int t = s_fix2[pe * kTcFix + f];
                        const int pg = a.c.table[(long long)s.b * a.c.max_pages + (t >> a.c.ps_log2)];
                        const long long at = pg * a.c.sp + s.g * a.c.sh + (t & (ps - 1)) * a.c.st + d;
                        float val;
                        if (E4M3) val = (reinterpret_cast<const uint8_t*>(a.c.v)[at] & 0x7F) == 0x7F ? __uint_as_float(0x7FC00000u) : 0.f;
                        else val = bf16_to_f32(reinterpret_cast<const uint16_t*>(a.c.v)[at]);
                        if (val - val == 0.f) continue;
#pragma unroll
                        for (int r = 0; r < RW; ++r)
                            if (attends(a.c, t, s_pos2[pe * RT + rw + r])) o[r] += val;
                    }
#pragma unroll
                    for (int r = 0; r < RW; ++r) {
                        if (rw + r >= s.rows) break;
                        if (part) part[(rw + r) * HD + d] = o[r];
                        else reinterpret_cast<uint16_t*>(a.out)[(long long)s_row2[pe * RT + rw + r] * HD + d] = (uint16_t)pack_bf16(o[r] * s_inv[rw + r], 0.f);
                    }
                }
                if (!E4M3 && __builtin_expect(!(odd == 0.f), 0))
                    infinite_values<RW>(&a, plan, s.x, tok, s_pos2 + pe * RT + rw, s_row2 + pe * RT + rw, s_inv + rw,
                                        part ? part + rw * HD : nullptr, s.rows - rw);
                tc_fence_before();
            }
            both_sync();   // the next segment's row tables stand; this one's are read
            if (!more) break;
            s = nx;
            have = true;
            par0 ^= 1;
            const int p_first = s_pos2[par0 * RT], p_last = s_pos2[par0 * RT + RT - 1];
#pragma unroll
            for (int r = 0; r < RW; ++r) {
                l[r] = 0.f;
                m[r] = kNoScore;
                c[r] = E4M3 ? s_c[rw + r] : 1.f;
            }

            for (int k = 0; k < s.n; ++k) {
                const unsigned int t = ti + k, buf = t & 1, par = (t >> 1) & 1;
                wait(meta_full + t % kTcMeta, (t / kTcMeta) & 1);
                const int t0 = tile_at(s.map, s.t0 + k) * kTcTile, pos = t0 + tok;
                const float ks = m_ks[(t % kTcMeta) * 8 + (tok >> box_log2)];
                const float ev = E4M3 ? m_vs[(t % kTcMeta) * 8 + (tok >> box_log2)] : 0.f;
                // every row attends every position of the tile
                const bool whole = m_all[t % kTcMeta] && t0 + kTcTile - 1 <= p_first &&
                                   (a.c.window == 0 || t0 > p_last - a.c.window || t0 + kTcTile <= a.c.sink);
                if (k == s.n - 1 && s.next < xe) open_next(s.next);   // its rows come in during this tile
                wait(s_full + buf, par);
                tc_fence_after();
                float z[RW];
                {
                    constexpr int CW = RW < 16 ? RW : 16;   // rows at a time: all parts of 32 would spill
#pragma unroll
                    for (int b = 0; b < RW; b += CW) {
                        uint32_t v[S::NQ][CW];
#pragma unroll
                        for (int part = 0; part < S::NQ; ++part)
#pragma unroll
                            for (int i = 0; i < CW; i += 8) tmem_ld8(my + buf * S::SCOLS + part * RT + rw + b + i, v[part] + i);
                        tmem_ld_wait();
#pragma unroll
                        for (int r = 0; r < CW; ++r) {
                            z[b + r] = __uint_as_float(v[0][r]) + __uint_as_float(v[1][r]);
                            if (S::NQ == 3) z[b + r] += __uint_as_float(v[S::NQ - 1][r]);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_free + buf);
                if (E4M3) {
#pragma unroll
                    for (int r = 0; r < RW; ++r) z[r] = fmaf(z[r], ks * c[r], ev);
                }
                if (!whole) {
                    // rows at positions [pos, pos + span) attend this one (see attends())
                    const unsigned span = ks == 0.f ? 0u : a.c.window == 0 || pos < a.c.sink ? 1u << 31 : (unsigned)a.c.window;
                    const int4* rows = reinterpret_cast<const int4*>(s_pos2 + par0 * RT + rw);
#pragma unroll
                    for (int r = 0; r < RW; r += 4) {
                        const int4 p = rows[r / 4];
                        if ((unsigned)(p.x - pos) >= span) z[r] = -__int_as_float(0x7F800000);
                        if ((unsigned)(p.y - pos) >= span) z[r + 1] = -__int_as_float(0x7F800000);
                        if ((unsigned)(p.z - pos) >= span) z[r + 2] = -__int_as_float(0x7F800000);
                        if ((unsigned)(p.w - pos) >= span) z[r + 3] = -__int_as_float(0x7F800000);
                    }
                }
                bool over = false;
#pragma unroll
                for (int r = 0; r < RW; ++r) over = over || z[r] > m[r] + S::kSlack;
                if (vote_or(wg, over)) {
                    // move the references: the column maxima of this tile
                    const float mx = rows_reduce<true, RW>(z, lane);
                    if (lane % (32 / RW) == 0) s_red[(rw + lane / (32 / RW)) * 4 + w4] = mx;
                    wg_sync(wg);
#pragma unroll
                    for (int r = 0; r < RW; ++r) {
                        const float4 q = *reinterpret_cast<const float4*>(s_red + (rw + r) * 4);
                        const float mn = fmaxf(fmaxf(fmaxf(q.x, q.y), fmaxf(q.z, q.w)), m[r]);
                        const float f = fexp2(m[r] - mn);
                        l[r] *= f;
                        m[r] = mn;
                        if (tok == r) s_f[rw + r] = f;
                    }
                    if (k > 0) {   // the accumulator, between two tiles' MMAs
                        wait(pv_done + ((t - 1) & 1), ((t - 1) >> 1) & 1);
                        wg_sync(wg);
                        tc_fence_after();
#pragma unroll 1
                        for (int b = 0; b < S::D * S::NO; ++b)
#pragma unroll 1
                            for (int i = 0; i < RW; i += 8) {
                                uint32_t v[8];
                                const uint32_t at = my + S::O0 + b * RT + rw + i;
                                tmem_ld8(at, v);
                                tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 8; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * s_f[rw + i + e]);
                                tmem_st8(at, v);
                            }
                        tmem_st_wait();
                        tc_fence_before();
                    }
                }
                // the tile whose P lay here is read
                if (t >= S::PBUF) wait(pv_done + ((t - S::PBUF) & 1), ((t - S::PBUF) >> 1) & 1);
                unsigned char* P = sP + (t % S::PBUF) * S::PB + tok * 16;
                if (E4M3) {
                    const float unscale = fexp2(-ev);
                    uint32_t w[3][RW / 4];   // four rows a word
#pragma unroll
                    for (int r = 0; r < RW; r += 2) {
                        const float e0 = fexp2(z[r] - m[r] + S::kBias), e1 = fexp2(z[r + 1] - m[r + 1] + S::kBias);
                        l[r] = fmaf(e0, unscale, l[r]);
                        l[r + 1] = fmaf(e1, unscale, l[r + 1]);
                        __half2 h = __floats2half2_rn(e0, e1);
#pragma unroll
                        for (int part = 0; part < 3; ++part) {
                            const uint32_t b = __nv_cvt_halfraw2_to_fp8x2((__half2_raw)h, __NV_SATFINITE, __NV_E5M2);
                            w[part][r >> 2] = r & 2 ? w[part][r >> 2] | (b << 16) : b;
                            if (part < 2) {
                                const uint32_t back = __byte_perm(b, 0, 0x1404);   // e5m2 is fp16's upper byte
                                h = __hsub2(h, *reinterpret_cast<const __half2*>(&back));
                            }
                        }
                    }
#pragma unroll
                    for (int part = 0; part < 3; ++part) {
                        unsigned char* d = P + (part * RT + rw) / 16 * 2048 + rw % 16;
                        if (RW == 8) *reinterpret_cast<uint2*>(d) = make_uint2(w[part][0], w[part][1]);
                        else
#pragma unroll
                            for (int i = 0; i < RW / 16; ++i)
                                *reinterpret_cast<uint4*>(d + i * 2048) =
                                    make_uint4(w[part][4 * i], w[part][4 * i + 1], w[part][4 * i + 2], w[part][4 * i + 3]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < RW / 8; ++i) {
                        uint32_t w[4], v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int r = 8 * i + 2 * e;
                            const float e0 = fexp2(z[r] - m[r]), e1 = fexp2(z[r + 1] - m[r + 1]);
                            l[r] += e0;
                            l[r + 1] += e1;
                            w[e] = pack_bf16(e0, e1);
                            v[e] = pack_bf16(e0 - bf16_lo(w[e]), e1 - bf16_hi(w[e]));
                        }
                        *reinterpret_cast<uint4*>(P + (rw / 8 + i) * 2048) = make_uint4(w[0], w[1], w[2], w[3]);
                        *reinterpret_cast<uint4*>(P + ((RT + rw) / 8 + i) * 2048) = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                }
                if (!whole) {
                    // a value row that not every row attends: zero it where it would
                    // turn a zero weight into a NaN (all of it where nobody attends
                    // it: the slot may hold anything; else only what is not finite,
                    // which the epilogue adds to the rows that do attend it)
                    const bool here = ks != 0.f;
                    const bool any = here && pos <= p_last && (a.c.window == 0 || pos > p_first - a.c.window || pos < a.c.sink);
                    const bool each = here && pos <= p_first && (a.c.window == 0 || pos > p_last - a.c.window || pos < a.c.sink);
                    const unsigned int v0 = g0 + (k == s.n - 1 ? (2 * s.n - 1) * S::D : (2 * k + 2) * S::D);
                    bool listed = false;
                    for (int d = 0; d < S::D; ++d) {
                        const unsigned int g = v0 + d, sl = g % (unsigned)NS;
                        wait(full + sl, (g / (unsigned)NS) & 1);
                        if (each) continue;
                        unsigned char* row = ring + (size_t)sl * S::SLOTB;
                        constexpr int CH = S::NBOX * S::ROWB / 16;   // 16-byte chunks of a row: the warpgroups take turns
                        auto chunk = [&](int i) {
                            return reinterpret_cast<uint4*>(row + (i / (S::ROWB / 16)) * S::BOXB + swz<S::ROWB>(tok, i % (S::ROWB / 16)));
                        };
                        if (!any) {
#pragma unroll
                            for (int i = 0; i < CH; i += 2) *chunk(i + wg) = make_uint4(0, 0, 0, 0);
                            continue;
                        }
                        // one look at the whole row (the largest magnitude bits), value by
                        // value only where that shows something
                        uint32_t top = 0u;
#pragma unroll
                        for (int i = 0; i < CH; i += 2) {
                            const uint4 v = *chunk(i + wg);
                            constexpr uint32_t mask = E4M3 ? 0x7F7F7F7Fu : 0x7FFF7FFFu;
                            top = E4M3 ? __vmaxu4(__vmaxu4(top, v.x & mask), __vmaxu4(v.y & mask, __vmaxu4(v.z & mask, v.w & mask)))
                                       : __vmaxu2(__vmaxu2(top, v.x & mask), __vmaxu2(v.y & mask, __vmaxu2(v.z & mask, v.w & mask)));
                        }
                        if (E4M3 ? __vcmpeq4(top, 0x7F7F7F7Fu) == 0u : __vcmpgeu2(top, 0x7F807F80u) == 0u) continue;
#pragma unroll 1
                        for (int i = wg; i < CH; i += 2) {
                            uint4* e = chunk(i);
                            uint4 v = *e;
                            uint32_t* q = reinterpret_cast<uint32_t*>(&v);
                            bool hit = false;
#pragma unroll
                            for (int n = 0; n < 4; ++n) {
                                if (E4M3) {
#pragma unroll
                                    for (int y = 0; y < 4; ++y)
                                        if (((q[n] >> (8 * y)) & 0x7Fu) == 0x7Fu) {
                                            q[n] &= ~(0xFFu << (8 * y));
                                            hit = true;
                                        }
                                } else {
#pragma unroll
                                    for (int y = 0; y < 2; ++y)
                                        if (((q[n] >> (16 * y)) & 0x7F80u) == 0x7F80u) {
                                            q[n] &= ~(0xFFFFu << (16 * y));
                                            hit = true;
                                        }
                                }
                            }
                            if (hit) {
                                *e = v;
                                listed = true;
                            }
                        }
                    }
                    if (listed) {   // (both warpgroups may list it: an infinity or NaN added twice is the same)
                        const int i = atomicAdd(&s_nfix[par0], 1);
                        if (i < kTcFix) s_fix2[par0 * kTcFix + i] = pos;
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive(p_full + buf);
            }
            ti += s.n;
            g0 += 2 * s.n * S::D;
            x = s.next;
        }
    }
    __syncthreads();
    if (tid == 0) a.cta_status[blockIdx.x] = s_abort ? MTP_ERR_TIMEOUT : s_bad ? MTP_ERR_ARG : MTP_OK;
    if (warp == 9) tmem_dealloc(tmem, S::COLS);
}

template <bool E4M3, int HD, int RT>
cudaError_t go(const PagedTcArgs& p, cudaStream_t s) {
    static int ready[64] = {0};   // the attribute is set, per device
    const int smem = p.slots * tc_slot_bytes(E4M3, HD) + tc_other(E4M3, HD, RT, p.a.B);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || ready[dev] == 0) {
        e = cudaFuncSetAttribute(paged_attn_tc_kernel<E4M3, HD, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmemLimit);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) ready[dev] = 1;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.a.grid);
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // set up while the kernel before it ends
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_attn_tc_kernel<E4M3, HD, RT>, p);
}
template <bool E4M3, int HD>
cudaError_t rows(const PagedTcArgs& p, cudaStream_t s) {
    if (p.a.RT == 16) return go<E4M3, HD, 16>(p, s);
    if (p.a.RT == 32) return go<E4M3, HD, 32>(p, s);
    if constexpr (HD < 512) return go<E4M3, HD, 64>(p, s);
    return cudaErrorInvalidValue;
}

}  // namespace

#ifdef MTP_PAGED_E4M3
cudaError_t launch_paged_attn_tc_e4m3(const PagedTcArgs& p, cudaStream_t s) {
    constexpr bool E = true;
#else
cudaError_t launch_paged_attn_tc_bf16(const PagedTcArgs& p, cudaStream_t s) {
    constexpr bool E = false;
#endif
    switch (p.a.hd) {
    case 64: return rows<E, 64>(p, s);
    case 128: return rows<E, 128>(p, s);
    case 256: return rows<E, 256>(p, s);
    case 512: return rows<E, 512>(p, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace mtp
