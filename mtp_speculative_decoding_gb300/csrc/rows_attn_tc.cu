// rows_attn_tc.cu -- attention of many rows over the paged cache on tcgen05
// tensor cores: whole prompts, and batches that share prefixes.
//
// The rows take the MMA's M side: S [rows, 128 positions] = Q K^T, with the rows
// as rows_prepare.cu has staged them (normed, rotated, rounded once), and O [rows,
// hd] += P V, with P read from tensor memory, where the softmax leaves it over the
// scores it came from, and V's tile as it lies in the page (its dimensions
// contiguous: the N-major operand).  K and V come from the pages by TMA; an e4m3
// cache's codes are opened to fp16, which holds them exactly, and multiplied
// with queries and probabilities in fp16, the page scales folded into the
// scores.
//
// A worker holds 256 rows.  Head dimensions 64 and 128: one CTA with two row
// tiles of 128, whose softmax and MMAs take turns.  Head dimension 256: a pair
// of CTAs (cta_group::2, M = 256) with a row tile each, because the accumulator
// fills half of the tensor memory; each CTA brings half of every K and V tile,
// which halves their traffic, and the scores have two buffers.
//
// Softmax: a thread is a row, or half of one.  The reference m of a row moves only
// when scores lie far above it, so the accumulator is rescaled a few times at most.
// What says so depends on what the registers of a thread hold.  Head dimension 256, half a
// row a thread: the largest score of the tile, found beside the probabilities.  Up to 128,
// where the softmax is the bound: over bf16 caches the sum of the probabilities (a tile's
// largest score is looked for only then: 285 to 270 us at 8192 tokens of 128 dimensions;
// at 256 dimensions e4m3 430 to 448); over e4m3 ones, with fewer registers, a look over
// the scores first, so that no probability waits for the last one (515 to 496 us).
//
// Roundings.  bf16 caches: a rotated query and a probability once to bf16 (2^-8 each),
// half the bits that the attention of a verify step keeps in two parts of each.  A second
// part doubles one of the two products: 361 to 448 (probabilities) or 456 us (queries) for
// 8192 tokens at head dimension 256, where the products are the bound.  Elsewhere they
// are not (13 packed prompts of 128: 170 to 183 or 219 us, 64 sequences behind a prefix: 57
// to 60 for either, each without the softmax's share of it), and the one form is kept for
// its simplicity; against 64 bits results are off by 0.0022 to 0.0029 of their rms, of which
// their own rounding is 0.0016.  e4m3 caches: both to fp16 (2^-11), which the codes need
// anyway; the probabilities with their page's value scale, so that they keep their bits
// down to 2^-25 of the row's largest such product.
//
// Measured, the whole call, one behind another: 8192 tokens, 16 heads of 256 over 4 KV
// heads, bf16: 361 us, 1520 TFLOP/s (in turn with other work 379; the matrix units at what
// clock the power limit leaves them).  The same with 128 dimensions over 8 KV heads: 277
// us, 990 TFLOP/s: matrix units 47 % and issue slots 32 % busy, the two row tiles' chain of
// product, softmax and hand-over bounds it.  e4m3, two pieces of 1024 tokens behind 15000:
// 391 us, 1340 TFLOP/s, bound by opening the codes (4 warps) and the softmax, neither at
// its rate.  64 sequences of up to 3 rows behind 8192 common positions: 54 to 57 us, of
// which this kernel 42: half of its tiles are the sequences' own, where few of 256 rows
// count.
//
// A result that is not finite is computed again, position by position, by the
// kernel behind this one (rows_attn.cu): the products here multiply masked
// positions by a weight of zero, which makes a NaN of an infinity.
#include "rows_attn_tc.cuh"

namespace mtp {

namespace {

// ---- instructions of this kernel; CG: CTAs of an MMA ----
template <int CG>
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t acc) {
    if (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
            "setp.ne.b32 p, %5, 0;\n\tmov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
            "setp.ne.b32 p, %5, 0;\n\tmov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(acc)
            : "memory");
}
// A from tensor memory
template <int CG>
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t acc) {
    if (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
            "setp.ne.b32 p, %5, 0;\n\tmov.b64 db, {%2, %3};\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d), "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
            "setp.ne.b32 p, %5, 0;\n\tmov.b64 db, {%2, %3};\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d), "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(acc)
            : "memory");
}
// arrive once on `bar` (of both CTAs of a pair) when the MMAs issued so far are done
template <int CG>
__device__ __forceinline__ void commit(unsigned long long* bar) {
    if (CG == 1) umma_commit(bar);
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                         smem_addr(bar)),
                     "h"((unsigned short)3)
                     : "memory");
}
template <int CG>
__device__ __forceinline__ void alloc_columns(unsigned int* dst, unsigned int n) {
    if (CG == 1) {
        tmem_alloc(dst, n);
        tmem_relinquish();
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(n) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int CG>
__device__ __forceinline__ void free_columns(unsigned int at, unsigned int n) {
    if (CG == 1) tmem_dealloc(at, n);
    else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(n) : "memory");
}
__device__ __forceinline__ void pair_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// arrive on the leading CTA's barrier of the same place
template <int CG>
__device__ __forceinline__ void arrive_lead(unsigned long long* bar) {
    if (CG == 1) mbar_arrive(bar);
    else
        asm volatile(
            "{\n\t.reg .b32 a;\n\t"
            "mapa.shared::cluster.u32 a, %0, 0;\n\t"
            "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_addr(bar))
            : "memory");
}
// The same for what lies in tensor memory alone, which the tcgen05 fences order: a
// release at cluster scope would wait for the epilogue's stores to global memory.
template <int CG>
__device__ __forceinline__ void arrive_lead_relaxed(unsigned long long* bar) {
    if (CG == 1) mbar_arrive(bar);
    else
        asm volatile(
            "{\n\t.reg .b32 a;\n\t"
            "mapa.shared::cluster.u32 a, %0, 0;\n\t"
            "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_addr(bar))
            : "memory");
}
template <int CG>
__device__ __forceinline__ bool try_wait(unsigned long long* bar, unsigned int parity) {
    if (CG == 1) return mbar_try_wait(bar, parity);
    unsigned int ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool elect() {
    unsigned int p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void ld32(uint32_t at, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
        "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at));
}
__device__ __forceinline__ void st32(uint32_t at, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
        "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(at)
        : "memory");
}
[[maybe_unused]] __device__ __forceinline__ void st16(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
        "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(at)
        : "memory");
}
__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tma_4d(void* dst, const void* tmap, int x, int y, int z, int w, unsigned long long* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
            smem_addr(dst)),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void tma_2d(void* dst, const void* tmap, int x, int y, unsigned long long* bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                     smem_addr(dst)),
                 "l"(tmap), "r"(x), "r"(y), "r"(smem_addr(bar))
                 : "memory");
}
// 32 bytes (a whole sector, where p is aligned to as many) in one store
__device__ __forceinline__ void store_32b(void* p, const uint32_t* w) {
    asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
                 "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
// the same to 16-byte aligned memory
__device__ __forceinline__ void store_2x16b(void* p, const uint32_t* w) {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}
// two warps (64 threads) at barrier `id`: whether any of them says so
__device__ __forceinline__ bool pair_vote(int id, bool x) {
    unsigned int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %2, 0;\n\t"
        "barrier.cta.red.or.aligned.pred q, %1, 64, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"((unsigned)x)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void pair_barrier(int id) { asm volatile("barrier.cta.sync.aligned %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }
__device__ __forceinline__ float most_of(const float* z) {   // of 16
    float x = z[0], y = z[1];
#pragma unroll
    for (int i = 2; i < 14; i += 4) {
        x = max3(x, z[i], z[i + 1]);
        y = max3(y, z[i + 2], z[i + 3]);
    }
    return max3(x, y, fmaxf(z[14], z[15]));
}
// two lanes of fp32 in one instruction
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Operand rows of 128 bytes under the 128-byte swizzle, 8-row groups following
// one another: K-major operands (Q, K: a row, 64 dimensions), and the N-major V (a
// position, 64 dimensions; `lead`: bytes between its 64-wide blocks)
constexpr uint32_t kDescHi = (1024 >> 4) | 1u << 14 | 2u << 29;
__host__ __device__ constexpr uint32_t lead_bits(uint32_t lead) { return (lead >> 4) << 16; }
// fp32 accumulator, M x N, bf16 (1) or fp16 (0) operands, B N-major or not
__host__ __device__ constexpr uint32_t idesc(int type, bool bn, int M, int N) {
    return (1u << 4) | ((uint32_t)type << 7) | ((uint32_t)type << 10) | (bn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ int swz128(int row, int ch) { return row * 128 + ((ch ^ (row & 7)) << 4); }

// e4m3 codes (boxes of 128 or 64 a row, swizzled) to fp16 rows of 64 dimensions, the 16
// codes of a chunk at a time; thread ct of 128
template <int ROWS, int HD, int BYTES>
__device__ __forceinline__ void open_codes(const unsigned char* src, unsigned char* dst, int ct) {
    constexpr int CW = HD < 128 ? 64 : 128, CH = CW / 16;   // codes and chunks of a row
#pragma unroll
    for (int c0 = 0; c0 < BYTES / 16; c0 += 128) {
        const int c = c0 + ct, box = c / (ROWS * CH), r = c / CH % ROWS, ch = c % CH;
        const uint4 v = *reinterpret_cast<const uint4*>(src + box * ROWS * CW + (CW == 128 ? swz128(r, ch) : r * 64 + ((ch ^ ((r >> 1) & 3)) << 4)));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
                : "=r"(o[2 * e]), "=r"(o[2 * e + 1])
                : "r"(w[e]));
        // (lanes of the row's second half begin with the other piece: eight lanes then write
        // to all banks)
        unsigned char* q = dst + (box * (CW / 64) + ch / 4) * ROWS * 128;
        const int turn = ch / 4 & 1, p0 = 2 * (ch & 3) + turn, p1 = p0 ^ 1;
        const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
        *reinterpret_cast<uint4*>(q + swz128(r, p0)) = turn ? hi : lo;
        *reinterpret_cast<uint4*>(q + swz128(r, p1)) = turn ? lo : hi;
    }
}

// What a tile of a piece may take at most, some fifty times what it does
constexpr unsigned long long kTileLimitNs = 100000;

template <bool E4M3, int HD, bool SHARED>
struct RowShape {
    static constexpr int CG = rows_pair(HD), NQ = 2 / CG;          // CTAs of a worker, row tiles of a CTA
    static constexpr int KP = kPosTile / CG, VD = HD / CG;         // positions of K, dimensions of V in this CTA
    static constexpr int QB = 128 * HD * 2;                        // bytes of a row tile
    static constexpr int SLOTB = rows_slot_bytes(HD), RAWB = SLOTB / 2;
    static constexpr int NH = rows_halves(HD);               // threads of a row: each takes its share of a tile's positions
    static constexpr int CW = kPosTile / NH;                       // positions of a thread
    static constexpr int SW = 4 * NQ * NH;                         // softmax warps
    static constexpr int CONV = SW, PROD = SW + (E4M3 ? 4 : 0), MMA = PROD + 1, QUERY = PROD + 2, PARTS = PROD + 3;
    static constexpr int THREADS = (SHARED ? PARTS + 1 : QUERY + 1) * 32;
    static constexpr int O0 = 256, OC = HD;                        // accumulators' columns, behind two score buffers of 128
    // A probability is 2^(z - m), at most 2^kSlack; in fp16 times 2^kBias: with 2^15 at most it
    // stays finite, and down to 2^-25 of the reference it keeps all bits of a normal fp16.
    // TWO: the scores are looked over first.  SUMS: the probabilities' sum is looked at; kMost is
    // what those of a tile may sum to (128 of at most one stay below).
    static constexpr bool TWO = HD < 256 && E4M3, SUMS = HD < 256 && !TWO;
    static constexpr float kBias = E4M3 ? 11.f : 0.f, kSlack = E4M3 ? 4.f : 8.f, kMost = 256.f;
    // place of V tile k among a piece's n tile pairs
    static __device__ __forceinline__ unsigned v_at(int k, int n) { return CG == 1 ? 2 * k + 1 : k == n - 1 ? 2 * n - 1 : 2 * k + 2; }
};

// The part that row r (of sequence seq) of a block's KV head leaves; `dense`: where the
// block's rows begin there
__device__ __forceinline__ RowPart part_of(const RowsTcArgs& t, const Sequences& sq, const PlanHead& plan, const BlockRec& k, int g, int r,
                                           int seq, long long dense) {
    const int rt = r / kRowTile;
    const Item it = item_of<true>(t.a, sq, k, rt);
    const long long U = (long long)kPosTile * t.a.G;
    const long long at = k.pre + g * units_before(t, k, plan.open, row_tiles_of(t.a, k)) + units_before(t, k, plan.open, rt) + plan.open * U;
    int x0 = 0, x1 = it.n - 1;        // tiles that the row has a share in: a sequence's, or all
    if (k.kind == kOwn) {
        x0 = sq.cumt[seq] - it.lt;
        x1 = sq.cumt[seq + 1] - it.lt - 1;
    }
    RowPart p;
    p.there = 1;
    p.dense = RowPart::kSlots;
    p.r = (uint16_t)(r % kRowTile);
    p.first = p.w0 = p.w1 = (uint16_t)worker_of(plan.T, plan.workers, at);
    if (p.first == worker_of(plan.T, plan.workers, at + (it.n - 1) * U)) {
        p.dense = (uint32_t)(k.q_row + (long long)g * k.q_stride + r + dense);
    } else {
        p.w0 = (uint16_t)worker_of(plan.T, plan.workers, at + x0 * U);
        p.w1 = (uint16_t)worker_of(plan.T, plan.workers, at + x1 * U);
    }
    return p;
}

// Score buffer of a tile that concerns one row tile: two such in a row take turns, so
// that one's scores are computed while the other's weights are (both row tiles: a buffer
// each).  rows, was: row tiles of this tile and of the one before, side: the buffer then.
__device__ __forceinline__ int score_side(int rows, int was, int side) { return rows == 3 || was == 3 ? 0 : side ^ 1; }

template <bool E4M3, int HD, bool SHARED>
__global__ void __launch_bounds__(RowShape<E4M3, HD, SHARED>::THREADS, 1) rows_tc_kernel(const __grid_constant__ RowsTcParams pp) {
    using S = RowShape<E4M3, HD, SHARED>;
    constexpr int CG = S::CG, NQ = S::NQ, NR = rows_raw(E4M3, HD), NS = rows_slots(E4M3, HD);
    static_assert(NS >= 2 && NS <= kRowsSlots && NR <= kRowsRaw, "ring");
    const RowsTcArgs& t = pp.t;
    const RowsArgs& a = t.a;
    extern __shared__ unsigned char raw_smem[];
    unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~(uintptr_t)1023);
    unsigned char* sQ = base;
    unsigned char* ring = sQ + NQ * S::QB;
    unsigned char* raw = ring + (size_t)NS * S::SLOTB;
    uint4* m_bits = reinterpret_cast<uint4*>(raw + (size_t)NR * S::RAWB);       // [kRowsMeta] positions that are there
    float2* m_sc = reinterpret_cast<float2*>(m_bits + kRowsMeta);               // [kRowsMeta][8] key scale, value scale's exponent, every 16 positions
    int4* m_flag = reinterpret_cast<int4*>(m_sc + kRowsMeta * 8);               // [kRowsMeta] x: row tiles, 4: all positions there, 8: score buffer (one row tile); y: sequence; z, w: the tile's [pos, end)
    float* s_x = reinterpret_cast<float*>(m_flag + kRowsMeta);                  // [NQ][2][128] what the threads of a row tell each other
    unsigned long long* bars = reinterpret_cast<unsigned long long*>(s_x + 2 * kRowTile);
    unsigned long long *full = bars, *empty = full + kRowsSlots, *peer = empty + kRowsSlots, *rfull = peer + kRowsSlots,
                       *rempty = rfull + kRowsRaw, *meta = rempty + kRowsRaw, *s_full = meta + kRowsMeta, *p_full = s_full + 4,
                       *pv_done = p_full + 2, *o_free = pv_done + 4, *q_full = o_free + 2, *q_peer = q_full + 1, *q_free = q_peer + 1,
                       *end_bar = q_free + 1, *mfree = end_bar + 1;
    int* s_tab = reinterpret_cast<int*>(bars + 3 * kRowsSlots + 2 * kRowsRaw + 2 * kRowsMeta + 16);   // shared prefixes: the sequences' tables
    const Sequences sq = {s_tab, s_tab + a.B + 1, s_tab + 2 * a.B + 2};
    __shared__ unsigned int s_tmem;
    __shared__ int s_bad;
    __shared__ volatile int s_abort;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int rank = CG == 1 ? 0 : (int)cta_rank(), me = (int)blockIdx.x / CG;
    if (tid == 0) {
        for (int i = 0; i < kRowsSlots; ++i) {
            mbar_init(full + i, E4M3 ? 4 : 1);
            mbar_init(empty + i, 1);
            mbar_init(peer + i, 1);
        }
        for (int i = 0; i < kRowsRaw; ++i) {
            mbar_init(rfull + i, 1);
            mbar_init(rempty + i, 4);
        }
        for (int i = 0; i < kRowsMeta; ++i) {
            mbar_init(meta + i, 1);
            mbar_init(mfree + i, S::SW);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(s_full + i, 1);     // [row tile][score buffer]
            mbar_init(pv_done + i, 1);    // [row tile][its tiles in turns: a wait may be two of them behind]
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(p_full + i, 4 * CG * S::NH);   // [score buffer]
            mbar_init(o_free + i, 4 * CG * S::NH);
        }
        mbar_init(q_full, 1);
        mbar_init(q_peer, 1);
        mbar_init(q_free, 1);
        mbar_init(end_bar, 1);
        s_bad = 0;
        s_abort = 0;
    }
    mbar_fence_init();
    if (tid < 3) {
        const CUtensorMap* m = tid == 0 ? &pp.tk : tid == 1 ? &pp.tv : &pp.tq;
        asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
    }
    if (CG == 2) pair_sync();   // the peer's barriers stand
    if (warp == S::MMA) alloc_columns<CG>(&s_tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");      // the plan and the staged rows are there
    const WorkerRec first = t.worker[me];
    if (SHARED && a.n_groups > 0) {
        for (int i = tid; i <= a.B; i += S::THREADS) {
            s_tab[i] = t.cum[i];
            s_tab[a.B + 1 + i] = t.cumt[i];
            if (i < a.B) s_tab[2 * a.B + 2 + i] = t.lens[i];
        }
        __syncthreads();
    }
    // bounded wait; after one gave up every other does too
    auto wait_for = [&](unsigned long long* bar, unsigned int parity, unsigned long long limit) -> bool {
        if (try_wait<CG>(bar, parity)) return true;
        const unsigned long long t0 = global_ns();
        while (!try_wait<CG>(bar, parity)) {
            if (s_abort) return false;
            if (global_ns() - t0 > limit) {
                s_abort = 1;
                return false;
            }
        }
        return true;
    };
    auto wait = [&](unsigned long long* bar, unsigned int parity) { return wait_for(bar, parity, t.timeout_ns); };
    auto wait_all = [&](unsigned long long* bar, unsigned int parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
    const int ps = 1 << a.c.ps_log2;
    constexpr uint32_t idS = idesc(E4M3 ? 0 : 1, false, 128 * CG, kPosTile), idO = idesc(E4M3 ? 0 : 1, true, 128 * CG, HD);

    if (warp == S::PROD) {
        // ------------------------------------------------------------------
        // producer: K and V tiles in the order the MMAs take them; lane i of a tile
        // holds page i of its positions
        // ------------------------------------------------------------------
        const int vl = a.c.ps_log2 < 7 ? a.c.ps_log2 : 7, kl = vl < (CG == 2 ? 6 : 7) ? vl : (CG == 2 ? 6 : 7);   // box rows (log2)
        const int vr = 1 << vl, nv = kPosTile >> vl, kr = 1 << kl, nk = S::KP >> kl;
        constexpr int KB = E4M3 ? (HD < 128 ? 64 : 128) : 64;   // dimensions of a box
        constexpr int ESZ = E4M3 ? 1 : 2;
        constexpr int SLOTS = E4M3 ? NR : NS, DSTB = E4M3 ? S::RAWB : S::SLOTB;
        unsigned char* dst0 = E4M3 ? raw : ring;
        unsigned long long *bf = E4M3 ? rfull : full, *be = E4M3 ? rempty : empty;
        unsigned slot = 0, phase = 0, ti = 0;
        bool ok = true, bad = false;
        RowNote note = {-1, 0, 0, 0, 0, {0, 0, 0}};
        Walk<SHARED> p;
        p.start(first, sq);
        while (ok && p.next(t)) {
            const int wlo = a.c.window > 0 && p.it.p_first + 1 > a.c.window ? p.it.p_first + 1 - a.c.window : 0;
            const int wfar = a.c.window > 0 && p.it.p_last + 1 > a.c.window ? p.it.p_last + 1 - a.c.window : 0;
            const int sink = a.c.sink < wfar ? a.c.sink : wfar;
            auto entry = [&](int k, Tile& tl) -> int {   // page of this lane's positions of tile k; below 0: not loaded
                if (k >= p.n) return -2;
                tl = tile_of<SHARED>(a, sq, p.k, p.it, p.t0 + k);
                const int p0 = tl.pos + (lane << vl);
                if (lane >= nv || p0 >= tl.end || p0 + vr <= p.k.lo || (p0 + vr <= wlo && p0 >= sink)) return -2;
                const int pg = a.c.table[(long long)tl.seq * a.c.max_pages + (p0 >> a.c.ps_log2)];
                if ((unsigned)pg < (unsigned)a.c.n_pages) return pg;
                bad = true;
                return -1;
            };
            auto load = [&](bool key, int pos, int pg) {
                ok = wait_all(be + slot, phase ^ 1);
                if (!ok) return;
                unsigned char* dst = dst0 + (size_t)slot * DSTB;
                if (key) {
                    const int off = rank * S::KP + (lane << kl);      // this lane's first position in the tile
                    const int kp = __shfl_sync(0xffffffffu, pg, (off >> vl) & 31);
                    const bool mine = lane < nk && kp >= 0;
                    const unsigned cnt = __popc(__ballot_sync(0xffffffffu, mine));
                    if (lane == 0) mbar_arrive_expect_tx(bf + slot, cnt * (unsigned)(kr * HD * ESZ));
                    __syncwarp();
                    if (mine)
#pragma unroll
                        for (int c = 0; c < HD / KB; ++c)
                            tma_4d(dst + c * (S::KP * KB * ESZ) + (lane << kl) * (KB * ESZ), &pp.tk, c * KB, (pos + off) & (ps - 1), p.g, kp, bf + slot);
                } else {
                    const bool mine = lane < nv && pg >= 0;
                    const unsigned cnt = __popc(__ballot_sync(0xffffffffu, mine));
                    if (lane == 0) mbar_arrive_expect_tx(bf + slot, cnt * (unsigned)(vr * S::VD * ESZ));
                    __syncwarp();
                    if (mine)
#pragma unroll
                        for (int c = 0; c < S::VD / KB; ++c)
                            tma_4d(dst + c * (kPosTile * KB * ESZ) + (lane << vl) * (KB * ESZ), &pp.tv, rank * S::VD + c * KB,
                                   (pos + (lane << vl)) & (ps - 1), p.g, pg, bf + slot);
                }
                if (++slot == (unsigned)SLOTS) {
                    slot = 0;
                    phase ^= 1;
                }
            };
            Tile nt = {};
            int npg = entry(0, nt), held = -2, held_pos = 0, was = 3, side = 0;
#pragma unroll 1
            for (int k = 0; k <= p.n && ok; ++k) {
                const int pg = npg;
                const Tile tile = nt;
                npg = entry(k + 1, nt);
                if (k < p.n) {
                    load(true, tile.pos, pg);
                    // the tile's masks and scales, while its keys are on their way
                    bool there = pg >= 0;
                    float ks = 1.f, ev = 0.f;
                    if (E4M3 && there) {
                        const long long o = (long long)pg * a.c.Hkv + p.g;
                        const float kss = a.c.ks[o], vss = a.c.vs[o];
                        there = scale_ok(kss) && scale_ok(vss);   // else the page counts as absent
                        bad = bad || !there;
                        ks = there ? kss : 1.f;
                        ev = there ? (float)((int)(__float_as_uint(vss) >> 23) - 127) : 0.f;
                    }
                    // lane i < 8: positions [16 i, 16 i + 16)
                    const int src = lane < 8 ? (lane << 4) >> vl : 0;
                    const bool th = __shfl_sync(0xffffffffu, (int)there, src) != 0;
                    const float k8 = __shfl_sync(0xffffffffu, ks, src), e8 = __shfl_sync(0xffffffffu, ev, src);
                    const unsigned have = __ballot_sync(0xffffffffu, lane < 8 && th) & 0xFFu;
                    const unsigned mi = ti % kRowsMeta;
                    // (a pair's warps all answer every tile, so none of them is that far behind; here a
                    // row tile's warps pass over the other's tiles)
                    if (CG == 1) {
                        ok = wait_all(mfree + mi, ((ti / kRowsMeta) & 1) ^ 1);
                        if (!ok) break;
                    }
                    side = score_side(tile.rows, was, side);
                    was = tile.rows;
                    if (lane < 8 && E4M3) m_sc[mi * 8 + lane] = make_float2(k8, e8);
                    if (lane == 0) {
                        auto word = [&](int i) { return ((have >> (2 * i)) & 1u ? 0xFFFFu : 0u) | ((have >> (2 * i + 1)) & 1u ? 0xFFFF0000u : 0u); };
                        m_bits[mi] = make_uint4(word(0), word(1), word(2), word(3));
                        m_flag[mi] = make_int4((have == 0xFFu ? 4 : 0) | tile.rows | side << 3, tile.seq, tile.pos, tile.end);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(meta + mi);
                    ++ti;
                }
                if (CG == 1) {
                    if (k < p.n && ok) load(false, tile.pos, pg);
                } else {
                    if (k > 0 && ok) load(false, held_pos, held);
                    held = pg;
                    held_pos = tile.pos;
                }
            }
            if (!SHARED && p.slot == 2 && p.t0 == 0)
                note = RowNote{worker_of(t.head->T, t.head->workers, p.tiles_at + (long long)(p.it.n - 1) * kPosTile * a.G), p.it.rows, p.it.r0,
                               p.g, p.k.row0, {0, 0, 0}};
        }
        if (!SHARED && rank == 0 && lane == 0) t.note[me] = note;
        if (__any_sync(0xffffffffu, bad) && lane == 0) s_bad = 1;
        if (!ok) {   // gave up: this warp's copies in flight end before the CTA does
            const unsigned long long t0 = global_ns();
            for (int i = 0; i < SLOTS; ++i) {
                const unsigned ph = i < (int)slot ? phase : phase ^ 1;
                while (!try_wait<CG>(bf + i, ph) && global_ns() - t0 < t.timeout_ns) {}
            }
        }
    } else if (warp == S::QUERY) {
        // ------------------------------------------------------------------
        // the items' staged rows; the second CTA of a pair tells the first
        // ------------------------------------------------------------------
        unsigned seg = 0;
        bool ok = true;
        unsigned long long limit = t.timeout_ns;
        Walk<SHARED> p;
        p.start(first, sq);
        while (ok && p.next(t)) {
            // as long as the piece before takes, the one wait here that is not for a tile's work
            // (a piece of 10^6 tiles takes longer than any other wait may)
            ok = __all_sync(0xffffffffu, wait_for(q_free, (seg & 1) ^ 1, limit)) != 0;
            if (!ok) break;
            limit = t.timeout_ns + (unsigned long long)p.n * kTileLimitNs;
            const int tiles = CG == 1 && p.it.rows <= 128 ? 1 : NQ;
            const long long row = p.k.q_row + (long long)p.g * p.k.q_stride + p.it.r0 + rank * 128;
            if (lane == 0) mbar_arrive_expect_tx(q_full, (unsigned)(tiles * S::QB));
            __syncwarp();
            if (lane < tiles * (HD / 64)) {
                const int q = lane / (HD / 64), c = lane % (HD / 64);
                tma_2d(sQ + q * S::QB + c * 128 * 128, &pp.tq, c * 64, (int)row + q * 128, q_full);
            }
            __syncwarp();
            ok = wait_all(q_full, seg & 1);
            if (!ok) {   // gave up: the copy in flight ends before the CTA does
                const unsigned long long t0 = global_ns();
                while (!try_wait<CG>(q_full, seg & 1) && global_ns() - t0 < t.timeout_ns) {}
                __syncwarp();
            }
            if (CG == 2 && rank == 1 && ok && lane == 0) arrive_lead<CG>(q_peer);
            __syncwarp();
            ++seg;
        }
    } else if (SHARED && warp == S::PARTS) {
        // ------------------------------------------------------------------
        // where the parts of the rows will lie, for the merge (which would take 8 us for
        // it with nothing beside it): lane = row of out
        // ------------------------------------------------------------------
        const PlanHead plan = *t.head;
        const Sequences s = a.n_groups > 0 ? sq : Sequences{t.cum, t.cumt, t.lens};
        const long long rows = (long long)a.B * a.M * a.Hq;
        for (long long id = (long long)blockIdx.x * 32 + lane; id < rows; id += (long long)gridDim.x * 32) {
            const int tok = (int)(id / a.Hq), h = (int)(id - (long long)tok * a.Hq), b = tok / a.M, j = tok - b * a.M, c0 = s.cum[b];
            RowPart own = {}, pre = {};
            if (j < s.cum[b + 1] - c0) {
                const int g = h / a.G, rj = j * a.G + h - g * a.G;
                const BlockRec k = t.blocks[2 * a.n_groups + b];
                if (k.n > 0) {
                    own = part_of(t, s, plan, k, g, rj, b, rows);
                } else {   // of a group
                    const int i = last_at_most(a.group_start, a.n_groups, b);
                    const BlockRec o = t.blocks[a.n_groups + i], p = t.blocks[i];
                    const int r = (c0 - s.cum[o.table]) * a.G + rj;
                    own = part_of(t, s, plan, o, g, r, b, rows);
                    if (p.n > 0) pre = part_of(t, s, plan, p, g, r, b, 0);
                }
            }
            t.row_parts[2 * id] = own;
            t.row_parts[2 * id + 1] = pre;
        }
    } else if (E4M3 && warp >= S::CONV && warp < S::CONV + 4) {
        // ------------------------------------------------------------------
        // codes to fp16: a thread opens 16 of them at a time
        // ------------------------------------------------------------------
        const int ct = tid - S::CONV * 32;
        unsigned slot = 0, phase = 0, rs = 0, rp = 0;
        bool ok = true;
        Walk<SHARED> p;
        p.start(first, sq);
        while (ok && p.next(t)) {
#pragma unroll 1
            for (int i = 0; i < 2 * p.n && ok; ++i) {
                // K tiles and V tiles take turns: K0 V0 K1 V1 .., or K0 K1 V0 K2 V1 .. Kn-1 Vn-2 Vn-1
                const bool key = CG == 1 ? (i & 1) == 0 : i == 0 || ((i & 1) != 0 && i != 2 * p.n - 1);
                ok = wait_all(rfull + rs, rp);
                ok = ok && wait_all(empty + slot, phase ^ 1);
                if (!ok) break;
                const unsigned char* src = raw + (size_t)rs * S::RAWB;
                unsigned char* dst = ring + (size_t)slot * S::SLOTB;
                if (key) open_codes<S::KP, HD, S::RAWB>(src, dst, ct);
                else open_codes<kPosTile, HD, S::RAWB>(src, dst, ct);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(full + slot);
                    mbar_arrive(rempty + rs);
                }
                if (++slot == (unsigned)NS) {
                    slot = 0;
                    phase ^= 1;
                }
                if (++rs == (unsigned)NR) {
                    rs = 0;
                    rp ^= 1;
                }
            }
        }
    } else if (warp == S::MMA) {
        // ------------------------------------------------------------------
        // MMA issue: the whole warp walks, one elected lane issues; the second CTA
        // of a pair tells the first what has come in
        // ------------------------------------------------------------------
        unsigned slot = 0, phase = 0, seg = 0;
        bool ok = true;
        auto hold = [&](unsigned long long* bar, unsigned parity) {
            ok = ok && wait_all(bar, parity);
            tc_fence_after();
        };
        auto next = [&] {
            if (++slot == (unsigned)NS) {
                slot = 0;
                phase ^= 1;
            }
        };
        Walk<SHARED> p;
        p.start(first, sq);
        if (CG == 2 && rank == 1) {
            while (ok && p.next(t))
                for (int i = 0; i < 2 * p.n && ok; ++i) {
                    hold(full + slot, phase);
                    if (ok && lane == 0) arrive_lead<CG>(peer + slot);
                    __syncwarp();
                    next();
                }
        } else {
            const uint32_t q0 = smem_addr(sQ) >> 4, r0 = smem_addr(ring) >> 4;
            // bit i: odd uses of score buffer i, pieces and products of row tile i so far (a pair's
            // score buffers take turns: t0 tiles)
            unsigned sbit = 0u, pbit = 0u, vbit = 0u, t0 = 0u;
            auto arrived = [&] {
                hold(full + slot, phase);
                if (CG == 2) hold(peer + slot, phase);
            };
            // the products of a step, by one lane: first P V of tile k - 1, then Q K^T of tile k (each
            // where it is asked for), and what they free
            auto issue = [&](bool pv, int q, int pbuf, unsigned at, bool first, bool v_done, bool qk, int sq_, int sbuf, bool k_done, bool q_done) {
                if (ok && elect()) {
                    if (pv) {
                        const uint32_t bl = r0 + at * (S::SLOTB >> 4) + lead_bits(S::VD > 64 ? kPosTile * 128 : 16);
#pragma unroll
                        for (int ks = 0; ks < kPosTile / 16; ++ks)
                            umma_ts<CG>(tmem + S::O0 + q * S::OC, tmem + pbuf * 128 + ks * 8, bl + (ks * 16 * 128 >> 4), kDescHi, idO, !first || ks > 0);
                        commit<CG>(pv_done + 2 * q + (vbit >> q & 1u));
                        if (v_done) commit<CG>(empty + at);
                    }
                    if (qk) {
                        const uint32_t al = q0 + sq_ * (S::QB >> 4) + lead_bits(16), bl = r0 + slot * (S::SLOTB >> 4) + lead_bits(16);
#pragma unroll
                        for (int b = 0; b < HD / 64; ++b)
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                umma_ss<CG>(tmem + sbuf * 128, al + (b * 128 * 128 + ks * 32 >> 4), bl + (b * S::KP * 128 + ks * 32 >> 4), kDescHi,
                                            idS, b > 0 || ks > 0);
                        commit<CG>(s_full + 2 * sq_ + sbuf);
                        if (k_done) commit<CG>(empty + slot);
                        if (q_done) commit<CG>(q_free);
                    }
                }
                __syncwarp();
                if (pv) vbit ^= 1u << q;
                if (qk) sbit ^= 1u << sbuf;
            };
            bool more_pieces = p.next(t);
            while (ok && more_pieces) {
                const int n = p.n;   // (p moves on before this piece's last product)
                hold(q_full, seg & 1);
                if (CG == 2) hold(q_peer, seg & 1);
                ++seg;
                if (CG == 2) {
#pragma unroll 1
                    for (int k = 0; k <= n && ok; ++k) {
                        if (k < n) {
                            arrived();
                            issue(false, 0, 0, 0, false, false, true, 0, (t0 + k) & 1, true, k == n - 1);
                            next();
                        } else {
                            more_pieces = p.next(t);
                        }
                        if (k > 0) {
                            const unsigned u = t0 + k - 1;
                            if (k == 1) hold(o_free, (pbit & 1u) ^ 1u);
                            arrived();
                            hold(p_full + (u & 1), (u >> 1) & 1);
                            issue(true, 0, u & 1, slot, k == 1, true, false, 0, 0, false, false);
                            next();
                        }
                    }
                    t0 += n;
                    pbit ^= 1u;
                } else {
                    // slots take turns: K tile k, V tile k; a tile concerns one row tile or both
                    unsigned vslot = 0, vphase = 0;
                    int rows = 0, had = 0;           // row tiles of tile k - 1, of the piece so far
                    int side = 0;                    // score buffer of tile k - 1
                    auto rows_at = [&](int k) { return SHARED && p.k.kind == kOwn ? tile_of<SHARED>(a, sq, p.k, p.it, p.t0 + k).rows : p.it.rows > 128 ? 3 : 1; };
                    int ahead = rows_at(0);          // looked up while the products before run
                    auto weights = [&](int q, int buf) {   // row tile q's of tile k - 1 are there, and its accumulator is free
                        if (!(had >> q & 1)) hold(o_free + q, (pbit >> q & 1u) ^ 1u);
                        hold(p_full + buf, (sbit >> buf & 1u) ^ 1u);
                    };
#pragma unroll 1
                    for (int k = 0; k <= n && ok; ++k) {
                        const bool more = k < n, end = k == n - 1;
                        const int now = more ? ahead : 0;
                        if (more) arrived();
                        else more_pieces = p.next(t);
                        if (k > 0) hold(full + vslot, vphase);
                        if (!SHARED || (rows == 3 && now != 1 && now != 2)) {   // a buffer a row tile
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                const bool pv = rows >> q & 1, qk = now >> q & 1, last = q == 1 || !((rows | now) >> 1);
                                if (!pv && !qk) continue;
                                if (pv) weights(q, q);
                                issue(pv, q, q, vslot, !(had >> q & 1), last, qk, q, q, last, last && end);
                                if (pv) had |= 1 << q;
                            }
                            side = 0;
                        } else {
                            const int to = score_side(now, k == 0 ? 3 : rows, side);
                            const bool one = now == 1 || now == 2;
                            // (scores of one row tile first, unless both buffers hold weights)
                            if (one && rows != 3) issue(false, 0, 0, 0, false, false, true, now - 1, to, true, end);
                            if (rows == 3) {
#pragma unroll
                                for (int q = 0; q < 2; ++q) {
                                    weights(q, q);
                                    issue(true, q, q, vslot, !(had >> q & 1), q == 1, false, 0, 0, false, false);
                                }
                            } else if (rows) {
                                weights(rows - 1, side);
                                issue(true, rows - 1, side, vslot, !(had >> (rows - 1) & 1), true, false, 0, 0, false, false);
                            }
                            had |= rows;
                            if (one && rows == 3) issue(false, 0, 0, 0, false, false, true, now - 1, to, true, end);
                            if (now == 3) {
                                issue(false, 0, 0, 0, false, false, true, 0, 0, false, false);
                                issue(false, 0, 0, 0, false, false, true, 1, 1, true, end);
                            }
                            side = to;
                        }
                        rows = now;
                        if (more) {
                            next();
                            vslot = slot;
                            vphase = phase;
                            next();
                            if (k + 1 < n) ahead = rows_at(k + 1);
                        }
                    }
                    pbit ^= (unsigned)had;
                }
            }
            if (elect()) commit<CG>(end_bar);   // whatever was issued has ended before its memory goes
            __syncwarp();
        }
        const unsigned long long t0 = global_ns();
        while (!try_wait<CG>(end_bar, 0) && global_ns() - t0 < 2 * t.timeout_ns) {}
        __syncwarp();
    } else {
        // ------------------------------------------------------------------
        // softmax and epilogue: thread = row
        // ------------------------------------------------------------------
        constexpr int NH = S::NH, CW = S::CW;
        const int q = warp / (4 * NH), half = (warp >> 2) % NH, row = tid & 127;   // row tile of this CTA, share of a tile, row
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t oat = tmem + lanes + S::O0 + q * S::OC + half * (HD / NH);   // this thread's part of the accumulator
        unsigned tc = 0, ti = 0, g0 = 0;                     // tiles of this row tile, of the CTA; ring slots before this piece
        unsigned used = 0;                                   // bit b: odd uses of score buffer b by this row tile
        const bool sectors = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;   // (the caller owes 16 bytes; rows are multiples of 128)
        auto meet = [&](unsigned long long* bar, unsigned parity) {
            wait(bar, parity);
            __syncwarp();
        };
        // tile i of this row tile is in the accumulator
        auto meet_values = [&](unsigned i) {
            wait(pv_done + 2 * q + (i & 1), (i >> 1) & 1);
            __syncwarp();
            tc_fence_after();
        };
        // the warps of the same 32 rows: whether any of their threads says so; and what the
        // other thread of this row has
        auto any_of_rows = [&](bool x) -> bool {
            if (NH == 1) return __any_sync(0xffffffffu, x);
            return pair_vote(1 + q * 4 + (warp & 3), x);
        };
        auto others = [&](float x) -> float {
            s_x[(q * 2 + half) * 128 + row] = x;
            pair_barrier(1 + q * 4 + (warp & 3));
            const float y = s_x[(q * 2 + (half ^ 1)) * 128 + row];
            pair_barrier(1 + q * 4 + (warp & 3));
            return y;
        };
        Walk<SHARED> p;
        p.start(first, sq);
        bool more_pieces = p.next(t);
        while (more_pieces) {
            const int ofs = (CG == 2 ? rank : q) * 128;      // of the row tile in the item
            const bool live = ofs + row < p.it.rows;
            const int r = p.it.r0 + (live ? ofs + row : p.it.rows - 1);   // row of the block
            int tok = (int)udiv((unsigned)r, (unsigned)a.G), seq = p.k.table, pos_q = p.k.len + tok;   // its token, sequence, position
            if (SHARED && p.k.kind == kOwn) {
                const int x = sq.cum[p.k.table] + tok;
                seq += last_at_most(sq.cum + p.k.table, p.k.len - p.k.table, x);
                pos_q = sq.lens[seq] + x - sq.cum[seq];
            }
            const int end = SHARED && p.k.kind == kPrefix ? p.k.hi : pos_q + 1;     // attends [.., end)
            const int low = a.c.window > 0 && pos_q + 1 > a.c.window ? pos_q + 1 - a.c.window : 0;
            // what a score is multiplied by: the softmax scale, and what the staged row was divided by
            const float qc = E4M3 ? t.q_scale[p.k.q_row + (long long)p.g * p.k.q_stride + r] : a.scale;
            float m = kNoScore, l = 0.f;
            bool none = true, touched = false;               // no tile of this row tile yet; of this row
#pragma unroll 1
            for (int k = 0; k < p.n; ++k, ++ti) {
                const unsigned mi = ti % kRowsMeta;
                meet(meta + mi, (ti / kRowsMeta) & 1);
                const int4 flag = m_flag[mi];
                const int t0 = SHARED ? flag.z : tile_of<SHARED>(a, sq, p.k, p.it, p.t0 + k).pos;
                const bool mine = !SHARED || p.k.kind != kOwn || seq == flag.y;   // the tile is on this row's sequence
                int zq = 0;                                  // the row tile that looks after the tile's values
                int buf = CG == 2 ? (int)(tc & 1) : q;
                if (CG == 1) {
                    if (!(flag.x >> q & 1)) {                // the other row tile's alone
                        __syncwarp();
                        if (lane == 0) mbar_arrive(mfree + mi);
                        continue;
                    }
                    if (SHARED && (flag.x & 3) != 3) buf = flag.x >> 3 & 1;
                    zq = flag.x & 1 ? 0 : 1;
                }
                const unsigned parity = used >> buf & 1u;
                used ^= 1u << buf;
                const uint32_t sat = tmem + lanes + buf * 128;
                // every row of the item attends every position of the tile
                const bool whole = (flag.x & 4) && (!SHARED || (p.k.kind != kOwn && t0 >= p.k.lo)) &&
                                   (SHARED && p.k.kind == kPrefix ? t0 + kPosTile <= p.k.hi : t0 + kPosTile - 1 <= p.it.p_first) &&
                                   (a.c.window == 0 || t0 > p.it.p_last - a.c.window || t0 + kPosTile <= a.c.sink);
                uint32_t bits[CW / 32];
#pragma unroll
                for (int i = 0; i < CW / 32; ++i) bits[i] = ~0u;
                auto on_bits = [&](int i) {   // positions [32 i, 32 i + 32) of the tile that this row attends
                    const uint32_t there = reinterpret_cast<const uint32_t*>(m_bits + mi)[i];
                    const int c0 = t0 + 32 * i;
                    auto below = [&](int e) { return e - c0 >= 32 ? ~0u : e - c0 <= 0 ? 0u : (1u << (e - c0)) - 1u; };   // positions < e
                    uint32_t on = below(end) & ~below(p.k.lo);
                    if (low > 0) on &= ~below(low) | below(a.c.sink);
                    return mine ? there & on : 0u;
                };
                if (!whole)
#pragma unroll
                    for (int i = 0; i < CW / 32; ++i) bits[i] = on_bits(half * (CW / 32) + i);
                meet(s_full + 2 * q + buf, parity);
                tc_fence_after();
                if (!S::TWO && (none || (SHARED && __any_sync(0xffffffffu, mine && !touched)))) {
                    // a first reference from the tile's first 16 positions: seldom does a score lie far
                    // above it
                    uint32_t s[16];
                    tmem_ld16(sat, s);
                    tmem_ld_wait();
                    const uint32_t on = whole ? ~0u : on_bits(0);
                    float x = -__int_as_float(0x7F800000);
#pragma unroll
                    for (int i = 0; i < 16; ++i) x = fmaxf(x, on >> i & 1u ? __uint_as_float(s[i]) : -__int_as_float(0x7F800000));
                    if (E4M3) x = fmaf(x, m_sc[mi * 8].x * qc, m_sc[mi * 8].y);
                    else x *= qc;
                    if (!SHARED || !touched) m = fmaxf(m, x);
                }
                const bool idle = SHARED && p.k.kind == kOwn && !__any_sync(0xffffffffu, mine);   // none of this warp's rows: weights of zero
                // ---- probabilities against the reference there is; where a score lies too far above
                // it, once more against the largest one (the scores stay in place until all is well;
                // TWO: the reference is right at once, and probabilities go over the scores piece by piece) ----
                constexpr int CH = HD < 256 ? 16 : 32;   // positions of a load (registers)
                // the references to mx, and with them what has been summed
                auto move = [&](float mx) {
                    if (NH == 2) mx = fmaxf(mx, others(mx));
                    const float mn = fmaxf(mx, m), f = ex2(m - mn);
                    const bool scale = any_of_rows((!SHARED || touched) && f != 1.f);   // (where nothing is summed yet all is zero)
                    l *= f;
                    m = mn;
                    if (!none && scale) {
                        meet_values(tc - 1);
#pragma unroll 1
                        for (int c = 0; c < HD / NH; c += 32) {
                            uint32_t v[32];
                            ld32(oat + c, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
                            st32(oat + c, v);
                        }
                        st_wait();
                        tc_fence_before();
                    }
                };
                if (S::TWO && !idle) {
                    float mx = -__int_as_float(0x7F800000);   // the row's largest score, in bits, with the value scale
                    uint32_t v[2][32];
                    ld32(sat, v[0]);
#pragma unroll
                    for (int c = 0; c < CW / 32; ++c) {
                        tmem_ld_wait();
                        if (c + 1 < CW / 32) ld32(sat + 32 * (c + 1), v[(c + 1) & 1]);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float* z = reinterpret_cast<float*>(v[c & 1]) + 16 * h;
                            if (!whole) {
#pragma unroll
                                for (int i = 0; i < 16; ++i) z[i] = bits[c] >> (16 * h + i) & 1u ? z[i] : -__int_as_float(0x7F800000);
                            }
                            const float2 sc = m_sc[mi * 8 + 2 * c + h];
                            mx = fmaxf(mx, fmaf(most_of(z), sc.x * qc, sc.y));
                        }
                    }
                    if (any_of_rows(live && mx > m + S::kSlack)) move(mx);
                }
                uint32_t o[S::TWO ? 16 : CW / 2];
#pragma unroll 1
                for (int turn = 0; !idle; ++turn) {
                    uint32_t s[2][CH];
                    auto fetch = [&](int c) {
                        if constexpr (CH == 16) tmem_ld16(sat + half * CW + CH * c, s[c & 1]);
                        else ld32(sat + half * CW + CH * c, s[c & 1]);
                    };
                    fetch(0);
                    if (CW / CH == 2) fetch(1);
                    float2 sum = make_float2(0.f, 0.f), sum2 = make_float2(0.f, 0.f);
                    float mx = -__int_as_float(0x7F800000);   // the row's largest score (in bits; fp16: with the value scale)
#pragma unroll
                    for (int c = 0; c < CW / CH; ++c) {
                        if (c == 0 || CW / CH > 2) tmem_ld_wait();
                        if (CW / CH > 2 && c + 1 < CW / CH) fetch(c + 1);
#pragma unroll
                        for (int h = 0; h < CH / 16; ++h) {
                            float* z = reinterpret_cast<float*>(s[c & 1]) + 16 * h;
                            const int at = c * CH + 16 * h;     // of this thread's positions
                            if (!whole) {
                                const uint32_t on = bits[at >> 5] >> (at & 31);
#pragma unroll
                                for (int i = 0; i < 16; ++i) z[i] = on >> i & 1u ? z[i] : -__int_as_float(0x7F800000);
                            }
                            float x = S::SUMS || S::TWO ? 0.f : most_of(z);
                            float2 cm = make_float2(qc, qc), ca = make_float2(-m, -m), part = make_float2(0.f, 0.f);
                            float un = 1.f;
                            if (E4M3) {
                                const float2 sc = m_sc[mi * 8 + half * (CW / 16) + (at >> 4)];
                                cm.x = cm.y = sc.x * qc;
                                ca.x = ca.y = sc.y + S::kBias - m;
                                un = ex2(-sc.y);   // the sum goes without the value scale
                                x = fmaf(x, cm.x, sc.y);
                            }
                            if (!S::SUMS) mx = fmaxf(mx, x);
#pragma unroll
                            for (int i = 0; i < 16; i += 2) {
                                float2 e = fma2(make_float2(z[i], z[i + 1]), cm, ca);
                                e.x = ex2(e.x);
                                e.y = ex2(e.y);
                                if (E4M3) part = add2(part, e);
                                else if (i & 2) sum2 = add2(sum2, e);
                                else sum = add2(sum, e);
                                o[(at + i) >> 1 & (S::TWO ? 15 : CW / 2 - 1)] = E4M3 ? pack_f16(e.x, e.y) : pack_bf16(e.x, e.y);
                            }
                            if (E4M3) sum = fma2(part, make_float2(un, un), sum);
                            // over scores that have been read: the columns in front of these
                            if constexpr (S::TWO)
                                if (at & 16) st16(sat + half * (CW / 2) + (at >> 1) - 8, o);
                        }
                    }
                    const float all = (sum.x + sum.y) + (sum2.x + sum2.y);
                    if (S::TWO) {
                        l += all;
                        break;
                    }
                    if (!S::SUMS && !E4M3) mx *= qc;
                    // (with two threads a row the vote says also that both have read their scores)
                    const bool over = any_of_rows(live && (S::SUMS ? all > S::kMost : mx > m + S::kSlack));
                    if (turn > 0 || !over) {
                        l += all;
                        break;
                    }
                    if (S::SUMS)
#pragma unroll
                        for (int c = 0; c < CW / 16; ++c) {
                            uint32_t v[16];
                            tmem_ld16(sat + half * CW + 16 * c, v);
                            tmem_ld_wait();
                            const uint32_t on = bits[c >> 1] >> (16 * (c & 1));
                            float x = -__int_as_float(0x7F800000);
#pragma unroll
                            for (int i = 0; i < 16; ++i) x = fmaxf(x, on >> i & 1u ? __uint_as_float(v[i]) : -__int_as_float(0x7F800000));
                            mx = fmaxf(mx, x * qc);
                        }
                    move(mx);
                }
                if (idle) {
                    if (NH == 2) pair_barrier(1 + q * 4 + (warp & 3));   // (both have read: the first reference)
#pragma unroll
                    for (int i = 0; i < (S::TWO ? 16 : CW / 2); ++i) o[i] = 0u;
                    if constexpr (S::TWO)
                        for (int i = 0; i < CW / 32; ++i) st16(sat + half * (CW / 2) + 16 * i, o);
                }
                none = false;
                if (SHARED) touched = touched || mine;
                if constexpr (!S::TWO)
#pragma unroll
                    for (int i = 0; i < CW / 64; ++i)   // over the scores
                        st32(sat + half * (CW / 2) + 32 * i, *reinterpret_cast<const uint32_t(*)[32]>(o + 32 * i));
                bool zeroed = false;
                if (!whole && q == zq && half == 0) {
                    // value rows that no row of the item attends may hold anything: zero
                    // them (this thread's position; a weight of zero would make a NaN of it)
                    const int pos = t0 + row;
                    const uint32_t word = reinterpret_cast<const uint32_t*>(m_bits + mi)[row >> 5];
                    const bool any = (word >> (row & 31) & 1u) && pos >= p.k.lo && pos < flag.w &&
                                     (a.c.window == 0 || pos > p.it.p_first - a.c.window || pos < a.c.sink);
                    if (!__all_sync(0xffffffffu, any)) {
                        const unsigned v = g0 + S::v_at(k, p.n);
                        meet(full + v % (unsigned)NS, (v / (unsigned)NS) & 1);
                        if (!any) {
                            unsigned char* at = ring + (size_t)(v % (unsigned)NS) * S::SLOTB;
#pragma unroll 1
                            for (int c = 0; c < S::VD / 64; ++c)
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    *reinterpret_cast<uint4*>(at + c * kPosTile * 128 + swz128(row, i)) = make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        zeroed = true;
                    }
                }
                st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (zeroed) arrive_lead<CG>(p_full + buf);
                    else arrive_lead_relaxed<CG>(p_full + buf);
                    if (CG == 1) mbar_arrive(mfree + mi);
                }
                ++tc;
            }
            g0 += 2 * p.n;
            if (none) {                                      // nothing of this row tile
                more_pieces = p.next(t);
                continue;
            }
            // ---- the accumulator ----
            if (NH == 2) l += others(l);
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const bool out = !SHARED && p.slot == 0;        // the row's whole result
            const long long orow = ((long long)p.k.row0 + tok) * a.Hq + p.g * a.G + r - tok * a.G;   // (sequences)
            uint16_t* dst = reinterpret_cast<uint16_t*>(a.out) + orow * HD + half * (HD / NH);
            float* part = nullptr;
            const bool keep = live && (!SHARED || touched);
            if (!out && keep) {
                if (SHARED && p.slot == 0) {
                    const long long at = p.k.q_row + (long long)p.g * p.k.q_stride + r + (p.k.kind == kPrefix ? 0 : (long long)a.B * a.M * a.Hq);
                    part = t.dense + at * HD + half * (HD / NH);
                    if (half == 0) t.dense_ml[at] = make_float2(m, l);
                } else {
                    const long long at = (2ll * me + p.slot - 1) * kRowTile + ofs + row;
                    part = t.part + at * HD + half * (HD / NH);
                    if (half == 0) t.part_ml[at] = make_float2(m, l);
                }
            }
            more_pieces = p.next(t);                         // while the last product runs
            meet_values(tc - 1);
            float odd[4] = {0.f, 0.f, 0.f, 0.f};             // NaN: the product left something that is not finite
#pragma unroll 1
            for (int c = 0; c < HD / NH; c += 32) {
                uint32_t v[32];
                ld32(oat + c, v);
                tmem_ld_wait();
                if (!keep) {
                } else if (out) {
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float x = __uint_as_float(v[i]) * inv, y = __uint_as_float(v[i + 1]) * inv;
                        odd[i >> 1 & 3] = fmaf(x, 0.f, fmaf(y, 0.f, odd[i >> 1 & 3]));
                        w[i >> 1] = pack_bf16(x, y);
                    }
                    if (sectors) {
                        store_32b(dst + c, w);
                        store_32b(dst + c + 16, w + 8);
                    } else {
                        store_2x16b(dst + c, w);
                        store_2x16b(dst + c + 16, w + 8);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i += 8) store_32b(part + c + i, v + i);
                }
                __syncwarp();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_lead_relaxed<CG>(o_free + q);
            if (!SHARED && live) t.odd[half * t.odd_plane + orow] = out && !((odd[0] + odd[1]) + (odd[2] + odd[3]) == 0.f);
        }
    }
    __syncthreads();
    if (tid == 0) t.cta_status[blockIdx.x] = s_abort ? MTP_ERR_TIMEOUT : s_bad ? MTP_ERR_ARG : MTP_OK;
    if (CG == 2) pair_sync();   // nothing of the peer's is on its way here
    if (warp == S::MMA) free_columns<CG>(tmem, 512);
}

template <bool E4M3, int HD, bool SHARED>
cudaError_t go(const RowsTcParams& p, cudaStream_t s) {
    using S = RowShape<E4M3, HD, SHARED>;
    static int ready[64] = {0};   // the attribute is set, per device
    constexpr int base = rows_slots(E4M3, HD) * S::SLOTB + S::NQ * S::QB + rows_raw(E4M3, HD) * S::RAWB + kRowsOther;
    static_assert(base + rows_tables(MTP_MAX_PAGED_BATCH) <= kRowsSmemLimit, "shared memory");
    const int smem = base + (p.t.a.n_groups > 0 ? rows_tables(p.t.a.B) : 0);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || ready[dev] == 0) {
        e = cudaFuncSetAttribute(rows_tc_kernel<E4M3, HD, SHARED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowsSmemLimit);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) ready[dev] = 1;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.t.workers * S::CG));
    cfg.blockDim = dim3(S::THREADS);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // set up while the kernel before it ends
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = S::CG;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = S::CG == 1 ? 1 : 2;
    return cudaLaunchKernelEx(&cfg, rows_tc_kernel<E4M3, HD, SHARED>, p);
}

}  // namespace

#ifdef MTP_PAGED_E4M3
#define MTP_ROWS_FORMAT e4m3
constexpr bool kE4m3 = true;
#else
#define MTP_ROWS_FORMAT bf16
constexpr bool kE4m3 = false;
#endif
#ifdef MTP_ROWS_SHARED
#define MTP_ROWS_NAME(f) MTP_ROWS_NAME_(f, _shared)
constexpr bool kShared = true;
#else
#define MTP_ROWS_NAME(f) MTP_ROWS_NAME_(f, )
constexpr bool kShared = false;
#endif
#define MTP_ROWS_NAME_(f, s) launch_rows_tc_##f##s
#define MTP_ROWS_LAUNCH(f) MTP_ROWS_NAME(f)

cudaError_t MTP_ROWS_LAUNCH(MTP_ROWS_FORMAT)(const RowsTcParams& p, cudaStream_t s) {
    switch (p.t.a.hd) {
    case 64: return go<kE4m3, 64, kShared>(p, s);
    case 128: return go<kE4m3, 128, kShared>(p, s);
    case 256: return go<kE4m3, 256, kShared>(p, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace mtp
