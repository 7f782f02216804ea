// paged.cuh -- argument blocks, launchers and row helpers of the paged KV
// cache's append and attention kernels (internal).
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace mtp {

// The paged cache as the kernels take it (see mtp_kv_cache).
struct PagedKV {
    void *k, *v;
    float *ks, *vs;            // e4m3: scale of (page, KV head)
    const int32_t* table;      // [B, max_pages]
    long long sp, sh, st;      // strides of page, KV head, slot (elements)
    int n_pages, ps_log2, max_pages, Hkv;
    int window, sink;
};

// Turns (angle / 2 pi) per position of the rotation pair i, as a sum of two
// floats (48 bits): theta^(-2 i / hd) / (2 pi).  Rounded to one float, a
// position of 10^5 would already be 10^-2 radians off.
struct RopeTab {
    float hi[256], lo[256];
    int on;
};

// ---------------------------------------------------------------------------
// a row in units: thread c of a row's hd/16 threads holds the dimensions
// [8c, 8c + 8) in a and [hd/2 + 8c, hd/2 + 8c + 8) in b -- the rotation's
// pairs (i, i + hd/2) meet in one thread, and each half is a 16-byte load of
// bf16
// ---------------------------------------------------------------------------
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
    const uint4 u = ld_stream16(p), w = ld_stream16(p + 4);
    x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y); x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
    x[4] = __uint_as_float(w.x); x[5] = __uint_as_float(w.y); x[6] = __uint_as_float(w.z); x[7] = __uint_as_float(w.w);
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&x)[8]) {
    const uint4 u = ld_stream16(p);
    x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x); x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
    x[4] = bf16_lo(u.z); x[5] = bf16_hi(u.z); x[6] = bf16_lo(u.w); x[7] = bf16_hi(u.w);
}
__device__ __forceinline__ void open_unit(const uint4& u, float (&x)[8]) {
    x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x); x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
    x[4] = bf16_lo(u.z); x[5] = bf16_hi(u.z); x[6] = bf16_lo(u.w); x[7] = bf16_hi(u.w);
}
// two floats rounded to bf16 (nearest even), lo in the low half
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// RMSNorm of a row spread over U = hd/16 consecutive lanes (a power of two;
// every lane of the warp takes part); unit_norm_staged: the gains in 16-byte
// aligned (shared) memory
__device__ __forceinline__ float unit_rms(const float (&a)[8], const float (&b)[8], int hd, float eps) {
    float s = 0.f, t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        s = fmaf(a[i], a[i], s);
        t = fmaf(b[i], b[i], t);
    }
    s += t;
    for (int o = hd >> 5; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return rsqrtf(fmaf(s, __uint_as_float((uint32_t)(127 - (31 - __clz(hd))) << 23), eps));   // 1 / hd is a power of two
}
__device__ __forceinline__ void unit_norm(float (&a)[8], float (&b)[8], const float* gain, int c, int hd, float eps) {
    const float r = unit_rms(a, b, hd, eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a[i] = a[i] * r * __ldg(gain + 8 * c + i);
        b[i] = b[i] * r * __ldg(gain + (hd >> 1) + 8 * c + i);
    }
}
__device__ __forceinline__ void unit_norm_staged(float (&a)[8], float (&b)[8], const float* gain, int c, int hd, float eps) {
    const float r = unit_rms(a, b, hd, eps);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float4 g = *reinterpret_cast<const float4*>(gain + 8 * c + 4 * h);
        const float4 k = *reinterpret_cast<const float4*>(gain + (hd >> 1) + 8 * c + 4 * h);
        a[4 * h] *= r * g.x; a[4 * h + 1] *= r * g.y; a[4 * h + 2] *= r * g.z; a[4 * h + 3] *= r * g.w;
        b[4 * h] *= r * k.x; b[4 * h + 1] *= r * k.y; b[4 * h + 2] *= r * k.z; b[4 * h + 3] *= r * k.w;
    }
}

// cos and sin of the unit's 8 pairs at position pos.  pos = 4096 ph + pl; each
// product with the table's high part is split exactly by an fma, whole turns
// are dropped, and what the remaining fp32 sum cannot hold turns the result
// by a first-order correction -- the angle keeps about 2^-45 of its size plus
// 2^-40 turns, so only the rounding of cos and sin themselves is left.
// FAST: the sine and cosine instructions (2^-20), for rows that round to 16
// bits or fewer right after.
template <bool FAST>
__device__ __forceinline__ void pair_angle(float pl, float ph, float h, float l, float& cs, float& sn) {
    float x = __fmul_rn(pl, h), y = __fmul_rn(ph, h);   // (no contraction: the products' own roundings are wanted)
    float e = fmaf(pl, h, -x) + fmaf(ph, h, -y);
    x -= rintf(x);
    y -= rintf(y);
    float s = x + y;
    const float z = s - x;
    e += (x - (s - z)) + (y - z);      // the rounding of x + y
    s -= rintf(s);
    e = fmaf(ph + pl, l, e);           // up to 2^-7 turns at positions of 2^19: most of it joins s
    const float t = s + e;
    e -= t - s;
    s = t;
    if (FAST) {
        s -= rintf(s);
        const float r = 6.2831853f * s;
        asm("sin.approx.f32 %0, %1;" : "=f"(sn) : "f"(r));
        asm("cos.approx.f32 %0, %1;" : "=f"(cs) : "f"(r));
    } else {
        float sv, cv;
        sincospif(2.f * s, &sv, &cv);
        const float d = 6.2831853f * e;
        cs = fmaf(-sv, d, cv);
        sn = fmaf(cv, d, sv);
    }
}
__device__ __forceinline__ void split_pos(long long pos, float& pl, float& ph) {
    pl = (float)(int)(pos & 4095);
    ph = (float)(int)(pos >> 12) * 4096.f;
}
// hi, lo: the table's 8 entries of this unit
template <bool FAST>
__device__ __forceinline__ void unit_angles(long long pos, const float* hi, const float* lo, float (&cs)[8], float (&sn)[8]) {
    float pl, ph;
    split_pos(pos, pl, ph);
#pragma unroll
    for (int i = 0; i < 8; ++i) pair_angle<FAST>(pl, ph, hi[i], lo[i], cs[i], sn[i]);
}
__device__ __forceinline__ void unit_rotate(float (&a)[8], float (&b)[8], const float (&cs)[8], const float (&sn)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = a[i], y = b[i];
        a[i] = fmaf(x, cs[i], -y * sn[i]);
        b[i] = fmaf(y, cs[i], x * sn[i]);
    }
}

// A sequence's lengths are usable: 0 <= len, 0 <= n <= M, len + n <= the
// positions its table row can map.
__device__ __forceinline__ bool seq_ok(int len, int n, int M, const PagedKV& c) {
    return len >= 0 && n >= 0 && n <= M && (long long)len + n <= (long long)c.max_pages << c.ps_log2;
}

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
struct AppendArgs {
    PagedKV c;
    int hd, B, M;
    const int32_t *kv_len, *n_new;
    const void *k, *v;
    long long sb, sm, sh;      // input strides (elements)
    const float* k_norm;
    float eps;
    WsHeader* hdr;
    RopeTab rope;
    int hpt;                   // KV heads per thread (fp32 / bf16 caches; set by the launcher)
};
cudaError_t launch_kv_append(const AppendArgs& a, int in_dtype, int kv_dtype, int sms, cudaStream_t s);

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------
// An item is (sequence, KV head, row tile): RT of the sequence's n * G
// rows (row r: new row r / G, query head r % G of the group) against its
// attended positions in tiles of `tile` positions.  The items lie end to end,
// sequence-major, each as `open` units (what it costs a CTA to begin an item:
// its queries, an epilogue, and a pipeline that fills anew) and one unit a
// tile; T units in all.  CTA c takes the units [T c / grid, T (c + 1) / grid),
// so ragged lengths cost the same on every CTA.  A segment is the part of one
// item's tiles inside one CTA's range.  A whole item is written out directly;
// a part is left as (o, m, l) in slot 2c if it begins inside the item (at most
// the CTA's first) and in 2c + 1 if it only ends there (at most its last), and
// a second kernel merges the parts.
struct PagedAttnArgs {
    PagedKV c;
    int hd, B, M, Hq, G;
    const int32_t *kv_len, *n_new;
    const void* q;
    long long sb, sm, sh;
    const float* q_norm;
    float eps, scale;          // scale: attn_scale * log2(e) (scores are in bits)
    void* out;
    WsHeader* hdr;
    int* cta_status;           // [grid]: MTP_OK or an error, written by every CTA
    // For the merge, [grid]: an item that begins in one CTA's share and ends in
    // another's: KV head, first row | rows << 16, first CTA, last CTA (-1: none).
    // Entry c is CTA c's (at most one item begins in its share and ends behind
    // it), or, where there are no more items than CTAs, every item has its own.
    int4* split;
    int by_item, rows_max;     // that, and rows of an item at most (min(RT, M G))
    float* part;               // [2 grid] slots of RT * (hd + 2) floats
    int RT, rt_log2, tile_log2, grid;
    int open_max;              // units before an item's tiles at most
    unsigned long long timeout_ns;
    RopeTab rope;
};

// An e4m3 page's scale is one that the attention takes: a power of two within
// [2^-40, 2^40].  The tensor cores fold the value scale's exponent into the
// scores, so any other would be computed wrongly there.
__device__ __forceinline__ bool scale_ok(float s) {
    const uint32_t u = __float_as_uint(s);
    return (u & 0x7FFFFFu) == 0u && u >= (127u - 40u) << 23 && u <= (127u + 40u) << 23;
}

// attended tiles of a sequence: tiles [0, st) (the sink) and [lt, et)
struct TileMap { int st, lt, n; };
__device__ __forceinline__ TileMap tile_map(const PagedAttnArgs& a, int len, int n) {
    TileMap m = {0, 0, 0};
    if (n <= 0) return m;
    const int et = (len + n - 1 >> a.tile_log2) + 1;
    if (a.c.window > 0) {
        const int lo = len + 1 > a.c.window ? len + 1 - a.c.window : 0;             // the first row's window
        const int hi = len + n > a.c.window ? len + n - a.c.window : 0;             // the last row's
        m.lt = lo >> a.tile_log2;
        const int sk = a.c.sink < hi ? a.c.sink : hi;
        m.st = sk > 0 ? (sk - 1 >> a.tile_log2) + 1 : 0;
        if (m.st > m.lt) m.st = m.lt;
    }
    m.n = m.st + et - m.lt;
    return m;
}
__device__ __forceinline__ int tile_at(const TileMap& m, int k) { return k < m.st ? k : m.lt + (k - m.st); }
// position t is attended by the row at position p
__device__ __forceinline__ bool attends(const PagedKV& c, int t, int p) {
    return t <= p && (c.window == 0 || t > p - c.window || t < c.sink);
}

// row tiles that hold rows of a sequence with n new ones
__device__ __forceinline__ int row_tiles(const PagedAttnArgs& a, int n) { return (n * a.G + a.RT - 1) >> a.rt_log2; }

// What a CTA keeps of the call's sequences in shared memory.
struct Plan {
    long long* pre;            // [B + 1] units before a sequence
    int2* len;                 // [B] kv_len, n_new
    int open;                  // units before an item's tiles
};
__host__ __device__ constexpr int plan_bytes(int B) { return (2 * B + 1) * 8; }
constexpr int kPlanTmp = 2 * 16;   // two words a warp

// Fills the plan (tmp: shared, kPlanTmp); false for this thread if it saw
// lengths that are out of range.
template <int THREADS>
__device__ __forceinline__ bool schedule(const PagedAttnArgs& a, Plan& plan, long long* tmp) {
    static_assert(THREADS <= 512, "kPlanTmp");
    const int per = (a.B + THREADS - 1) / THREADS, b0 = (int)threadIdx.x * per;
    const int b1 = b0 + per < a.B ? b0 + per : a.B;
    long long* pre = plan.pre;
    auto items = [&](int2 l) { return (long long)row_tiles(a, l.y) * a.c.Hkv; };
    long long sum = 0, its = 0;   // tiles and items
    bool good = true;
    for (int b = b0; b < b1; ++b) {
        int2 l = make_int2(a.kv_len[b], a.n_new ? a.n_new[b] : a.M);
        if (!seq_ok(l.x, l.y, a.M, a.c)) {
            l = make_int2(0, 0);   // left out
            good = false;
        }
        plan.len[b] = l;
        sum += tile_map(a, l.x, l.y).n * items(l);
        its += items(l);
    }
    long long inc = sum, itc = its;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, inc, o);
        const long long w = __shfl_up_sync(0xffffffffu, itc, o);
        if (lane >= o) {
            inc += v;
            itc += w;
        }
    }
    if (lane == 31) {
        tmp[warp] = inc;
        tmp[16 + warp] = itc;
    }
    __syncthreads();
    long long base = inc - sum, all = 0;
    itc -= its;
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) {
            base += tmp[w];
            itc += tmp[16 + w];
        }
        all += tmp[w];
    }
    // where a share is few tiles, how they spread counts for more
    plan.open = a.open_max;
    while (plan.open > 0 && 2ll * plan.open * a.grid > all) --plan.open;
    base += plan.open * itc;
    for (int b = b0; b < b1; ++b) {
        const int2 l = plan.len[b];
        pre[b] = base;
        base += (plan.open + tile_map(a, l.x, l.y).n) * items(l);
        if (b == a.B - 1) pre[a.B] = base;
    }
    __syncthreads();
    return good;
}
// a / b; small numbers by one approximate division and a correction (an
// integer division is some 20 dependent instructions)
__device__ __forceinline__ unsigned udiv(unsigned a, unsigned b) {
    if (a >= 1u << 20) return a / b;
    unsigned q = (unsigned)__fdividef((float)a, (float)b);   // off by one at most
    const int r = (int)(a - q * b);
    q += r < 0 ? -1 : r >= (int)b ? 1 : 0;
    return q;
}
// first unit of CTA c's share, and the CTA whose share holds unit x.  With
// fewer units than CTAs the first T CTAs take one each.  So every CTA between
// the first and the last that hold tiles of an item holds one too: the merge
// reads written slots only.
__device__ __forceinline__ long long share_lo(long long T, int c, int grid) {
    if (T < grid) return c < T ? c : T;
    if (T < (1ll << 31) / (grid + 1)) return udiv((unsigned)T * (unsigned)c, (unsigned)grid);   // (a 64-bit division is slower still)
    return T * c / grid;
}
__device__ __forceinline__ int share_of(long long T, long long x, int grid) {
    if (T < grid) return (int)x;
    if (T < (1ll << 31) / (grid + 1)) return (int)udiv((unsigned)(x + 1) * (unsigned)grid - 1u, (unsigned)T);
    return (int)(((x + 1) * grid - 1) / T);
}

struct Segment {
    int b, g, rt;              // sequence, KV head, row tile
    int t0, n;                 // the item's tiles [t0, t0 + n)
    int len, n_new;            // of the sequence
    int rows, slot;            // rows of this tile, partial slot (-1: whole item)
    long long x, next;         // unit of its first tile, and where the one behind it begins
    TileMap map;
};
// CTA c's segment at x of its range [.., xe); n <= 0 if the range ends before
// its first tile (only where the whole range lies before an item's tiles)
__device__ __forceinline__ Segment segment_at(const PagedAttnArgs& a, const Plan& plan, long long x, long long xe, int c) {
    Segment s;
    int b = 0;
    for (int hi = a.B - 1; b < hi;) {   // the last b with pre[b] <= x
        const int mid = (b + hi + 1) >> 1;
        if (plan.pre[mid] <= x) b = mid;
        else hi = mid - 1;
    }
    const int2 l = plan.len[b];
    s.b = b;
    s.len = l.x;
    s.n_new = l.y;
    s.map = tile_map(a, l.x, l.y);
    const long long rel = x - plan.pre[b];
    const unsigned units = (unsigned)(plan.open + s.map.n);
    const unsigned item = rel < (1ll << 31) ? udiv((unsigned)rel, units) : (unsigned)(rel / units);
    s.t0 = (int)(rel - (long long)item * units) - plan.open;
    s.x = x;
    if (s.t0 < 0) {
        s.x -= s.t0;
        s.t0 = 0;
    }
    const unsigned nrt = (unsigned)row_tiles(a, l.y);
    s.g = (int)udiv(item, nrt);
    s.rt = (int)(item - s.g * nrt);
    const long long left = xe - s.x;
    s.n = s.map.n - s.t0 < left ? s.map.n - s.t0 : (int)left;
    s.next = s.x + s.n + (s.t0 + s.n == s.map.n ? plan.open : 0);
    const int R = l.y * a.G - s.rt * a.RT;
    s.rows = R < a.RT ? R : a.RT;
    s.slot = s.t0 > 0 ? 2 * c : (s.n < s.map.n ? 2 * c + 1 : -1);
    return s;
}

// row tiles that an item index counts for every sequence and KV head
__device__ __forceinline__ int item_tiles(const PagedAttnArgs& a) { return (a.M * a.G + a.RT - 1) >> a.rt_log2; }
// what CTA c notes for an item whose tiles begin in its share (one thread;
// `mine`: its own entry, written at its end)
__device__ __forceinline__ void note_split(const PagedAttnArgs& a, const Segment& s, long long T, int c, int4& mine) {
    if (s.t0 != 0) return;
    int4 r = make_int4(0, 0, 0, -1);
    if (s.slot >= 0) r = make_int4(s.b * a.c.Hkv + s.g, s.rt * a.RT | s.rows << 16, c, share_of(T, s.x + s.map.n - 1, a.grid));
    if (a.by_item) a.split[(s.b * a.c.Hkv + s.g) * item_tiles(a) + s.rt] = r;
    else if (s.slot >= 0) mine = r;
}

// The running maximum of a row that has attended nothing: below every score of
// an attended position, and finite, so that no difference from it is a NaN.
constexpr float kNoScore = -3.402823466e38f;

// floats of one partial slot
__host__ __device__ constexpr long long part_floats(int RT, int hd) { return (long long)RT * (hd + 2); }

constexpr int kCcTileLog2 = 5, kCcTile = 1 << kCcTileLog2, kCcRows = 16;   // positions and rows of a tile on the CUDA cores

cudaError_t launch_paged_attn_cc(const PagedAttnArgs& a, int dtype, int kv_dtype, cudaStream_t s);
cudaError_t launch_paged_merge(const PagedAttnArgs& a, int dtype, cudaStream_t s);

}  // namespace mtp
