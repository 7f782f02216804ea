// kv_append.cu -- new key and value rows into a paged KV cache: RMSNorm and
// rotation of the keys, one rounding to the cache's type.
//
// key = rope(rmsnorm(k), p), value = v.  Long calls are bound by the bytes in
// and out or by the instructions of an element (norm, angle, maximum,
// rounding), small ones by the launch and two dependent loads, the length and
// then the page.
#include "paged.cuh"

#include <cuda_fp8.h>

namespace mtp {

// The call's status, by one CTA that looks at every length and every page the
// rows go to (the other CTAs leave bad ones out without a word: no order
// between CTAs and no zeroing launch is needed).
__device__ void append_status(const AppendArgs& a) {
    bool bad = false;
    const int ps = 1 << a.c.ps_log2, nt = (a.M + ps - 2) / ps + 1;
    for (long long i = threadIdx.x; i < (long long)a.B * nt; i += blockDim.x) {
        const int b = (int)(i / nt), len = a.kv_len[b], n = a.n_new ? a.n_new[b] : a.M;
        if (!seq_ok(len, n, a.M, a.c)) {
            bad = true;
            continue;
        }
        const int p = (len >> a.c.ps_log2) + (int)(i % nt);
        if (n == 0 || (long long)p << a.c.ps_log2 >= (long long)len + n) continue;
        const int pg = a.c.table[(long long)b * a.c.max_pages + p];
        bad = bad || (unsigned)pg >= (unsigned)a.c.n_pages;
    }
    const int any = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
        a.hdr->status = any ? MTP_ERR_ARG : MTP_OK;
        a.hdr->barrier = 0;
        a.hdr->done = 0;
    }
}

// ---------------------------------------------------------------------------
// fp32 and bf16 caches: a thread takes one unit (16 elements) of `hpt` KV
// heads of one row, so that the angles of a row are computed once for those
// heads; gridDim.y: keys and values of every sequence.
// One sequence, 8191 rows x 8 heads of 128, fp32 to bf16 (101 MB): 19.8 us, 5.1
// TB/s (bound by the bytes; a copy takes 14.9).  One sequence, 4 rows x 4 heads
// of 256, bf16: 3.5 us.
// ---------------------------------------------------------------------------
template <typename IT, typename CT>
__global__ void __launch_bounds__(128) append_rows_kernel(const __grid_constant__ AppendArgs a) {
    __shared__ __align__(16) float s_hi[256], s_lo[256], s_gain[512];
    if (blockIdx.x == gridDim.x - 1) {
        if (blockIdx.y == 0) append_status(a);
        return;
    }
    const int b = blockIdx.y >> 1, ulog = 31 - __clz(a.hd >> 4), groups = a.c.Hkv / a.hpt;
    const bool key = (blockIdx.y & 1) == 0, rot = key && a.rope.on, nrm = key && a.k_norm;
    const int len = a.kv_len[b], n = a.n_new ? a.n_new[b] : a.M;
    if (!seq_ok(len, n, a.M, a.c)) return;
    const unsigned x = blockIdx.x * blockDim.x + threadIdx.x, t = x >> ulog;
    const int c = (int)(x & ((1u << ulog) - 1u));
    int j = groups == 1 ? (int)t : (int)(t / (unsigned)groups);
    if ((groups == 1 ? (blockIdx.x * blockDim.x) >> ulog : ((blockIdx.x * blockDim.x) >> ulog) / (unsigned)groups) >= (unsigned)n) return;
    const int g0 = ((int)t - j * groups) * a.hpt;
    if (rot)   // lanes read the tables at different places, which parameters serve one by one
        for (int i = threadIdx.x; i < a.hd >> 1; i += blockDim.x) {
            s_hi[i] = a.rope.hi[i];
            s_lo[i] = a.rope.lo[i];
        }
    if (nrm)
        for (int i = threadIdx.x; i < a.hd; i += blockDim.x) s_gain[i] = a.k_norm[i];
    if (rot || nrm) __syncthreads();
    const bool live = j < n;
    if (!live) j = n - 1;
    const IT* src = reinterpret_cast<const IT*>(key ? a.k : a.v) + b * a.sb + j * a.sm + g0 * a.sh + 8 * c;
    const long long pos = (long long)len + j;
    CT* dst = nullptr;
    if (live) {
        const int pg = a.c.table[(long long)b * a.c.max_pages + (int)(pos >> a.c.ps_log2)];
        if ((unsigned)pg < (unsigned)a.c.n_pages)
            dst = reinterpret_cast<CT*>(key ? a.c.k : a.c.v) + pg * a.c.sp + (pos & ((1 << a.c.ps_log2) - 1)) * a.c.st +
                  g0 * a.c.sh + 8 * c;
    }
    float cs[8], sn[8];
    if (rot) unit_angles<false>(pos, s_hi + 8 * c, s_lo + 8 * c, cs, sn);
#pragma unroll 4
    for (int h = 0; h < a.hpt; ++h) {
        float p[8], q[8];
        load8(src + h * a.sh, p);
        load8(src + h * a.sh + (a.hd >> 1), q);
        if (nrm) unit_norm_staged(p, q, s_gain, c, a.hd, a.eps);
        if (rot) unit_rotate(p, q, cs, sn);
        if (dst) {
            store8(dst + h * a.c.sh, p);
            store8(dst + h * a.c.sh + (a.hd >> 1), q);
        }
    }
}

// ---------------------------------------------------------------------------
// e4m3 cache: a CTA takes the new rows of one (sequence, page, KV head, key or
// value), because they share one scale
// ---------------------------------------------------------------------------

// smallest k with amax <= 448 * 2^k (448 = 1.75 * 2^8), within [-40, 40]
__device__ __forceinline__ int e4m3_exponent(float amax) {
    if (!(amax > 0.f)) return -40;
    const uint32_t u = __float_as_uint(amax);
    const int k = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);   // subnormals end below -40
    return k < -40 ? -40 : (k > 40 ? 40 : k);
}
__device__ __forceinline__ float pow2i(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }
// The largest finite magnitude of a unit.  fmaxf passes NaN over; an infinity
// shows in the result, and only then the values are looked at one by one.
__device__ __forceinline__ float unit_amax(const float (&p)[8], const float (&q)[8], bool finite_only) {
    float m = 0.f, n = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float x = fabsf(p[e]), y = fabsf(q[e]);
        m = fmaxf(m, finite_only && x > 3.402823466e38f ? 0.f : x);
        n = fmaxf(n, finite_only && y > 3.402823466e38f ? 0.f : y);
    }
    return fmaxf(m, n);
}
__device__ __forceinline__ bool is_inf(float x) { return x > 3.402823466e38f; }
// infinities to NaN (a unit of a page whose maximum showed one)
__device__ __forceinline__ void drop_inf(float (&p)[8], float (&q)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (is_inf(fabsf(p[e]))) p[e] = __uint_as_float(0x7FC00000u);
        if (is_inf(fabsf(q[e]))) q[e] = __uint_as_float(0x7FC00000u);
    }
}
// 8 values times inv as e4m3 codes (nearest even, saturating; NaN becomes NaN)
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t join16(uint32_t lo, uint32_t hi) { return __byte_perm(lo, hi, 0x5410); }
__device__ __forceinline__ uint2 pack_e4m3(const float (&x)[8], float inv) {
    return make_uint2(join16(e4m3x2(x[0] * inv, x[1] * inv), e4m3x2(x[2] * inv, x[3] * inv)),
                      join16(e4m3x2(x[4] * inv, x[5] * inv), e4m3x2(x[6] * inv, x[7] * inv)));
}

// The page's older codes, re-rounded to a scale that grew by 1/f.
__device__ __forceinline__ void reround(uint8_t* dst, long long st, int off, int ulog, float f) {
    for (int x = threadIdx.x; x < off << ulog; x += blockDim.x) {
        uint4* d = reinterpret_cast<uint4*>(dst + (x >> ulog) * st + 16 * (x & ((1 << ulog) - 1)));
        uint4 w = *d;
        uint32_t* ws = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t r = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const __half2_raw v = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(ws[i] >> (16 * h)), __NV_E4M3);
                float2 y = __half22float2(__half2(v));
                y.x *= f;
                y.y *= f;
                r |= (uint32_t)__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3) << (16 * h);
            }
            ws[i] = r;
        }
        *d = w;
    }
}

// Where the new rows of a (sequence, touched page) lie; false: nothing to do.
struct PageRows {
    int b, len, j0, j1, page, off;   // rows [j0, j1), slots [0, off) are the sequence's already
    long long first;                 // position of the page's slot 0
};
__device__ __forceinline__ bool page_rows(const AppendArgs& a, int nt, PageRows& r) {
    const int ps = 1 << a.c.ps_log2, it = blockIdx.x % nt;
    r.b = blockIdx.x / nt;
    r.len = a.kv_len[r.b];
    const int n = a.n_new ? a.n_new[r.b] : a.M;
    if (!seq_ok(r.len, n, a.M, a.c)) return false;
    const int pi = (r.len >> a.c.ps_log2) + it;
    r.first = (long long)pi << a.c.ps_log2;
    r.j0 = it == 0 ? 0 : (int)(r.first - r.len);
    r.j1 = r.first + ps - r.len < n ? (int)(r.first + ps - r.len) : n;
    if (r.j0 >= r.j1) return false;
    r.page = a.c.table[(long long)r.b * a.c.max_pages + pi];
    r.off = (int)(r.len + r.j0 - r.first);
    return (unsigned)r.page < (unsigned)a.c.n_pages;
}

// Few rows a page (decoding): a CTA takes one KV head; every thread's one unit
// stays in registers between the maximum and the rounding.  64 sequences x 3
// rows x 4 heads of 256: 4.7 us, all of it latency (launch, length, page, row,
// barrier).
template <typename IT>
__global__ void __launch_bounds__(256) append_e4m3_kernel(const __grid_constant__ AppendArgs a) {
    const int ps = 1 << a.c.ps_log2, nt = (a.M + ps - 2) / ps + 1;
    if (blockIdx.x == gridDim.x - 1) {
        if (blockIdx.y == 0 && blockIdx.z == 0) append_status(a);
        return;
    }
    __shared__ float red[8];
    PageRows w;
    if (!page_rows(a, nt, w)) return;
    const int g = blockIdx.y;
    const bool key = blockIdx.z == 0;
    float* sc = (key ? a.c.ks : a.c.vs) + (long long)w.page * a.c.Hkv + g;
    const float had = w.off > 0 ? *sc : 0.f;
    const int U = a.hd >> 4, ulog = 31 - __clz(U), units = (w.j1 - w.j0) << ulog;
    const IT* src = reinterpret_cast<const IT*>(key ? a.k : a.v) + w.b * a.sb + g * a.sh;
    uint8_t* dst = reinterpret_cast<uint8_t*>(key ? a.c.k : a.c.v) + w.page * a.c.sp + g * a.c.sh;
    const int x = threadIdx.x, c = x & (U - 1), j = w.j0 + (x < units ? x >> ulog : 0);
    float p[8], q[8];
    load8(src + j * a.sm + 8 * c, p);
    load8(src + j * a.sm + 8 * c + (a.hd >> 1), q);
    if (key && a.rope.on) {
        float cs[8], sn[8];
        unit_angles<false>((long long)w.len + j, a.rope.hi + 8 * c, a.rope.lo + 8 * c, cs, sn);
        if (a.k_norm) unit_norm(p, q, a.k_norm, c, a.hd, a.eps);
        unit_rotate(p, q, cs, sn);
    } else if (key && a.k_norm) {
        unit_norm(p, q, a.k_norm, c, a.hd, a.eps);
    }
    auto block_max = [&](float m) {
        m = warp_max(m);   // (threads without a unit hold the first row's again)
        __syncthreads();
        if ((x & 31) == 0) red[x >> 5] = m;
        __syncthreads();
        for (int i = 0; i < (int)(blockDim.x >> 5); ++i) m = fmaxf(m, red[i]);
        return m;
    };
    float m = block_max(unit_amax(p, q, false));
    const bool inf = is_inf(m);
    if (inf) {
        m = block_max(unit_amax(p, q, true));
        drop_inf(p, q);
    }
    const float now = fmaxf(pow2i(e4m3_exponent(m)), had), inv = 1.f / now;   // powers of two: exact
    if (x == 0) *sc = now;
    if (x < units) {
        uint8_t* d = dst + (w.off + (x >> ulog)) * a.c.st + 8 * c;
        *reinterpret_cast<uint2*>(d) = pack_e4m3(p, inv);
        *reinterpret_cast<uint2*>(d + (a.hd >> 1)) = pack_e4m3(q, inv);
    }
    if (had > 0.f && had != now) reround(dst, a.c.st, w.off, ulog, had * inv);
}

// Many rows a page (prompts): a CTA of up to 512 threads takes the keys or the
// values of a page for `hpt` KV heads after one another, a thread two units of
// them; the next head's rows are on their way while this one's are rounded, and
// the angles are computed once for all heads, slot s of the page as the product
// of the rotations by its 16-slot base and by s % 16 (20 sines a pair for a page
// of 64 instead of 64; the product costs the angle 3 u).  The norm's factor of
// a row only scales it, so it joins the maximum and the scale's inverse.  ONE:
// the page has at most 1024 units of a head, and they stay in registers between
// the maximum and the rounding; larger pages are read twice, the second time
// from L2.
// 8 sequences of up to 4096 rows x 4 heads of 256, bf16 in (a ragged batch of 104
// MB in and out): 44.6 us, 2.3 TB/s.  The 16 warps of an SM (123 registers a
// thread hold two units) bound it: they issue 46% of the time and wait at a
// barrier a head, on shared-memory tables and on each other's pipes.
constexpr int kPageThreads = 512;

template <typename IT> struct Raw { uint4 v[4 * sizeof(IT) / 4]; };   // a unit as loaded
__device__ __forceinline__ void raw_load(const uint16_t* p, int half, Raw<uint16_t>& r) {
    r.v[0] = ld_stream16(p);
    r.v[1] = ld_stream16(p + half);
}
__device__ __forceinline__ void raw_load(const float* p, int half, Raw<float>& r) {
    r.v[0] = ld_stream16(p);
    r.v[1] = ld_stream16(p + 4);
    r.v[2] = ld_stream16(p + half);
    r.v[3] = ld_stream16(p + half + 4);
}
__device__ __forceinline__ void raw_open(const Raw<uint16_t>& r, float (&p)[8], float (&q)[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint4 u = r.v[h];
        float* x = h ? q : p;
        x[0] = bf16_lo(u.x); x[1] = bf16_hi(u.x); x[2] = bf16_lo(u.y); x[3] = bf16_hi(u.y);
        x[4] = bf16_lo(u.z); x[5] = bf16_hi(u.z); x[6] = bf16_lo(u.w); x[7] = bf16_hi(u.w);
    }
}
__device__ __forceinline__ void raw_open(const Raw<float>& r, float (&p)[8], float (&q)[8]) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const uint4 u = r.v[h];
        float* x = (h < 2 ? p : q) + 4 * (h & 1);
        x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y); x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
    }
}

// gains, without the row's factor, which is returned
__device__ __forceinline__ float unit_gain(float (&a)[8], float (&b)[8], const float* gain, int c, int hd, float eps) {
    const float r = unit_rms(a, b, hd, eps);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float4 g = *reinterpret_cast<const float4*>(gain + 8 * c + 4 * h);
        const float4 k = *reinterpret_cast<const float4*>(gain + (hd >> 1) + 8 * c + 4 * h);
        a[4 * h] *= g.x; a[4 * h + 1] *= g.y; a[4 * h + 2] *= g.z; a[4 * h + 3] *= g.w;
        b[4 * h] *= k.x; b[4 * h + 1] *= k.y; b[4 * h + 2] *= k.z; b[4 * h + 3] *= k.w;
    }
    return r;
}

template <typename IT, bool ONE>
__global__ void __launch_bounds__(kPageThreads, 1) append_e4m3_pages_kernel(const __grid_constant__ AppendArgs a) {
    extern __shared__ __align__(16) float2 s_rot[];   // [ps / 16][hd / 2] bases, [16][hd / 2] steps
    __shared__ __align__(16) float s_gain[512];
    __shared__ unsigned red[2][32];
    const int ps = 1 << a.c.ps_log2, nt = (a.M + ps - 2) / ps + 1;
    if (blockIdx.x == gridDim.x - 1) {
        if (blockIdx.y == 0 && blockIdx.z == 0) append_status(a);
        return;
    }
    PageRows w;
    if (!page_rows(a, nt, w)) return;
    constexpr int UPT = 2;
    const bool key = blockIdx.z == 0, rot = key && a.rope.on, nrm = key && a.k_norm;
    const int tid = threadIdx.x, T = blockDim.x, lane = tid & 31, ulog = 27 - __clz(a.hd), half = a.hd >> 1;
    const int units = (w.j1 - w.j0) << ulog, g0 = blockIdx.y * a.hpt;
    const int c = tid & ((1 << ulog) - 1);   // the same for all of a thread's units
    const IT* src = reinterpret_cast<const IT*>(key ? a.k : a.v) + w.b * a.sb + w.j0 * a.sm + g0 * a.sh + 8 * c;
    uint8_t* dst = reinterpret_cast<uint8_t*>(key ? a.c.k : a.c.v) + w.page * a.c.sp + w.off * a.c.st + g0 * a.c.sh + 8 * c;
    float* scale = (key ? a.c.ks : a.c.vs) + (long long)w.page * a.c.Hkv + g0;
    auto row = [&](int x) { return x < units ? x >> ulog : 0; };
    const IT* from[UPT];   // the thread's units of this head, and where they go
    uint8_t* to[UPT];
    Raw<IT> raw[UPT];
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
        from[i] = src + row(tid + i * T) * a.sm;
        to[i] = tid + i * T < units ? dst + row(tid + i * T) * a.c.st : nullptr;
        raw_load(from[i], half, raw[i]);
    }
    if (nrm)
        for (int i = tid; i < a.hd; i += T) s_gain[i] = a.k_norm[i];
    const int nb = ps >> 4;
    if (rot) {
        // one pair a thread, whose table entries are read once; a second one where
        // there are fewer threads than pairs (head_dim 512, calls of 9 to 14 rows)
        const int step = T < half ? 1 : T / half;
        if (tid < step * half)
            for (int pr = tid & (half - 1); pr < half; pr += T) {
                const float hi = a.rope.hi[pr], lo = a.rope.lo[pr];
                for (int e = tid / half; e < nb + 16; e += step) {
                    float pl, ph;
                    split_pos(e < nb ? w.first + 16 * e : e - nb, pl, ph);
                    float2 r;
                    pair_angle<false>(pl, ph, hi, lo, r.x, r.y);
                    s_rot[e * half + pr] = r;
                }
            }
    }
    if (tid < 32) red[0][tid] = red[1][tid] = 0u;   // (warps that are not there)
    __syncthreads();
    auto angles = [&](int r, float (&cs)[8], float (&sn)[8]) {
        const int s = w.off + r;
        const float4* x = reinterpret_cast<const float4*>(s_rot + (s >> 4) * half + 8 * c);
        const float4* y = reinterpret_cast<const float4*>(s_rot + (nb + (s & 15)) * half + 8 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // two pairs a load
            const float4 u = x[i], v = y[i];
            cs[2 * i] = fmaf(u.x, v.x, -u.y * v.y);
            sn[2 * i] = fmaf(u.x, v.y, u.y * v.x);
            cs[2 * i + 1] = fmaf(u.z, v.z, -u.w * v.w);
            sn[2 * i + 1] = fmaf(u.z, v.w, u.w * v.z);
        }
    };
    float cs[ONE ? UPT : 1][8], sn[ONE ? UPT : 1][8];
    if (ONE && rot)
#pragma unroll
        for (int i = 0; i < UPT; ++i) angles(row(tid + i * T), cs[ONE ? i : 0], sn[ONE ? i : 0]);
    float p[UPT][8], q[UPT][8], f[UPT];   // a unit is f (p, q)
    auto turn = [&](int x, int i) {        // raw -> p, q, f
        raw_open(raw[i], p[i], q[i]);
        f[i] = 1.f;
        if (nrm) f[i] = unit_gain(p[i], q[i], s_gain, c, a.hd, a.eps);
        if (rot) {
            if (!ONE) angles(row(x), cs[0], sn[0]);
            unit_rotate(p[i], q[i], cs[ONE ? i : 0], sn[ONE ? i : 0]);
        }
    };
    // a unit's largest magnitude; its finite ones' where it is asked for
    auto unit_max = [&](int i, bool finite_only) { return unit_amax(p[i], q[i], finite_only) * f[i]; };
    int turns = 0;
    auto block_max = [&](float m) {   // (magnitudes order as their bits)
        const unsigned u = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
        if (lane == 0) red[turns & 1][tid >> 5] = u;
        __syncthreads();
        m = __uint_as_float(__reduce_max_sync(0xffffffffu, red[turns & 1][lane]));
        ++turns;
        return m;
    };
#pragma unroll 1
    for (int g = 0; g < a.hpt; ++g) {
        const float had = w.off > 0 ? scale[g] : 0.f;
        float m = 0.f;
        if (ONE) {
#pragma unroll
            for (int i = 0; i < UPT; ++i) {
                turn(0, i);
                from[i] += a.sh;
                if (g + 1 < a.hpt) raw_load(from[i], half, raw[i]);
            }
#pragma unroll
            for (int i = 0; i < UPT; ++i) m = fmaxf(m, unit_max(i, false));
        } else {
            for (int base = tid; base - tid < units; base += T) {
                raw_load(src + row(base) * a.sm + g * a.sh, half, raw[0]);
                turn(base, 0);
                m = fmaxf(m, unit_max(0, false));
            }
        }
        m = block_max(m);
        const bool inf = is_inf(m);
        if (inf) {   // the finite values alone
            m = 0.f;
            if (ONE) {
#pragma unroll
                for (int i = 0; i < UPT; ++i) m = fmaxf(m, is_inf(f[i]) ? 0.f : unit_max(i, true));
            } else {
                for (int base = tid; base - tid < units; base += T) {
                    raw_load(src + row(base) * a.sm + g * a.sh, half, raw[0]);
                    turn(base, 0);
                    m = fmaxf(m, is_inf(f[0]) ? 0.f : unit_max(0, true));
                }
            }
            m = block_max(is_inf(m) ? 3.402823466e38f : m);
        }
        const float now = fmaxf(pow2i(e4m3_exponent(m)), had), inv = 1.f / now;   // powers of two: exact
        if (tid == 0) scale[g] = now;
        if (ONE) {
#pragma unroll
            for (int i = 0; i < UPT; ++i) {
                if (inf) drop_inf(p[i], q[i]);
                if (to[i] != nullptr) {
                    *reinterpret_cast<uint2*>(to[i]) = pack_e4m3(p[i], inv * f[i]);
                    *reinterpret_cast<uint2*>(to[i] + half) = pack_e4m3(q[i], inv * f[i]);
                    to[i] += a.c.sh;
                }
            }
        } else {
            for (int base = tid; base - tid < units; base += T) {
                raw_load(src + row(base) * a.sm + g * a.sh, half, raw[0]);
                turn(base, 0);
                if (inf) drop_inf(p[0], q[0]);
                if (base < units) {
                    uint8_t* d = dst + g * a.c.sh + (base >> ulog) * a.c.st;
                    *reinterpret_cast<uint2*>(d) = pack_e4m3(p[0], inv * f[0]);
                    *reinterpret_cast<uint2*>(d + half) = pack_e4m3(q[0], inv * f[0]);
                }
            }
        }
        if (had > 0.f && had != now) reround(dst - 8 * c - w.off * a.c.st + g * a.c.sh, a.c.st, w.off, ulog, had * inv);
    }
}

template <typename IT, typename CT>
static cudaError_t launch_rows(AppendArgs a, int sms, cudaStream_t s) {
    const long long rows = (long long)a.B * a.M;
    const int U = a.hd >> 4;
    // as many heads in one thread as leave 256 threads an SM (each has four
    // heads' loads in flight): the angles of a row are computed once for them, and
    // an angle costs as much as four elements' other work.  One head for small
    // calls.  (8191 rows x 8 heads of 128, fp32 to bf16: 19.8 us with eight heads a
    // thread, 23.7 with one.)
    a.hpt = 1;
    while (a.c.Hkv % (2 * a.hpt) == 0 && rows * U * (a.c.Hkv / (2 * a.hpt)) >= (long long)sms * 256) a.hpt *= 2;
    const long long per_seq = (long long)a.M * (a.c.Hkv / a.hpt) * U;
    const dim3 grid((unsigned)((per_seq + 127) / 128) + 1, 2u * a.B);
    append_rows_kernel<IT, CT><<<grid, 128, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename IT>
static cudaError_t launch_e4m3(AppendArgs a, int sms, cudaStream_t s) {
    const int ps = 1 << a.c.ps_log2, nt = (a.M + ps - 2) / ps + 1, U = a.hd >> 4;
    const int units = (a.M < ps ? a.M : ps) * U;
    const unsigned pages = (unsigned)a.B * nt;
    if (units <= 256) {
        const int T = (units + 31) & ~31;
        append_e4m3_kernel<IT><<<dim3(pages + 1, (unsigned)a.c.Hkv, 2), T < 64 ? 64 : T, 0, s>>>(a);
        return cudaGetLastError();
    }
    // all heads in one CTA where the pages alone fill the GPU
    a.hpt = pages * 2 >= (unsigned)sms ? a.c.Hkv : 1;
    const dim3 grid(pages + 1, (unsigned)(a.c.Hkv / a.hpt), 2);
    const size_t smem = a.rope.on ? (size_t)((ps >> 4) + 16) * (a.hd >> 1) * sizeof(float2) : 0;
    const bool one = units <= 1024;
    const int T = one ? ((units + 1) / 2 + 31) & ~31 : kPageThreads;
    if (smem > 40 * 1024) {   // the most (head_dim 512, pages of 256), so that two host threads' calls do not disturb each other
        constexpr int most = ((MTP_MAX_PAGE_SIZE >> 4) + 16) * 256 * (int)sizeof(float2);
        const cudaError_t e = one ? cudaFuncSetAttribute(append_e4m3_pages_kernel<IT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, most)
                                  : cudaFuncSetAttribute(append_e4m3_pages_kernel<IT, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return e;
    }
    if (one) append_e4m3_pages_kernel<IT, true><<<grid, T, smem, s>>>(a);
    else append_e4m3_pages_kernel<IT, false><<<grid, T, smem, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_kv_append(const AppendArgs& a, int in_dtype, int kv_dtype, int sms, cudaStream_t s) {
    const bool f = in_dtype == MTP_DTYPE_F32;
    if (kv_dtype == MTP_DTYPE_E4M3) return f ? launch_e4m3<float>(a, sms, s) : launch_e4m3<uint16_t>(a, sms, s);
    if (kv_dtype == MTP_DTYPE_F32) return f ? launch_rows<float, float>(a, sms, s) : launch_rows<uint16_t, float>(a, sms, s);
    return f ? launch_rows<float, uint16_t>(a, sms, s) : launch_rows<uint16_t, uint16_t>(a, sms, s);
}

}  // namespace mtp
