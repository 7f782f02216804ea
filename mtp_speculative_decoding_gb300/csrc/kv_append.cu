// kv_append.cu -- new key and value rows into a paged KV cache: RMSNorm and
// rotation of the keys, one rounding to the cache's type.
//
// key = rope(rmsnorm(k), p), value = v.  Both are bound by the bytes in and
// out (small calls: by the launch and two dependent loads, the length and then
// the page).
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
// heads; gridDim.y: keys, values
// ---------------------------------------------------------------------------
template <typename IT, typename CT>
__global__ void __launch_bounds__(128) append_rows_kernel(const __grid_constant__ AppendArgs a) {
    if (blockIdx.x == gridDim.x - 1) {
        if (blockIdx.y == 0) append_status(a);
        return;
    }
    const int U = a.hd >> 4, groups = a.c.Hkv / a.hpt;
    const long long total = (long long)a.B * a.M * groups * U;
    const long long x = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const bool in = x < total;
    long long r = (in ? x : total - 1) / U;
    const int c = (int)((in ? x : total - 1) % U), g0 = (int)(r % groups) * a.hpt;
    r /= groups;
    const int b = (int)(r / a.M), j = (int)(r % a.M);
    const bool key = blockIdx.y == 0;
    const IT* src = reinterpret_cast<const IT*>(key ? a.k : a.v) + b * a.sb + j * a.sm + g0 * a.sh + 8 * c;
    const int len = a.kv_len[b], n = a.n_new ? a.n_new[b] : a.M;
    const bool live = in && seq_ok(len, n, a.M, a.c) && j < n;
    const long long pos = (long long)len + j;
    CT* dst = nullptr;
    if (live) {
        const int pg = a.c.table[(long long)b * a.c.max_pages + (int)(pos >> a.c.ps_log2)];
        if ((unsigned)pg < (unsigned)a.c.n_pages)
            dst = reinterpret_cast<CT*>(key ? a.c.k : a.c.v) + pg * a.c.sp + (pos & ((1 << a.c.ps_log2) - 1)) * a.c.st +
                  g0 * a.c.sh + 8 * c;
    }
    if (!__any_sync(0xffffffffu, dst != nullptr)) return;
    float cs[8], sn[8];
    const bool rot = key && a.rope.on;
    if (rot) unit_angles<false>(live ? pos : 0, a.rope.hi + 8 * c, a.rope.lo + 8 * c, cs, sn);
#pragma unroll 4
    for (int h = 0; h < a.hpt; ++h) {
        float p[8], q[8];
        load8(src + h * a.sh, p);
        load8(src + h * a.sh + (a.hd >> 1), q);
        if (key && a.k_norm) unit_norm(p, q, a.k_norm, c, a.hd, a.eps);
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
__device__ __forceinline__ float finite_abs(float x) {
    const float y = fabsf(x);
    return y <= 3.402823466e38f ? y : 0.f;   // NaN and infinity do not count
}
// 8 values times inv as e4m3 codes (nearest even, saturating; NaN and infinity become NaN)
__device__ __forceinline__ uint2 pack_e4m3(const float (&x)[8], float inv) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float lo = x[2 * i] - x[2 * i] == 0.f ? x[2 * i] * inv : __uint_as_float(0x7FC00000u);
        const float hi = x[2 * i + 1] - x[2 * i + 1] == 0.f ? x[2 * i + 1] * inv : __uint_as_float(0x7FC00000u);
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
    }
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// UPT: units of a thread that stay in registers between the maximum and the
// rounding; a page whose new rows need more is read twice (the second time
// from L2)
template <typename IT, int UPT>
__global__ void __launch_bounds__(512) append_e4m3_kernel(const __grid_constant__ AppendArgs a) {
    const int ps = 1 << a.c.ps_log2, nt = (a.M + ps - 2) / ps + 1;
    if (blockIdx.x == gridDim.x - 1) {
        if (blockIdx.y == 0 && blockIdx.z == 0) append_status(a);
        return;
    }
    __shared__ float red[16];
    const int b = blockIdx.x / nt, it = blockIdx.x % nt, g = blockIdx.y;
    const bool key = blockIdx.z == 0;
    const int len = a.kv_len[b], n = a.n_new ? a.n_new[b] : a.M;
    if (!seq_ok(len, n, a.M, a.c)) return;
    const int pi = (len >> a.c.ps_log2) + it;
    const long long first = (long long)pi << a.c.ps_log2;                     // position of the page's slot 0
    const int j0 = it == 0 ? 0 : (int)(first - len);
    const int j1 = first + ps - len < n ? (int)(first + ps - len) : n;
    if (j0 >= j1) return;
    const int page = a.c.table[(long long)b * a.c.max_pages + pi];
    if ((unsigned)page >= (unsigned)a.c.n_pages) return;
    const int off = (int)(len + j0 - first);                                   // slots the page holds already
    float* sc = (key ? a.c.ks : a.c.vs) + (long long)page * a.c.Hkv + g;
    const float had = off > 0 ? *sc : 0.f;
    const int U = a.hd >> 4, ulog = 31 - __clz(U), units = (j1 - j0) << ulog;
    const int step = (int)blockDim.x * UPT;
    const IT* src = reinterpret_cast<const IT*>(key ? a.k : a.v) + b * a.sb + g * a.sh;
    uint8_t* dst = reinterpret_cast<uint8_t*>(key ? a.c.k : a.c.v) + page * a.c.sp + g * a.c.sh;
    float p[UPT][8], q[UPT][8];
    auto fetch = [&](int base) {
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            const int x = base + i * (int)blockDim.x + (int)threadIdx.x, c = x & (U - 1);
            const int j = j0 + (x < units ? x >> ulog : 0);
            load8(src + j * a.sm + 8 * c, p[i]);
            load8(src + j * a.sm + 8 * c + (a.hd >> 1), q[i]);
        }
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            const int x = base + i * (int)blockDim.x + (int)threadIdx.x, c = x & (U - 1);
            if (key && a.k_norm) unit_norm(p[i], q[i], a.k_norm, c, a.hd, a.eps);
            if (key && a.rope.on) {
                float cs[8], sn[8];
                unit_angles<false>((long long)len + j0 + (x < units ? x >> ulog : 0), a.rope.hi + 8 * c, a.rope.lo + 8 * c, cs, sn);
                unit_rotate(p[i], q[i], cs, sn);
            }
        }
    };
    float m = 0.f;
    for (int base = 0; base < units; base += step) {
        fetch(base);
#pragma unroll
        for (int i = 0; i < UPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) m = fmaxf(m, fmaxf(finite_abs(p[i][e]), finite_abs(q[i][e])));
    }
    m = warp_max(m);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) m = fmaxf(m, red[w]);
    // largest scale: the new rows', or the one the older codes have
    float now = pow2i(e4m3_exponent(m));
    now = fmaxf(now, had);
    const float inv = 1.f / now;   // a power of two: exact
    if (threadIdx.x == 0) *sc = now;
    for (int base = 0; base < units; base += step) {
        if (step < units) fetch(base);
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            const int x = base + i * (int)blockDim.x + (int)threadIdx.x, c = x & (U - 1);
            if (x >= units) continue;
            uint8_t* d = dst + (off + (x >> ulog)) * a.c.st + 8 * c;
            *reinterpret_cast<uint2*>(d) = pack_e4m3(p[i], inv);
            *reinterpret_cast<uint2*>(d + (a.hd >> 1)) = pack_e4m3(q[i], inv);
        }
    }
    if (had > 0.f && had != now) {   // the page's older codes, re-rounded to the larger scale
        const float f = had * inv;
        for (int x = threadIdx.x; x < off << ulog; x += blockDim.x) {
            uint4* d = reinterpret_cast<uint4*>(dst + (x >> ulog) * a.c.st + 16 * (x & (U - 1)));
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
}

template <typename IT, typename CT>
static cudaError_t launch_rows(AppendArgs a, int sms, cudaStream_t s) {
    const long long rows = (long long)a.B * a.M;
    const int U = a.hd >> 4;
    // all heads in one thread where that still fills the GPU: the angles of a
    // row are then computed once; one head per thread for small calls
    a.hpt = rows * U >= (long long)sms * 512 ? a.c.Hkv : 1;
    const long long total = rows * (a.c.Hkv / a.hpt) * U;
    const dim3 grid((unsigned)((total + 127) / 128) + 1, 2);
    append_rows_kernel<IT, CT><<<grid, 128, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename IT>
static cudaError_t launch_e4m3(const AppendArgs& a, cudaStream_t s) {
    const int ps = 1 << a.c.ps_log2, nt = (a.M + ps - 2) / ps + 1, U = a.hd >> 4;
    const int units = (a.M < ps ? a.M : ps) * U;
    const dim3 grid((unsigned)a.B * nt + 1, (unsigned)a.c.Hkv, 2);
    if (units <= 256) {
        const int T = (units + 31) & ~31;
        append_e4m3_kernel<IT, 1><<<grid, T < 64 ? 64 : T, 0, s>>>(a);
    } else {
        int T = ((units + 3) / 4 + 31) & ~31;
        append_e4m3_kernel<IT, 4><<<grid, T > 512 ? 512 : T, 0, s>>>(a);
    }
    return cudaGetLastError();
}

cudaError_t launch_kv_append(const AppendArgs& a, int in_dtype, int kv_dtype, int sms, cudaStream_t s) {
    const bool f = in_dtype == MTP_DTYPE_F32;
    if (kv_dtype == MTP_DTYPE_E4M3) return f ? launch_e4m3<float>(a, s) : launch_e4m3<uint16_t>(a, s);
    if (kv_dtype == MTP_DTYPE_F32) return f ? launch_rows<float, float>(a, sms, s) : launch_rows<uint16_t, float>(a, sms, s);
    return f ? launch_rows<float, uint16_t>(a, sms, s) : launch_rows<uint16_t, uint16_t>(a, sms, s);
}

}  // namespace mtp
