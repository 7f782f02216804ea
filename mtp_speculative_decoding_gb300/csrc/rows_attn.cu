// rows_attn.cu -- attention of many rows over the paged cache on the CUDA cores:
// a warp takes one row (a token's query head) and walks the positions that it
// attends.
//
// Every score, maximum, sum and output is fp32.  A row's units (16 elements, see
// paged.cuh) lie in hd / 16 lanes, so the warp holds 32 / (hd / 16) positions at
// a time and reads each key and value as 16-byte pieces; every lane group keeps
// a running maximum and sum of its own, merged at the end.
#include "rows.cuh"

namespace mtp {

namespace {

__device__ __forceinline__ float zero_sum(float l) { return l == 0.f ? 0.f : 1.f / l; }
// 2^x, never 0: an infinite value keeps its sign whatever its weight (0 times it
// would be a NaN); a finite one's share is at most 2^-149 of it too much
__device__ __forceinline__ float weight(float x) {
    const float w = exp2f(x);
    return w == 0.f ? __uint_as_float(1u) : w;
}
__device__ __forceinline__ void row8(const float* p, float, float (&x)[8]) { load8(p, x); }
__device__ __forceinline__ void row8(const uint16_t* p, float, float (&x)[8]) { load8(p, x); }
__device__ __forceinline__ void row8(const uint8_t* p, float s, float (&x)[8]) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    const uint32_t w[2] = {u.x, u.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
        const float2 y = __half22float2(__half2(h));
        x[2 * i] = y.x * s;
        x[2 * i + 1] = y.y * s;
    }
}

// Token j, query head h of sequence s (index b): the whole warp.  Returns
// whether every attended position's page was there.
template <typename QT, typename KT>
__device__ bool attend_row(const RowsArgs& a, const Seq& s, int b, int j, int h, int lane) {
    const int hd = a.hd, U = hd >> 4, c = lane & (U - 1), grp = lane / U, NP = 32 / U, half = hd >> 1, g = h / a.G;
    const int p = s.len + j, ps_mask = (1 << a.c.ps_log2) - 1;
    float q0[8], q1[8];
    const QT* src = reinterpret_cast<const QT*>(a.q) + s.q0 + j * a.sm + h * a.sh + 8 * c;
    load8(src, q0);
    load8(src + half, q1);
    if (a.q_norm) unit_norm(q0, q1, a.q_norm, c, hd, a.eps);
    if (a.rope.on) {
        float cs[8], sn[8];
        unit_angles<false>((long long)p, a.rope.hi + 8 * c, a.rope.lo + 8 * c, cs, sn);
        unit_rotate(q0, q1, cs, sn);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        q0[e] *= a.scale;
        q1[e] *= a.scale;
    }
    float m = kNoScore, l = 0.f, o0[8], o1[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o0[e] = o1[e] = 0.f;
    bool bad = false;
    const int lo = a.c.window > 0 && p + 1 > a.c.window ? p + 1 - a.c.window : 0;
    const int sink = a.c.sink < lo ? a.c.sink : lo;
    constexpr int N = 4;   // positions of a lane group in flight
    for (int part = 0; part < 2; ++part) {
        const int t0 = part ? lo : 0, t1 = part ? p + 1 : sink;
#pragma unroll 1
        for (int tb = t0; tb < t1; tb += N * NP) {
            const KT* v[N];
            float vs[N], z[N], mx = m;
#pragma unroll
            for (int u = 0; u < N; ++u) {
                const int t = tb + u * NP + grp;
                v[u] = nullptr;
                vs[u] = 1.f;
                z[u] = 0.f;
                if (t < t1) {
                    const int pg = a.c.table[(long long)(t < s.P ? s.first : b) * a.c.max_pages + (t >> a.c.ps_log2)];
                    float ks = 1.f;
                    bool there = (unsigned)pg < (unsigned)a.c.n_pages;
                    if (there && a.c.ks) {
                        ks = a.c.ks[(long long)pg * a.c.Hkv + g];
                        vs[u] = a.c.vs[(long long)pg * a.c.Hkv + g];
                        there = scale_ok(ks) && scale_ok(vs[u]);
                    }
                    bad = bad || !there;
                    if (there) {
                        const long long at = pg * a.c.sp + g * a.c.sh + (t & ps_mask) * a.c.st + 8 * c;
                        v[u] = reinterpret_cast<const KT*>(a.c.v) + at;
                        float k0[8], k1[8];
                        row8(reinterpret_cast<const KT*>(a.c.k) + at, ks, k0);
                        row8(reinterpret_cast<const KT*>(a.c.k) + at + half, ks, k1);
#pragma unroll
                        for (int e = 0; e < 8; ++e) z[u] = fmaf(q0[e], k0[e], fmaf(q1[e], k1[e], z[u]));
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < N; ++u) {
                for (int o = U >> 1; o > 0; o >>= 1) z[u] += __shfl_xor_sync(0xffffffffu, z[u], o);
                if (v[u]) mx = fmaxf(mx, z[u]);
            }
            const float f = weight(m - mx);
            l *= f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                o0[e] *= f;
                o1[e] *= f;
            }
            m = mx;
#pragma unroll
            for (int u = 0; u < N; ++u) {
                if (!v[u]) continue;
                const float pr = exp2f(z[u] - mx), w = pr == 0.f ? __uint_as_float(1u) : pr;
                l += pr;   // (as it is: a row of scores of -inf has none)
                float v0[8], v1[8];
                row8(v[u], vs[u], v0);
                row8(v[u] + half, vs[u], v1);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    o0[e] = fmaf(w, v0[e], o0[e]);
                    o1[e] = fmaf(w, v1[e], o1[e]);
                }
            }
        }
    }
    for (int o = U; o < 32; o <<= 1) {   // the lane groups' parts
        const float om = __shfl_xor_sync(0xffffffffu, m, o), ol = __shfl_xor_sync(0xffffffffu, l, o), mn = fmaxf(m, om);
        const float f = weight(m - mn), of = weight(om - mn);
        l = l * f + ol * of;
        m = mn;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            o0[e] = o0[e] * f + __shfl_xor_sync(0xffffffffu, o0[e], o) * of;
            o1[e] = o1[e] * f + __shfl_xor_sync(0xffffffffu, o1[e], o) * of;
        }
    }
    const float inv = zero_sum(l);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        o0[e] *= inv;
        o1[e] *= inv;
    }
    if (grp == 0) {
        QT* dst = reinterpret_cast<QT*>(a.out) + ((s.row0 + j) * a.Hq + h) * hd + 8 * c;
        store8(dst, o0);
        store8(dst + half, o1);
    }
    return !bad;
}

constexpr int kRowThreads = 128;

template <typename QT, typename KT>
__global__ void __launch_bounds__(kRowThreads) rows_cc_kernel(const __grid_constant__ RowsArgs a) {
    const int lane = threadIdx.x & 31;
    bool bad = false;
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < a.B; b += kRowThreads) {
            Seq s;
            bad = !seq_at(a, b, s) || bad;
        }
    const long long row = (long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    const int tok = (int)(row / a.Hq), h = (int)(row - (long long)tok * a.Hq);
    const int b = a.M > 0 ? tok / a.M : last_at_most(a.row_start, a.B, tok);
    Seq s;
    if (b < a.B && seq_at(a, b, s)) {
        const int j = (int)(tok - s.row0);
        if (j >= 0 && j < s.n) bad = !attend_row<QT, KT>(a, s, b, j, h, lane) || bad;
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicCAS(&a.hdr->status, MTP_OK, MTP_ERR_ARG);
}

template <typename QT, typename KT>
cudaError_t cc(const RowsArgs& a, cudaStream_t s) {
    const cudaError_t e = cudaMemsetAsync(a.hdr, 0, sizeof(WsHeader), s);
    if (e != cudaSuccess) return e;
    const long long rows = (a.M > 0 ? (long long)a.B * a.M : a.T) * a.Hq;
    constexpr int per = kRowThreads / 32;
    rows_cc_kernel<QT, KT><<<(unsigned)((rows + per - 1) / per), kRowThreads, 0, s>>>(a);
    return cudaGetLastError();
}
template <typename QT>
cudaError_t cc_kv(const RowsArgs& a, int kv_dtype, cudaStream_t s) {
    return kv_dtype == MTP_DTYPE_F32 ? cc<QT, float>(a, s) : kv_dtype == MTP_DTYPE_BF16 ? cc<QT, uint16_t>(a, s) : cc<QT, uint8_t>(a, s);
}

}  // namespace

cudaError_t launch_rows_cc(const RowsArgs& a, int dtype, int kv_dtype, cudaStream_t s) {
    return dtype == MTP_DTYPE_F32 ? cc_kv<float>(a, kv_dtype, s) : cc_kv<uint16_t>(a, kv_dtype, s);
}

}  // namespace mtp
