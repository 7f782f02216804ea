// rotate.cu -- query and key rows normed and rotated by several positions.
//
// y = rope(rmsnorm(x)), where the pair (i, i + pairs) turns by the position of
// its axis times theta^(-i / pairs).  A thread takes one unit (8 pairs, or 16
// elements behind the rotated ones) of `hpt` heads of one row, so that the
// angles of a row are computed once for those heads.  Long calls are bound by
// the bytes in and out (8192 rows of 24 heads of 128, bf16: 18.6 us one call behind
// another, 5.4 TB/s, and 22.5 us, 4.5 TB/s, in turn with other work; captured, with
// nothing in L2, 25.7), in fp32 with a norm also by what 16 warps an SM have in flight
// (4093 rows of 20 heads of 256: 37.1 us, 4.5 TB/s), short ones by the launch and two
// dependent loads (4 rows: 9.3 us captured).  Four heads are in flight whatever a
// thread's number of heads is: with one or two (calls of up to some 1600 rows) the others
// load and turn the same head again.
#include "rows.cuh"

namespace mtp {

namespace {

// (plain loads: the rows may be rewritten in place)
__device__ __forceinline__ uint4 ld16(const void* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}
__device__ __forceinline__ void in8(const float* p, float (&x)[8]) {
    const uint4 u = ld16(p), w = ld16(p + 4);
    x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y); x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
    x[4] = __uint_as_float(w.x); x[5] = __uint_as_float(w.y); x[6] = __uint_as_float(w.z); x[7] = __uint_as_float(w.w);
}
__device__ __forceinline__ void in8(const uint16_t* p, float (&x)[8]) { open_unit(ld16(p), x); }

constexpr int kRotThreads = 128;

template <typename T>
__global__ void __launch_bounds__(kRotThreads) rotate_axes_kernel(const __grid_constant__ RotateArgs a) {
    constexpr bool FAST = sizeof(T) == 2;
    // lanes read the tables at different places, which parameters serve one by one
    __shared__ __align__(16) float s_hi[256], s_lo[256];
    __shared__ __align__(16) uint8_t s_axis[256];
    for (int i = threadIdx.x; i < a.pairs; i += kRotThreads) {
        s_hi[i] = a.rope.hi[i];
        s_lo[i] = a.rope.lo[i];
        s_axis[i] = a.axis[i];
    }
    __syncthreads();
    const int U = a.hd >> 4, ulog = 31 - __clz(U), all = a.groups[0] + a.groups[1];
    const long long x = (long long)blockIdx.x * kRotThreads + threadIdx.x, unit = x >> ulog;
    const int c = (int)(x & (U - 1));
    int row = (int)(unit / all), grp = (int)(unit - (long long)row * all);
    const bool live = row < a.rows;   // (whole rows' lanes; the others go along for the shuffles)
    if (!live) {
        row = a.rows - 1;
        grp = 0;
    }
    const int which = grp >= a.groups[0] ? 1 : 0;
    if (which) grp -= a.groups[0];
    const int h0 = grp * a.hpt, h1 = h0 + a.hpt < a.heads[which] ? h0 + a.hpt : a.heads[which];
    const bool turn = 8 * c < a.pairs;
    // the unit's two runs of eight elements
    const int e0 = turn ? 8 * c : 2 * a.pairs + 16 * (c - (a.pairs >> 3)), e1 = turn ? a.pairs + 8 * c : e0 + 8;
    const T* src = reinterpret_cast<const T*>(a.in[which]) + row * a.in_sm[which];
    T* dst = reinterpret_cast<T*>(a.out[which]) + row * a.out_sm[which];
    const float* gain = a.norm[which];
    float g0[8], g1[8];
    if (gain)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            g0[i] = __ldg(gain + e0 + i);
            g1[i] = __ldg(gain + e1 + i);
        }
    // heads in flight, the first ones while the angles are computed (fp32: 40.0 us with two
    // that come in behind them, 37.1 so)
    constexpr int N = 4;
    float p[N][8], q[N][8];
    auto fetch = [&](int i0) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int h = h0 + i0 + i < h1 ? h0 + i0 + i : h1 - 1;   // (every lane of the warp takes part in the norm)
            in8(src + h * a.in_sh[which] + e0, p[i]);
            in8(src + h * a.in_sh[which] + e1, q[i]);
        }
    };
    fetch(0);
    float cs[8], sn[8];
    if (turn) {
        int at[MTP_MAX_AXES];
#pragma unroll
        for (int i = 0; i < MTP_MAX_AXES; ++i) at[i] = i < a.axes ? a.pos[(long long)i * a.rows + row] : 0;
        const uint2 ax = *reinterpret_cast<const uint2*>(s_axis + 8 * c);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const unsigned k = ((i < 4 ? ax.x : ax.y) >> (8 * (i & 3))) & 3u;
            const int pos = k & 2u ? (k & 1u ? at[3] : at[2]) : (k & 1u ? at[1] : at[0]);
            float pl, ph;
            split_pos(pos, pl, ph);
            pair_angle<FAST>(pl, ph, s_hi[8 * c + i], s_lo[8 * c + i], cs[i], sn[i]);
        }
    }
#pragma unroll 1
    for (int i0 = 0; i0 < a.hpt; i0 += N) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int h = h0 + i0 + i;
            if (a.norm[0] || a.norm[1]) {   // (queries and keys may share a warp: all lanes take part)
                const float r = unit_rms(p[i], q[i], a.hd, a.eps);
                if (gain)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        p[i][e] *= r * g0[e];
                        q[i][e] *= r * g1[e];
                    }
            }
            if (turn) unit_rotate(p[i], q[i], cs, sn);
            if (live && h < h1) {
                store8(dst + h * a.out_sh[which] + e0, p[i]);
                store8(dst + h * a.out_sh[which] + e1, q[i]);
            }
        }
        if (i0 + N < a.hpt) fetch(i0 + N);
    }
}

}  // namespace

cudaError_t launch_rotate_axes(RotateArgs a, int dtype, int sms, cudaStream_t s) {
    // as many heads in one thread as leave 512 threads an SM: an angle costs as much as
    // the rest of four elements (128 to 1024 threads measure alike; with 2048 8192 rows of
    // bf16 take 20.7 us instead of 18.6, one call behind another), and no more than divide both counts, where that
    // leaves four: a group's missing heads cost as much as others
    a.hpt = 1;
    while (a.hpt < 16 && (a.hpt < 4 || (a.heads[0] | a.heads[1]) % (2 * a.hpt) == 0) &&
           (long long)a.rows * ((a.heads[0] + a.heads[1]) / (2 * a.hpt)) * (a.hd >> 4) >= (long long)sms * 512)
        a.hpt *= 2;
    for (int w = 0; w < 2; ++w) a.groups[w] = (a.heads[w] + a.hpt - 1) / a.hpt;
    const long long threads = (long long)a.rows * (a.groups[0] + a.groups[1]) * (a.hd >> 4);
    const unsigned grid = (unsigned)((threads + kRotThreads - 1) / kRotThreads);
    if (dtype == MTP_DTYPE_F32) rotate_axes_kernel<float><<<grid, kRotThreads, 0, s>>>(a);
    else rotate_axes_kernel<uint16_t><<<grid, kRotThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace mtp
