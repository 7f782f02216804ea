// rows_attn.cu -- attention of many rows over the paged cache on the CUDA cores:
// a warp takes one row (a token's query head) and walks the positions that it
// attends.  It serves fp32 queries or caches and the head dimensions 32 and 512,
// and the rows whose product on the tensor cores is not finite; with it, the merge
// of what the tensor cores left in parts.
//
// Every score, maximum, sum and output is fp32.  A row's units (16 elements, see
// paged.cuh) lie in hd / 16 lanes, so the warp holds 32 / (hd / 16) positions at
// a time and reads each key and value as 16-byte pieces; every lane group keeps
// a running maximum and sum of its own, merged at the end.
#include "rows_attn_tc.cuh"

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
            bad = !seq_at(a, b, s) || bad;   // (where bounds do not ascend, two neighbours do not)
            if (b < a.n_groups) bad = bad || a.group_start[b] > a.group_start[b + 1];
        }
    const long long row = (long long)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    const int tok = (int)(row / a.Hq), h = (int)(row - (long long)tok * a.Hq);
    const int b = a.M > 0 ? tok / a.M : last_at_most(a.row_start, a.B, tok);
    Seq s;
    if (b < a.B && seq_at(a, b, s)) {
        const int j = (int)(tok - s.row0);
        bool mine = j >= 0 && j < s.n;
        if (mine && (a.M == 0 || a.n_groups > 0)) {   // (32 bounds at a time: little beside the positions that a row walks)
            if (a.M == 0)
                for (int i = lane; i <= a.B; i += 32) mine = mine && bound_agrees(a.row_start, b, i);
            else   // groups that do not ascend: all are left out
                for (int i = lane; i < a.n_groups; i += 32) mine = mine && a.group_start[i] <= a.group_start[i + 1];
            mine = __all_sync(0xffffffffu, mine);
        }
        if (mine) bad = !attend_row<QT, KT>(a, s, b, j, h, lane) || bad;
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

// ---------------------------------------------------------------------------
// merge of the parts that the tensor cores left: out = sum_s 2^(m_s - M) o_s /
// sum_s 2^(m_s - M) l_s over a row's parts, hd / 16 threads a row.  A prompt's row has
// parts where its item was cut between workers; with shared prefixes every row has its
// prefix's and its own (found by the attention while it runs: searching the plan here
// took 8 us of a call's 57).  A result that is not finite is computed again by
// attend_row, and so are the rows that the attention marked.  A call is 6 us longer for
// it: the launch, two dependent loads, and with many workers 40 MB of parts.
// ---------------------------------------------------------------------------
// kOddRows: rows whose marks a CTA looks at.  (4096 of them left most SMs idle where every
// row is marked: 2.3 s for 8192 tokens of 16 heads of 256.)
constexpr int kMergeRowThreads = 256, kOddRows = 2 * kMergeRowThreads;
__host__ __device__ constexpr int merge_rows(int hd) { return kMergeRowThreads / (hd >> 4); }   // rows of a CTA

// attend_row out of line: seldom called, and the merge keeps its registers
template <typename KT>
__device__ __noinline__ void attend_again(const RowsArgs* a, long long id) {
    const int tok = (int)(id / a->Hq), h = (int)(id - (long long)tok * a->Hq), b = a->M > 0 ? tok / a->M : last_at_most(a->row_start, a->B, tok);
    Seq s;
    if (!seq_at(*a, b, s)) return;
    const int j = (int)(tok - s.row0);
    if (j >= 0 && j < s.n) attend_row<uint16_t, KT>(*a, s, b, j, h, threadIdx.x & 31);
}

template <typename KT, bool PROMPT>
__global__ void __launch_bounds__(kMergeRowThreads, PROMPT ? 3 : 2) rows_merge_kernel(const __grid_constant__ RowsTcArgs t, int statuses, int merges,
                                                                                     int planes) {
    __shared__ long long s_odd[merge_rows(64)];             // rows of out whose result is not finite (< 0: none)
    __shared__ uint16_t s_list[PROMPT ? kOddRows : 1];
    __shared__ int s_n;
    const RowsArgs& a = t.a;
    const int tid = threadIdx.x, warp = tid >> 5;
    if (tid == 0) s_n = 0;
    if (tid < merge_rows(64)) s_odd[tid] = -1;
    __syncthreads();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if ((int)blockIdx.x == (int)gridDim.x - 1) {   // the call's status from the CTAs'
        int bad = 0;
        for (int c = tid; c < statuses; c += kMergeRowThreads) {
            const int st = t.cta_status[c];
            if (st == MTP_ERR_TIMEOUT) bad |= 2;
            else if (st != MTP_OK) bad |= 1;
        }
        const int any1 = __syncthreads_or(bad & 1), any2 = __syncthreads_or(bad & 2);
        if (tid == 0) {
            a.hdr->status = any2 ? MTP_ERR_TIMEOUT : any1 ? MTP_ERR_ARG : MTP_OK;
            a.hdr->barrier = 0;
            a.hdr->done = 0;
        }
        return;
    }
    if (PROMPT && (int)blockIdx.x >= merges) {   // rows that the attention marked
        const long long first = (long long)(blockIdx.x - merges) * kOddRows, rows = (long long)a.T * a.Hq;
        uint32_t v = *reinterpret_cast<const uint16_t*>(t.odd + first + 2 * tid);
        if (planes > 1) v |= *reinterpret_cast<const uint16_t*>(t.odd + t.odd_plane + first + 2 * tid);   // (both threads of a row)
        for (int i = 0; v && i < 2; ++i)
            if ((v >> (8 * i)) & 0xFFu && first + 2 * tid + i < rows) s_list[atomicAdd(&s_n, 1)] = (uint16_t)(2 * tid + i);
        __syncthreads();
        for (int i = warp; i < s_n; i += kMergeRowThreads / 32) attend_again<KT>(&a, first + s_list[i]);
        return;
    }
    const int hd = a.hd, gt = hd >> 4, per = kMergeRowThreads / gt, sub = tid / gt, d = 4 * (tid - sub * gt), quarter = hd >> 2;
    RowPart parts[2];
    long long row = -1;                                     // row of out (in heads)
    if (PROMPT) {
        const int chunks = kRowTile / per > 0 ? kRowTile / per : 1, w = blockIdx.x / chunks, r = (blockIdx.x - w * chunks) * per + sub;
        const RowNote n = t.note[w];
        // (an attention that gave up may have left anything: it stays in bounds)
        if (n.last > w && n.last < t.workers && r < n.rows && n.rows <= kRowTile && n.r0 >= 0 && n.g >= 0 && n.g < a.c.Hkv) {
            const int at = n.r0 + r, j = at / a.G;
            row = ((long long)n.row0 + j) * a.Hq + n.g * a.G + at - j * a.G;
            if (row >= (long long)a.T * a.Hq) row = -1;
            parts[0] = {RowPart::kSlots, (uint16_t)w, (uint16_t)n.last, (uint16_t)w, (uint16_t)r, 1};
        }
    } else {
        const long long id = (long long)blockIdx.x * per + sub;
        if (id < (long long)a.B * a.M * a.Hq) {
            parts[0] = t.row_parts[2 * id];
            parts[1] = t.row_parts[2 * id + 1];
            if (parts[0].there) row = id;
        }
    }
    if (row >= 0) {
        float M = kNoScore, l = 0.f;
        float4 acc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int N = PROMPT ? 2 : 4;   // parts in flight
#pragma unroll
        for (int which = 0; which < (PROMPT ? 1 : 2); ++which) {
            const RowPart p = parts[which];
            if (!p.there) continue;
            const bool dense = p.dense != RowPart::kSlots;
#pragma unroll 1
            for (int w = p.w0; w <= p.w1; w += N) {
                float2 ml[N];
                float4 o[N][4];
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    ml[e] = make_float2(kNoScore, 0.f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[e][i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (w + e > p.w1) continue;
                    const long long at = (2ll * (w + e) + (w + e == p.first ? 1 : 0)) * kRowTile + p.r;
                    const float* src = (dense ? t.dense + (long long)p.dense * hd : t.part + at * hd) + d;
                    ml[e] = dense ? t.dense_ml[p.dense] : t.part_ml[at];
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[e][i] = *reinterpret_cast<const float4*>(src + i * quarter);
                }
                float mn = M;
#pragma unroll
                for (int e = 0; e < N; ++e) mn = fmaxf(mn, ml[e].x);
                const float f = exp2f(M - mn);
                l *= f;
                M = mn;
                float x[N];
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    x[e] = exp2f(ml[e].x - mn);
                    l = fmaf(x[e], ml[e].y, l);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[i].x *= f;
                    acc[i].y *= f;
                    acc[i].z *= f;
                    acc[i].w *= f;
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        acc[i].x = fmaf(x[e], o[e][i].x, acc[i].x);
                        acc[i].y = fmaf(x[e], o[e][i].y, acc[i].y);
                        acc[i].z = fmaf(x[e], o[e][i].z, acc[i].z);
                        acc[i].w = fmaf(x[e], o[e][i].w, acc[i].w);
                    }
                }
            }
        }
        const float inv = zero_sum(l);
        float odd = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            acc[i].x *= inv;
            acc[i].y *= inv;
            acc[i].z *= inv;
            acc[i].w *= inv;
            odd += fmaf(acc[i].x, 0.f, fmaf(acc[i].y, 0.f, fmaf(acc[i].z, 0.f, acc[i].w * 0.f)));
            *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + row * hd + d + i * quarter) =
                make_uint2(pack_bf16(acc[i].x, acc[i].y), pack_bf16(acc[i].z, acc[i].w));
        }
        if (!(odd == 0.f)) s_odd[sub] = row;
    }
    __syncthreads();
    for (int i = warp; i < per; i += kMergeRowThreads / 32)
        if (s_odd[i] >= 0) attend_again<KT>(&a, s_odd[i]);
}

template <typename KT>
cudaError_t merge(const cudaLaunchConfig_t& cfg, const RowsTcArgs& t, int statuses, int merges, int planes) {
    return t.a.M > 0 ? cudaLaunchKernelEx(&cfg, rows_merge_kernel<KT, false>, t, statuses, merges, planes)
                     : cudaLaunchKernelEx(&cfg, rows_merge_kernel<KT, true>, t, statuses, merges, planes);
}

}  // namespace

cudaError_t launch_rows_merge(const RowsTcArgs& t, int kv_dtype, cudaStream_t s) {
    const RowsArgs& a = t.a;
    const int per = merge_rows(a.hd);
    const long long merges = a.M > 0 ? ((long long)a.B * a.M * a.Hq + per - 1) / per : (long long)t.workers * (kRowTile / per);
    const long long odd = a.M > 0 ? 0 : ((long long)a.T * a.Hq + kOddRows - 1) / kOddRows;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(merges + odd + 1));
    cfg.blockDim = dim3(kMergeRowThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // its CTAs come in while the attention ends
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const int planes = rows_halves(a.hd);
    const int statuses = t.workers * rows_pair(a.hd) + 1;   // the CTAs' and the plan's
    return kv_dtype == MTP_DTYPE_E4M3 ? merge<uint8_t>(cfg, t, statuses, (int)merges, planes) : merge<uint16_t>(cfg, t, statuses, (int)merges, planes);
}

cudaError_t launch_rows_cc(const RowsArgs& a, int dtype, int kv_dtype, cudaStream_t s) {
    return dtype == MTP_DTYPE_F32 ? cc_kv<float>(a, kv_dtype, s) : cc_kv<uint16_t>(a, kv_dtype, s);
}

}  // namespace mtp
