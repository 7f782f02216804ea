// paged_attn.cu -- attention over the paged cache on the CUDA cores, and the
// merge of split items.
//
// Every score, maximum, sum and output is fp32; this path serves fp32 queries
// or caches and the head dimension 32 (the bf16 and e4m3 caches of bf16
// queries run on the tensor cores).
#include "paged.cuh"

namespace mtp {

__device__ __forceinline__ void kv8(const float* p, float, float (&x)[8]) { load8(p, x); }
__device__ __forceinline__ void kv8(const uint16_t* p, float, float (&x)[8]) { load8(p, x); }
__device__ __forceinline__ void kv8(const uint8_t* p, float s, float (&x)[8]) {
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
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(uint16_t* p, float x) { *p = (uint16_t)pack_bf16(x, 0.f); }

// 2^x, never 0: an infinite value keeps its sign whatever its weight (0 times it
// would be a NaN); a finite one's share is at most 2^-149 of it too much
__device__ __forceinline__ float least(float w) { return w == 0.f ? __uint_as_float(1u) : w; }
__device__ __forceinline__ float weight(float x) { return least(exp2f(x)); }

constexpr int kCcThreads = 128;

// One CTA: 16 rows x 32 positions a tile, K and then V staged as fp32 in
// shared memory.  Not the bytes bound it but a group's few rows against
// every position in fp32 through shared memory: 64 sequences x 3 rows of fp32
// queries over 4096 positions of an e4m3 cache (16 heads, 4 KV heads of 256)
// take 2060 us, where the tensor cores take 98 for bf16 queries; one sequence x
// 4 rows over 8192 positions of a bf16 cache 72 us.  Warp w scores rows 4w..4w+3
// with lane = position; thread d owns output dimensions d, d + 128, .. of all 16
// rows.
template <typename QT, typename KT>
__global__ void __launch_bounds__(kCcThreads) paged_attn_cc_kernel(const __grid_constant__ PagedAttnArgs a) {
    extern __shared__ __align__(16) float sm[];
    const int hd = a.hd, pitch = hd + 4, U = hd >> 4;
    float* sq = sm;                               // [16][hd]
    float* skv = sq + kCcRows * hd;               // [32][pitch]
    float* sp = skv + kCcTile * pitch;            // [16][32]
    float* sf = sp + kCcRows * kCcTile;           // [16] rescale factors
    Plan plan;
    plan.pre = reinterpret_cast<long long*>(sf + kCcRows);
    plan.len = reinterpret_cast<int2*>(plan.pre + a.B + 1);
    __shared__ long long tmp[kPlanTmp];
    __shared__ const KT *skp[kCcTile], *svp[kCcTile];   // a position's K and V rows (null: absent)
    __shared__ float sks[kCcTile], svs[kCcTile];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    bool bad = !schedule<kCcThreads>(a, plan, tmp) && blockIdx.x == 0;
    int4 split = make_int4(0, 0, 0, -1);
    const long long T = plan.pre[a.B];
    long long x = share_lo(T, blockIdx.x, a.grid);
    const long long xe = share_lo(T, blockIdx.x + 1, a.grid);
    const QT* q = reinterpret_cast<const QT*>(a.q);
    while (x < xe) {
        const Segment s = segment_at(a, plan, x, xe, blockIdx.x);
        if (s.n <= 0) break;
        const int r0 = s.rt * a.RT;
        if (tid == 0) note_split(a, s, T, blockIdx.x, split);
        // queries: norm, rotation, scale
        for (int i0 = 0; i0 < kCcRows * U; i0 += kCcThreads) {
            const int i = i0 + tid, r = i / U, c = i % U;
            const bool in = r < s.rows;
            const int j = in ? (r0 + r) / a.G : 0, h = in ? (r0 + r) % a.G : 0;
            float p[8], w[8];
            const QT* src = q + s.b * a.sb + j * a.sm + (s.g * a.G + h) * a.sh + 8 * c;
            load8(src, p);
            load8(src + (hd >> 1), w);
            if (a.q_norm) unit_norm(p, w, a.q_norm, c, hd, a.eps);
            if (a.rope.on) {
                float cs[8], sn[8];
                unit_angles<false>((long long)s.len + j, a.rope.hi + 8 * c, a.rope.lo + 8 * c, cs, sn);
                unit_rotate(p, w, cs, sn);
            }
            if (r < kCcRows)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    sq[r * hd + 8 * c + e] = in ? p[e] * a.scale : 0.f;
                    sq[r * hd + (hd >> 1) + 8 * c + e] = in ? w[e] * a.scale : 0.f;
                }
        }
        float acc[kCcRows][4], m[4], l[4];
#pragma unroll
        for (int r = 0; r < kCcRows; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[r][i] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = kNoScore;
            l[i] = 0.f;
        }
        const int p_last = s.len + (r0 + s.rows - 1) / a.G;   // position of the tile's last row
        for (int k = 0; k < s.n; ++k) {
            const int t0 = tile_at(s.map, s.t0 + k) * kCcTile;
            __syncthreads();
            if (tid < kCcTile) {
                const int t = t0 + tid;
                const KT *kp = nullptr, *vp = nullptr;
                float ks = 1.f, vs = 1.f;
                if (s.rows > 0 && t <= p_last) {
                    const int pg = a.c.table[(long long)s.b * a.c.max_pages + (t >> a.c.ps_log2)];
                    bool there = (unsigned)pg < (unsigned)a.c.n_pages;
                    if (there && a.c.ks) {
                        ks = a.c.ks[(long long)pg * a.c.Hkv + s.g];
                        vs = a.c.vs[(long long)pg * a.c.Hkv + s.g];
                        there = scale_ok(ks) && scale_ok(vs);
                    }
                    if (there) {
                        const long long o = pg * a.c.sp + s.g * a.c.sh + (t & ((1 << a.c.ps_log2) - 1)) * a.c.st;
                        kp = reinterpret_cast<const KT*>(a.c.k) + o;
                        vp = reinterpret_cast<const KT*>(a.c.v) + o;
                    } else {
                        // absent: an error only where a row attends it
                        for (int r = 0; r < s.rows; r += a.G) bad = bad || attends(a.c, t, s.len + (r0 + r) / a.G);
                        bad = bad || attends(a.c, t, p_last);
                    }
                }
                skp[tid] = kp;
                svp[tid] = vp;
                sks[tid] = ks;
                svs[tid] = vs;
            }
            __syncthreads();
            auto stage = [&](const KT* const* rows, const float* sc) {
                const int per = hd >> 3;
                for (int i = tid; i < kCcTile * per; i += kCcThreads) {
                    const int t = i / per, c = i % per;
                    float v[8];
                    if (rows[t]) kv8(rows[t] + 8 * c, sc[t], v);
                    else
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = 0.f;
                    store8(skv + t * pitch + 8 * c, v);
                }
            };
            stage(skp, sks);
            __syncthreads();
            float z[4] = {0.f, 0.f, 0.f, 0.f};
            for (int d = 0; d < hd; d += 4) {
                const float4 kk = *reinterpret_cast<const float4*>(skv + lane * pitch + d);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 qq = *reinterpret_cast<const float4*>(sq + (4 * warp + i) * hd + d);
                    z[i] = fmaf(qq.x, kk.x, fmaf(qq.y, kk.y, fmaf(qq.z, kk.z, fmaf(qq.w, kk.w, z[i]))));
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 4 * warp + i;
                const bool see = r < s.rows && skp[lane] && attends(a.c, t0 + lane, s.len + (r0 + r) / a.G);
                const float v = see ? z[i] : -__int_as_float(0x7F800000);
                const float mn = fmaxf(m[i], warp_max(v));
                const float p = exp2f(v - mn);   // (the sum takes it as it is: a row of scores of -inf has none)
                const float f = weight(m[i] - mn);
                l[i] = l[i] * f + warp_sum(see ? p : 0.f);
                m[i] = mn;
                sp[r * kCcTile + lane] = see ? least(p) : -1.f;   // -1: masked, whatever the value row holds
                if (lane == 0) sf[r] = f;
            }
            __syncthreads();
            stage(svp, svs);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int d = tid + kCcThreads * i;
                if (d >= hd) break;
#pragma unroll
                for (int r = 0; r < kCcRows; ++r) acc[r][i] *= sf[r];
                for (int t = 0; t < kCcTile; ++t) {
                    const float v = skv[t * pitch + d];
#pragma unroll
                    for (int r = 0; r < kCcRows; ++r) {
                        const float p = sp[r * kCcTile + t];
                        if (!(p < 0.f)) acc[r][i] = fmaf(p, v, acc[r][i]);
                    }
                }
            }
        }
        // l of every row to all threads
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (lane == 0) {
                sf[4 * warp + i] = l[i];
                sp[4 * warp + i] = m[i];
            }
        __syncthreads();
        float* part = s.slot >= 0 ? a.part + s.slot * part_floats(a.RT, hd) : nullptr;
#pragma unroll
        for (int r = 0; r < kCcRows; ++r) {
            if (r >= s.rows) break;
            const int j = (r0 + r) / a.G, h = s.g * a.G + (r0 + r) % a.G;
            QT* o = reinterpret_cast<QT*>(a.out) + (((long long)s.b * a.M + j) * a.Hq + h) * hd;
            const float inv = sf[r] == 0.f ? 0.f : 1.f / sf[r];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int d = tid + kCcThreads * i;
                if (d >= hd) break;
                if (part) part[r * hd + d] = acc[r][i];
                else put(o + d, acc[r][i] * inv);
            }
            if (part && tid == 0) {
                part[a.RT * hd + r] = sp[r];
                part[a.RT * (hd + 1) + r] = sf[r];
            }
        }
        x = s.next;
    }
    const int any = __syncthreads_or(bad);
    if (tid == 0) {
        a.cta_status[blockIdx.x] = any ? MTP_ERR_ARG : MTP_OK;
        if (!a.by_item) a.split[blockIdx.x] = split;
    }
}

// ---------------------------------------------------------------------------
// merge: a CTA takes one row of an item that begins in CTA c0's share of the
// attention and ends in CTA c1's (an item that one CTA held whole is written
// already).  out = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s.  The
// parts are spread over the CTA's thread groups (hd / 4 threads each, four
// dimensions a thread), eight a turn with all their loads in flight, so it is
// bound by the latency of two dependent loads: the item, then its parts.  It
// takes 4.7 to 7.1 us alone, of which two to three lie behind the attention's end
// (its CTAs are in place by then).
// ---------------------------------------------------------------------------
constexpr int kMergeThreads = 512, kMergeBatch = 8;   // threads at most

__device__ __forceinline__ void put4(float* p, const float4& x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void put4(uint16_t* p, const float4& x) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
}

template <typename QT>
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const __grid_constant__ PagedAttnArgs a) {
    __shared__ float4 s_o[kMergeThreads];
    __shared__ float2 s_ml[kMergeThreads];
    const int tid = threadIdx.x;
    const int idx = (int)(blockIdx.x / (unsigned)a.rows_max), r = (int)blockIdx.x - idx * a.rows_max, hd = a.hd;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x == gridDim.x - 1) {   // the call's status from the CTAs'
        int bad = 0;
        for (int c = tid; c < a.grid; c += (int)blockDim.x) {
            const int st = a.cta_status[c];
            if (st == MTP_ERR_TIMEOUT) bad |= 2;
            else if (st != MTP_OK) bad |= 1;
        }
        const int any1 = __syncthreads_or(bad & 1), any2 = __syncthreads_or(bad & 2);
        if (tid == 0) {
            a.hdr->status = any2 ? MTP_ERR_TIMEOUT : (any1 ? MTP_ERR_ARG : MTP_OK);
            a.hdr->barrier = 0;
            a.hdr->done = 0;
        }
        return;
    }
    const int4 it = a.split[idx];
    if (a.by_item) {   // an item without tiles has no note
        const int ib = (int)udiv((unsigned)idx, (unsigned)(a.c.Hkv * item_tiles(a))), len = a.kv_len[ib], n = a.n_new ? a.n_new[ib] : a.M;
        if (!seq_ok(len, n, a.M, a.c) || n * a.G <= (idx % item_tiles(a)) << a.rt_log2) return;
    }
    const int c0 = it.z, c1 = it.w;
    // (an attention that gave up may have left no note: whatever is there stays in bounds)
    if (c1 < 0 || c0 < 0 || c0 >= a.grid || c1 >= a.grid || r >= it.y >> 16 || (it.y & 0xFFFF) + r >= a.M * a.G || it.x < 0 ||
        it.x >= a.B * a.c.Hkv)
        return;
    const long long psz = part_floats(a.RT, hd);
    auto slot = [&](int c) { return a.part + (c == c0 ? 2 * c + 1 : 2 * c) * psz; };
    const int gt = hd >> 2, groups = (int)blockDim.x / gt;   // threads of a group, groups
    const int my = tid / gt, d = 4 * (tid - my * gt);
    float M = kNoScore, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int cb = c0 + my; cb <= c1; cb += kMergeBatch * groups) {
        float m[kMergeBatch], ls[kMergeBatch];
        float4 o[kMergeBatch];
#pragma unroll
        for (int k = 0; k < kMergeBatch; ++k) {
            const int c = cb + k * groups;
            m[k] = kNoScore;
            ls[k] = 0.f;
            o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c > c1) continue;
            const float* p = slot(c);
            m[k] = p[a.RT * hd + r];
            ls[k] = p[a.RT * (hd + 1) + r];
            o[k] = *reinterpret_cast<const float4*>(p + r * hd + d);
        }
        float nm = M;
#pragma unroll
        for (int k = 0; k < kMergeBatch; ++k) nm = fmaxf(nm, m[k]);
        const float f = weight(M - nm);
        acc.x *= f;
        acc.y *= f;
        acc.z *= f;
        acc.w *= f;
        l *= f;
        M = nm;
#pragma unroll
        for (int k = 0; k < kMergeBatch; ++k) {
            const float w = weight(m[k] - nm);
            acc.x = fmaf(w, o[k].x, acc.x);
            acc.y = fmaf(w, o[k].y, acc.y);
            acc.z = fmaf(w, o[k].z, acc.z);
            acc.w = fmaf(w, o[k].w, acc.w);
            l = fmaf(w, ls[k], l);
        }
    }
    s_o[tid] = acc;
    s_ml[tid] = make_float2(M, l);
    __syncthreads();
    if (tid >= gt) return;
    for (int k = 0; k < groups; ++k) M = fmaxf(M, s_ml[tid + k * gt].x);
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    l = 0.f;
    for (int k = 0; k < groups; ++k) {
        const float2 ml = s_ml[tid + k * gt];
        const float4 o = s_o[tid + k * gt];
        const float w = weight(ml.x - M);
        acc.x = fmaf(w, o.x, acc.x);
        acc.y = fmaf(w, o.y, acc.y);
        acc.z = fmaf(w, o.z, acc.z);
        acc.w = fmaf(w, o.w, acc.w);
        l = fmaf(w, ml.y, l);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    acc.x *= inv;
    acc.y *= inv;
    acc.z *= inv;
    acc.w *= inv;
    const int rr = (it.y & 0xFFFF) + r, j = (int)udiv((unsigned)rr, (unsigned)a.G), b = it.x / a.c.Hkv, g = it.x - b * a.c.Hkv;
    QT* o = reinterpret_cast<QT*>(a.out) + (((long long)b * a.M + j) * a.Hq + g * a.G + rr - j * a.G) * hd;
    put4(o + d, acc);
}

namespace {
size_t cc_smem(const PagedAttnArgs& a) {
    return ((size_t)kCcRows * a.hd + (size_t)kCcTile * (a.hd + 4) + kCcRows * kCcTile + kCcRows) * sizeof(float) +
           (size_t)plan_bytes(a.B);
}
// most that any call asks for
constexpr int kCcSmemMax = (kCcRows * 512 + kCcTile * (512 + 4) + kCcRows * kCcTile + kCcRows) * (int)sizeof(float) + plan_bytes(MTP_MAX_PAGED_BATCH);
template <typename QT, typename KT>
cudaError_t cc(const PagedAttnArgs& a, cudaStream_t s) {
    // the most, so that calls of two sizes from two host threads do not disturb each other
    const cudaError_t e = cudaFuncSetAttribute(paged_attn_cc_kernel<QT, KT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kCcSmemMax);
    if (e != cudaSuccess) return e;
    paged_attn_cc_kernel<QT, KT><<<a.grid, kCcThreads, cc_smem(a), s>>>(a);
    return cudaGetLastError();
}
template <typename QT>
cudaError_t cc_kv(const PagedAttnArgs& a, int kv_dtype, cudaStream_t s) {
    return kv_dtype == MTP_DTYPE_F32 ? cc<QT, float>(a, s) : kv_dtype == MTP_DTYPE_BF16 ? cc<QT, uint16_t>(a, s) : cc<QT, uint8_t>(a, s);
}
}  // namespace

cudaError_t launch_paged_attn_cc(const PagedAttnArgs& a, int dtype, int kv_dtype, cudaStream_t s) {
    return dtype == MTP_DTYPE_F32 ? cc_kv<float>(a, kv_dtype, s) : cc_kv<uint16_t>(a, kv_dtype, s);
}

cudaError_t launch_paged_merge(const PagedAttnArgs& a, int dtype, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    const long long items = (long long)a.B * a.c.Hkv * ((a.M * a.G + a.RT - 1) / a.RT);
    cfg.gridDim = dim3((unsigned)(a.by_item ? items : a.grid) * a.rows_max + 1);
    // items cut into eight parts or more: more parts in flight (38 parts of 16 rows: 16.4 us a call, 20.5 with 128)
    cfg.blockDim = dim3(items * 8 <= a.grid ? kMergeThreads : 128);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // its CTAs come in while the attention ends
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return dtype == MTP_DTYPE_F32 ? cudaLaunchKernelEx(&cfg, paged_merge_kernel<float>, a)
                                  : cudaLaunchKernelEx(&cfg, paged_merge_kernel<uint16_t>, a);
}

}  // namespace mtp
