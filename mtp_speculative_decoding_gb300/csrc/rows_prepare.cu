// rows_prepare.cu -- what the attention of many rows on the tensor cores starts
// from: the rows as operands (normed, rotated, rounded once), and the plan of the
// call (see rows_attn_tc.cuh), by one CTA of the same launch.
//
// The rows of an item end up one after another, whatever the heads of a group are,
// so the attention fetches them by tensor copies.  Norm and rotation inside the
// attention kernel cost it 15 us an item (256 rows x 256) between two pieces of
// work; here they cost their bytes: 12288 rows of 16 heads of 256, 201 MB in and out,
// take 50 us behind a flushed cache (4 TB/s).  Fewer heads a thread (8, 4), two in
// flight instead of four, three or four CTAs an SM instead of two measured the same.
// With few rows the plan's chain of scans and searches is what takes time: run a second
// time, its parts lengthen a call of 4 sequences behind a prefix by 8 us.
#include "rows_attn_tc.cuh"

namespace mtp {

namespace {

constexpr int kPrepThreads = 256;

// group_start and prefix_len, copied to shared memory; prompts whose row_start does not
// ascend: whether a sequence's rows are its alone (otherwise null)
struct Groups { const int32_t *start, *len, *alone; };
__device__ __forceinline__ bool seq_at(const RowsArgs& a, int b, Seq& s, const Groups& gr) {
    bool ok = seq_at(a, b, s, gr.start, gr.len);
    if (gr.alone && !gr.alone[b]) {
        s.n = 0;
        ok = false;
    }
    return ok;
}

// The plan's code runs once a call, on one SM, and its instructions come from memory each
// time: no loop is unrolled and nothing is computed twice (8192 prompt rows: 360 to 352 us;
// 64 sequences behind a prefix: 56.4 to 55.1).  Out of line, with its structs on the stack, it
// is slower (57.0 to 59.3).

// sums of v over the threads in front of this one, and over all of the CTA
__device__ __forceinline__ long long scan(long long v, long long* s, long long& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long inc = v;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    __syncthreads();
    if (lane == 31) s[warp] = inc;
    __syncthreads();
    long long base = inc - v;
    total = 0;
#pragma unroll 1
    for (int w = 0; w < kPrepThreads / 32; ++w) {
        if (w < warp) base += s[w];
        total += s[w];
    }
    return base;
}

// own tiles of a sequence
__device__ __forceinline__ int own_tiles(const Seq& s) { return s.n > 0 ? (s.len + s.n - 1) / kPosTile - s.P / kPosTile + 1 : 0; }

// Tokens and own tiles before every sequence, cached positions (shared prefixes); false
// if this thread saw something out of range.  cumt, lens null: tokens alone.
__device__ __forceinline__ bool count_tokens(const RowsArgs& a, const Groups& gr, int* cum, int* cumt, int* lens, long long* tmp) {
    bool good = true;
    const int per = (a.B + kPrepThreads - 1) / kPrepThreads, b0 = (int)threadIdx.x * per, b1 = b0 + per < a.B ? b0 + per : a.B;
    long long sum = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        Seq s;
        good = seq_at(a, b, s, gr) && good;
        const int tl = own_tiles(s);
        cum[b] = s.n;
        if (cumt) {
            cumt[b] = tl;
            lens[b] = s.len;
        }
        sum += (long long)s.n << 40 | tl;          // (at most 2^16 tokens, 2^31 tiles)
    }
    long long all;
    const long long before = scan(sum, tmp, all);
    int at = (int)(before >> 40), tat = (int)(before & 0xFFFFFFFFFFll);
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        const int n = cum[b];
        cum[b] = at;
        at += n;
        if (cumt) {
            const int tl = cumt[b];
            cumt[b] = tat;
            tat += tl;
        }
    }
    if (threadIdx.x == 0) {
        cum[a.B] = (int)(all >> 40);
        if (cumt) cumt[a.B] = (int)(all & 0xFFFFFFFFFFll);
    }
    __syncthreads();
    return good;
}

// The staged row of (sequence, token 0, KV head 0), and the rows of a KV head there.
// Prompts: a sequence's own rows.  Shared prefixes: its group's.
struct StagedAt { long long row; int stride; };
__device__ __forceinline__ StagedAt staged_at(const RowsArgs& a, const Groups& gr, const int* cum, const Seq& s, int b) {
    StagedAt w;
    if (a.M == 0) {
        w.row = s.row0 * a.Hq;
        w.stride = s.n * a.G;
    } else {
        const int g0 = s.group >= 0 ? s.first : b, g1 = s.group >= 0 ? gr.start[s.group + 1] : b + 1;
        w.stride = (cum[g1] - cum[g0]) * a.G;
        w.row = (long long)cum[g0] * a.Hq + (cum[b] - cum[g0]) * a.G;
    }
    return w;
}

__device__ __forceinline__ BlockRec block_at(const RowsArgs& a, const Groups& gr, const int* cum, int blk, bool& good) {
    BlockRec k = {};
    if (blk < 2 * a.n_groups) {
        const bool own = blk >= a.n_groups;
        const int i = own ? blk - a.n_groups : blk, g0 = gr.start[i], g1 = gr.start[i + 1], P = gr.len[i];
        // (a group that is out of range is reported by the sequences in it: one without any concerns no one)
        const bool ok = g0 >= 0 && g0 <= g1 && g1 <= a.B && P >= 0 && P <= (long long)a.c.max_pages << a.c.ps_log2;
        k.kind = own ? kOwn : kPrefix;
        if (ok) {
            k.n = own || P > 0 ? cum[g1] - cum[g0] : 0;
            k.len = own ? g1 : 0;
            k.lo = own ? P : 0;
            k.hi = own ? 0 : P;
            k.table = g0;
            k.q_stride = (cum[g1] - cum[g0]) * a.G;
            k.q_row = (long long)cum[g0] * a.Hq;
        }
        return k;
    }
    Seq s;
    const int b = blk - 2 * a.n_groups;
    good = seq_at(a, b, s, gr) && good;
    k.table = b;
    if (s.n > 0 && s.group < 0) {
        const StagedAt w = staged_at(a, gr, cum, s, b);
        k.n = s.n;
        k.len = s.len;
        k.hi = s.len + s.n;
        k.q_stride = w.stride;
        k.q_row = w.row;
        k.row0 = (int)s.row0;
    }
    return k;
}

// The tiles before each item of the groups' own positions, group by group, and the
// groups' first entries (rt0: [n_groups + 1] row tiles before a group)
__device__ void count_items(const RowsTcArgs& t, const Groups& gr, const Sequences& sq, int* rt0, long long* tmp) {
    const RowsArgs& a = t.a;
    bool good = true;
    const int tid = threadIdx.x, per = (a.n_groups + kPrepThreads - 1) / kPrepThreads, i0 = tid * per,
              i1 = i0 + per < a.n_groups ? i0 + per : a.n_groups;
    long long sum = 0, all;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) sum += rt0[i] = row_tiles_of(a, block_at(a, gr, sq.cum, a.n_groups + i, good));
    int at = (int)scan(sum, tmp, all);
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
        const int n = rt0[i];
        rt0[i] = at;
        at += n;
    }
    if (tid == 0) rt0[a.n_groups] = (int)all;
    __syncthreads();
    const int items = (int)all, pi = (items + kPrepThreads - 1) / kPrepThreads, x0 = tid * pi, x1 = x0 + pi < items ? x0 + pi : items;
    sum = 0;
#pragma unroll 1
    for (int x = x0; x < x1; ++x) {
        const int i = last_at_most(rt0, a.n_groups, x);
        sum += t.items[x] = item_of<true>(a, sq, block_at(a, gr, sq.cum, a.n_groups + i, good), x - rt0[i]).n;
    }
    long long before = scan(sum, tmp, all);
#pragma unroll 1
    for (int x = x0; x < x1; ++x) {
        const long long n = t.items[x];
        t.items[x] = before;
        before += n;
    }
    if (tid == 0) t.items[items] = all;
    __syncthreads();
}

__device__ void make_plan(const RowsTcArgs& t, const Groups& gr, const int* cum, const int* rt0, long long* tmp, long long* pre, int* nrt, bool good) {
    const RowsArgs& a = t.a;
    const int tid = threadIdx.x, nb = rows_blocks(a), per = (nb + kPrepThreads - 1) / kPrepThreads, k0 = tid * per,
              k1 = k0 + per < nb ? k0 + per : nb;
    const long long U = (long long)kPosTile * a.G;
    long long tiles = 0, items = 0;
#pragma unroll 1
    for (int i = k0; i < k1; ++i) {
        BlockRec k = block_at(a, gr, cum, i, good);
        if (k.kind == kOwn) k.row0 = rt0[i - a.n_groups];
        t.blocks[i] = k;
        nrt[i] = row_tiles_of(a, k);
        pre[i] = a.c.Hkv * tile_units(t, k, nrt[i]);
        tiles += pre[i];
        items += (long long)a.c.Hkv * nrt[i];
    }
    long long units, n_items;
    long long at = scan(tiles, tmp, units);
    const long long it = scan(items, tmp, n_items);
    // where a share is few tiles, how they spread counts for more
    int open = kRowsOpen;
    while (open > 0 && 2ll * open * U * t.workers > units) --open;
    at += it * open * U;
    const long long T = units + n_items * open * U, most = quotient(T, U);
    const int workers = most < t.workers ? (most > 1 ? (int)most : 1) : t.workers;
#pragma unroll 1
    for (int i = k0; i < k1; ++i) {
        const long long u = pre[i] + (long long)a.c.Hkv * nrt[i] * open * U;
        pre[i] = at;
        t.blocks[i].pre = at;
        at += u;
    }
    __syncthreads();   // (the records of the other threads too)
    const long long base = quotient(T, workers), rem = T - base * workers;   // (see worker_of)
#pragma unroll 1
    for (int w = tid; w < t.workers; w += kPrepThreads) {
        WorkerRec r = {};
        r.open = open;
        r.xs = w < workers ? base * w + (w < rem ? w : rem) : T;
        r.xe = w < workers ? base * (w + 1) + (w + 1 < rem ? w + 1 : rem) : T;
        if (r.xs < r.xe) {
            int b = 0;
            for (int hi = nb - 1; b < hi;) {   // the last block that begins at xs or before
                const int mid = (b + hi + 1) >> 1;
                if (pre[mid] <= r.xs) b = mid;
                else hi = mid - 1;
            }
            const BlockRec k = t.blocks[b];
            const long long head = units_before(t, k, open, nrt[b]);
            long long rel = r.xs - pre[b];
            const int g = (int)quotient(rel, head);
            rel -= g * head;
            int rt = 0;
            for (int hi = nrt[b] - 1; rt < hi;) {
                const int mid = (rt + hi + 1) >> 1;
                if (units_before(t, k, open, mid) <= rel) rt = mid;
                else hi = mid - 1;
            }
            r.blk = b;
            r.g = g;
            r.rt = rt;
            r.begin = pre[b] + g * head + units_before(t, k, open, rt);
            r.k = k;
        } else {
            r.begin = T;
        }
        t.worker[w] = r;
    }
    if (tid == 0) {
        PlanHead h;
        h.T = T;
        h.open = open;
        h.workers = workers;
        *t.head = h;
    }
    const int any = __syncthreads_or(!good);
    if (tid == 0) t.cta_status[t.workers * rows_pair(a.hd)] = any ? MTP_ERR_ARG : MTP_OK;
}

__host__ __device__ constexpr size_t prep_ints(int B, int n_groups) { return (((size_t)4 * B + 5 * n_groups + 8) * 4 + 7) / 8 * 8; }

template <bool E4M3>
__global__ void __launch_bounds__(kPrepThreads) rows_prepare_kernel(const __grid_constant__ RowsTcArgs t, int hpt) {
    extern __shared__ __align__(16) unsigned char sm[];
    __shared__ long long tmp[kPrepThreads / 32];
    __shared__ __align__(16) float s_hi[256], s_lo[256];
    const RowsArgs& a = t.a;
    int* cum = reinterpret_cast<int*>(sm);                                     // [B + 1] prompts: row_start
    int *g_start = cum + a.B + 1, *g_len = g_start + a.n_groups + 1;           // [n_groups + 1], [n_groups]
    // the plan's CTA: own tiles before a sequence, cached positions, row tiles before a group and of a block, units before a block
    int *cumt = g_len + a.n_groups, *lens = cumt + a.B + 1, *rt0 = lens + a.B, *nrt = rt0 + a.n_groups + 1;
    long long* pre = reinterpret_cast<long long*>(sm + prep_ints(a.B, a.n_groups));
    Groups gr = {g_start, g_len, nullptr};
    const int tid = threadIdx.x;
    const bool planner = blockIdx.x == 0;
    if (a.rope.on && !planner)
        for (int i = tid; i < a.hd >> 1; i += kPrepThreads) {
            s_hi[i] = a.rope.hi[i];
            s_lo[i] = a.rope.lo[i];
        }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    bool good = true;
    if (a.n_groups > 0) {
        bool ascend = true;
        for (int i = tid; i <= a.n_groups; i += kPrepThreads) {
            g_start[i] = a.group_start[i];
            if (i < a.n_groups) {
                g_len[i] = a.prefix_len[i];
                ascend = ascend && g_start[i] <= a.group_start[i + 1];
            }
        }
        // groups that overlap could be more items than the plan has room for: one group of all
        // sequences with no possible prefix then, so that all are left out
        if (!__syncthreads_and(ascend)) {
            for (int i = tid; i <= a.n_groups; i += kPrepThreads) {
                g_start[i] = i > 0 ? a.B : 0;
                if (i < a.n_groups) g_len[i] = -1;
            }
            __syncthreads();
        }
    }
    if (a.M > 0) good = count_tokens(a, gr, cum, planner ? cumt : nullptr, planner ? lens : nullptr, tmp);
    else {
        bool ascend = true;
        for (int i = tid; i <= a.B; i += kPrepThreads) {
            cum[i] = a.row_start[i];
            ascend = ascend && (i == 0 || a.row_start[i - 1] <= cum[i]);
        }
        // rows of two sequences would be staged over one another (KV head by KV head: over
        // other tokens' rows too)
        if (!__syncthreads_and(ascend)) {
            for (int b = tid; b < a.B; b += kPrepThreads) {
                bool alone = true;
                for (int i = 0; i <= a.B; ++i) alone = alone && bound_agrees(cum, b, i);
                lens[b] = alone;
            }
            gr.alone = lens;
        }
    }
    __syncthreads();
    if (planner) {
        if (a.M > 0) {
            for (int i = tid; i <= a.B; i += kPrepThreads) {
                t.cum[i] = cum[i];
                t.cumt[i] = cumt[i];
                if (i < a.B) t.lens[i] = lens[i];
            }
            count_items(t, gr, Sequences{cum, cumt, lens}, rt0, tmp);
        }
        make_plan(t, gr, cum, rt0, tmp, pre, nrt, good);
        return;
    }
    const int hd = a.hd, U = hd >> 4, ulog = 31 - __clz(U), groups = (a.Hq + hpt - 1) / hpt, half = hd >> 1;
    const long long x = ((long long)(blockIdx.x - 1) * kPrepThreads + tid) >> ulog;
    const int c = tid & (U - 1), toks = a.M > 0 ? a.B * a.M : a.T;
    int tok = (int)(x / groups);
    const int h0 = (int)(x - (long long)tok * groups) * hpt;
    // (whole rows' lanes are out of range together; all lanes go along for the shuffles)
    bool live = tok < toks;
    const bool there = live;
    if (!live) tok = toks - 1;
    const int b = a.M > 0 ? tok / a.M : last_at_most(cum, a.B, tok);
    Seq s;
    live = seq_at(a, b, s, gr) && live;
    const int j = (int)(tok - s.row0);
    live = live && j >= 0 && j < s.n;
    // prompts' rows that the attention does not come to: not marked either
    if (a.M == 0 && there && !live && c == 0)
        for (int h = h0; h < h0 + hpt && h < a.Hq; ++h) {
            t.odd[(long long)tok * a.Hq + h] = 0;
            if (rows_halves(hd) > 1) t.odd[t.odd_plane + (long long)tok * a.Hq + h] = 0;
        }
    if (!__any_sync(0xffffffffu, live)) return;
    const StagedAt w = live ? staged_at(a, gr, cum, s, b) : StagedAt{0, 0};
    const long long src0 = live ? s.q0 + j * a.sm : 0;
    float cs[8], sn[8];
    if (a.rope.on) unit_angles<true>((long long)(live ? s.len + j : 0), s_hi + 8 * c, s_lo + 8 * c, cs, sn);
    float g0[8], g1[8];
    if (a.q_norm)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            g0[i] = __ldg(a.q_norm + 8 * c + i);
            g1[i] = __ldg(a.q_norm + half + 8 * c + i);
        }
    constexpr int N = 4;   // heads in flight
#pragma unroll 1
    for (int i0 = 0; i0 < hpt; i0 += N) {
        uint4 raw[N][2];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int h = h0 + i0 + i < a.Hq ? h0 + i0 + i : a.Hq - 1;
            const uint16_t* src = reinterpret_cast<const uint16_t*>(a.q) + (live ? src0 + h * a.sh : 0) + 8 * c;
            raw[i][0] = ld_stream16(src);
            raw[i][1] = ld_stream16(src + half);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i0 + i >= hpt) break;
            const int h = h0 + i0 + i;
            float p[8], q[8];
            open_unit(raw[i][0], p);
            open_unit(raw[i][1], q);
            if (a.q_norm) {
                const float r = unit_rms(p, q, hd, a.eps);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    p[e] *= r * g0[e];
                    q[e] *= r * g1[e];
                }
            }
            if (a.rope.on) unit_rotate(p, q, cs, sn);
            const int g = (int)udiv((unsigned)h, (unsigned)a.G);
            const long long row = w.row + (long long)g * w.stride + j * a.G + h - g * a.G;
            const bool mine = live && h < a.Hq;
            uint4 o[2];
            if (E4M3) {   // the largest of the row into [128, 256): no bits lost to fp16's range
                float big = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) big = fmaxf(big, fmaxf(fabsf(p[e]), fabsf(q[e])));
                for (int k = U >> 1; k > 0; k >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, k));
                int x2 = (int)(__float_as_uint(big) >> 23) - 127 - 7;
                x2 = x2 < -100 ? -100 : x2 > 100 ? 100 : x2;
                const float f = __uint_as_float((uint32_t)(127 - x2) << 23);
                if (mine && c == 0) t.q_scale[row] = __uint_as_float((uint32_t)(127 + x2) << 23) * a.scale;
                auto half2 = [&](float lo, float hi) {
                    uint32_t r;
                    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi * f), "f"(lo * f));
                    return r;
                };
                o[0] = make_uint4(half2(p[0], p[1]), half2(p[2], p[3]), half2(p[4], p[5]), half2(p[6], p[7]));
                o[1] = make_uint4(half2(q[0], q[1]), half2(q[2], q[3]), half2(q[4], q[5]), half2(q[6], q[7]));
            } else {
                o[0] = make_uint4(pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3]), pack_bf16(p[4], p[5]), pack_bf16(p[6], p[7]));
                o[1] = make_uint4(pack_bf16(q[0], q[1]), pack_bf16(q[2], q[3]), pack_bf16(q[4], q[5]), pack_bf16(q[6], q[7]));
            }
            if (mine) {
                uint16_t* dst = t.staged + row * hd + 8 * c;
                *reinterpret_cast<uint4*>(dst) = o[0];
                *reinterpret_cast<uint4*>(dst + half) = o[1];
            }
        }
    }
}

}  // namespace

cudaError_t launch_rows_prepare(const RowsTcArgs& t, int kv_dtype, int sms, cudaStream_t s) {
    const RowsArgs& a = t.a;
    const long long toks = a.M > 0 ? (long long)a.B * a.M : a.T;
    const int U = a.hd >> 4;
    // as many heads in one thread as leave 512 threads an SM: the angles of a row are
    // computed once for them
    int hpt = 1;
    while (hpt < a.Hq && toks * U * ((a.Hq + 2 * hpt - 1) / (2 * hpt)) >= (long long)sms * 512) hpt *= 2;
    const long long threads = toks * U * ((a.Hq + hpt - 1) / hpt);
    const int ctas = (int)((threads + kPrepThreads - 1) / kPrepThreads);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas + 1);
    cfg.blockDim = dim3(kPrepThreads);
    cfg.dynamicSmemBytes = prep_ints(a.B, a.n_groups) + (size_t)rows_blocks(a) * 8;
    if (cfg.dynamicSmemBytes > 40 * 1024) {   // the most, so that two host threads' calls do not disturb each other
        constexpr int most = (int)(prep_ints(MTP_MAX_PAGED_BATCH, MTP_MAX_PAGED_BATCH) + 3 * MTP_MAX_PAGED_BATCH * 8);
        const cudaError_t e = kv_dtype == MTP_DTYPE_E4M3 ? cudaFuncSetAttribute(rows_prepare_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, most)
                                                         : cudaFuncSetAttribute(rows_prepare_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return e;
    }
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return kv_dtype == MTP_DTYPE_E4M3 ? cudaLaunchKernelEx(&cfg, rows_prepare_kernel<true>, t, hpt)
                                      : cudaLaunchKernelEx(&cfg, rows_prepare_kernel<false>, t, hpt);
}

}  // namespace mtp
