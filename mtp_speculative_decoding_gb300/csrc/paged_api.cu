// paged_api.cu -- the C ABI of the paged KV cache's append and attention (a
// verify step's rows, prompts, shared prefixes), of the rotation by several
// positions and of the token log probabilities: argument checks, workspace
// layout, launches.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "common.cuh"
#include "host.cuh"
#include "logprobs.cuh"
#include "mtp.h"
#include "paged.cuh"
#include "paged_attn_tc.cuh"
#include "rows_attn_tc.cuh"

using namespace mtp;

namespace {

constexpr unsigned long long kWaitLimitNs = 1000000000ull;   // 1 s per wait inside a kernel

size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }
bool misaligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }
int elem_size(int dtype) { return dtype == MTP_DTYPE_F32 ? 4 : dtype == MTP_DTYPE_BF16 ? 2 : 1; }

int check_cache(const mtp_kv_cache* c, bool pointers) {
    if (!c) return MTP_ERR_ARG;
    if (c->kv_dtype != MTP_DTYPE_F32 && c->kv_dtype != MTP_DTYPE_BF16 && c->kv_dtype != MTP_DTYPE_E4M3) return MTP_ERR_UNSUPPORTED;
    if (c->n_pages < 1 || c->max_pages < 1 || c->n_kv_heads < 1 || c->page_size < 1) return MTP_ERR_ARG;
    const int hd = c->head_dim;
    if (hd != 32 && hd != 64 && hd != 128 && hd != 256 && hd != 512) return MTP_ERR_UNSUPPORTED;
    if (c->page_size < 16 || c->page_size > MTP_MAX_PAGE_SIZE || (c->page_size & (c->page_size - 1))) return MTP_ERR_UNSUPPORTED;
    if (c->n_kv_heads > 1024) return MTP_ERR_UNSUPPORTED;
    if (c->window < 0 || c->sink < 0 || (c->window == 0 && c->sink != 0)) return MTP_ERR_ARG;
    if (!(c->rope_theta >= 0.f) || isinf(c->rope_theta)) return MTP_ERR_ARG;
    if ((long long)c->max_pages * c->page_size > 0x7FFFFF00ll) return MTP_ERR_UNSUPPORTED;   // positions are 31-bit
    const int esz = elem_size(c->kv_dtype);
    if (c->stride_t < hd || c->stride_h < 0 || c->stride_p < 0) return MTP_ERR_ARG;
    if ((c->stride_t * esz) % 16 || (c->stride_h * esz) % 16 || (c->stride_p * esz) % 16) return MTP_ERR_ARG;
    if (pointers) {
        if (!c->k || !c->v || misaligned(c->k, 16) || misaligned(c->v, 16)) return MTP_ERR_ARG;
        if (!c->page_table || misaligned(c->page_table, 4)) return MTP_ERR_ARG;
        if (c->kv_dtype == MTP_DTYPE_E4M3 && (!c->k_scale || !c->v_scale || misaligned(c->k_scale, 4) || misaligned(c->v_scale, 4)))
            return MTP_ERR_ARG;
    }
    return MTP_OK;
}

int check_rows(const void* p, int dtype, int64_t sb, int64_t sm, int64_t sh) {
    if (!p || misaligned(p, 16)) return MTP_ERR_ARG;
    const int esz = elem_size(dtype);
    if (sb < 0 || sm < 0 || sh < 0 || (sb * esz) % 16 || (sm * esz) % 16 || (sh * esz) % 16) return MTP_ERR_ARG;
    return MTP_OK;
}

PagedKV device_cache(const mtp_kv_cache* c) {
    PagedKV d;
    d.k = c->k; d.v = c->v;
    d.ks = c->kv_dtype == MTP_DTYPE_E4M3 ? c->k_scale : nullptr;
    d.vs = c->kv_dtype == MTP_DTYPE_E4M3 ? c->v_scale : nullptr;
    d.table = c->page_table;
    d.sp = c->stride_p; d.sh = c->stride_h; d.st = c->stride_t;
    d.n_pages = c->n_pages; d.max_pages = c->max_pages; d.Hkv = c->n_kv_heads;
    d.ps_log2 = 0;
    while ((1 << d.ps_log2) < c->page_size) ++d.ps_log2;
    d.window = c->window; d.sink = c->sink;
    return d;
}

// turns per position of every pair, in two floats: powers of theta^(-2/hd) by
// repeated products in double (relative error below hd/2 * 2^-52)
void fill_rope(RopeTab* t, float theta, int hd) {
    t->on = theta > 0.f;
    if (!t->on) return;
    const double step = pow((double)theta, -2.0 / hd);
    double f = 1.0 / 6.283185307179586476925;
    for (int i = 0; i < hd / 2; ++i) {
        t->hi[i] = (float)f;
        t->lo[i] = (float)(f - (double)t->hi[i]);
        f *= step;
    }
}

// Tensor cores: bf16 queries, bf16 or e4m3 cache, head dimensions with a
// 64-element multiple
bool tc_path(const mtp_kv_cache* c, int dtype) {
    return dtype == MTP_DTYPE_BF16 && c->kv_dtype != MTP_DTYPE_F32 && c->head_dim >= 64;
}

// (dimension, slot, KV head, page) map of k or v: boxes of one 128-byte (64 for
// rows of 64 bytes) swizzled column by min(page_size, rows) slots
bool encode_pages(CUtensorMap* m, const void* base, const mtp_kv_cache* c, int rows = kTcTile) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const int esz = elem_size(c->kv_dtype);
    const uint64_t row = (uint64_t)c->head_dim * esz;
    const int box_bytes = row < 128 ? (int)row : 128;
    const cuuint64_t dims[4] = {(cuuint64_t)c->head_dim, (cuuint64_t)c->page_size, (cuuint64_t)c->n_kv_heads, (cuuint64_t)c->n_pages};
    // a stride that no index uses may be anything: give it a legal value
    const cuuint64_t strides[3] = {(cuuint64_t)c->stride_t * esz, c->n_kv_heads > 1 ? (cuuint64_t)c->stride_h * esz : row,
                                   c->n_pages > 1 ? (cuuint64_t)c->stride_p * esz : row};
    const cuuint32_t box[4] = {(cuuint32_t)(box_bytes / esz), (cuuint32_t)(c->page_size < rows ? c->page_size : rows), 1, 1};
    const cuuint32_t one[4] = {1, 1, 1, 1};
    return encoded([&] {
        return enc(m, esz == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims,
                   strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    });
}

// (dimension, row) map of staged rows of 16-bit values: boxes of a 128-byte column by 128 rows
bool encode_rows(CUtensorMap* m, void* base, int hd, int64_t rows) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)hd, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)hd * 2};
    const cuuint32_t box[2] = {64, 128}, one[2] = {1, 1};
    return encoded([&] {
        return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    });
}

struct AttnPlan {
    bool tc;
    int RT, tile_log2, grid;
    size_t status, split, part, end;
};
// (the workspace does not depend on the batch, so that one sized for more sequences serves fewer)
AttnPlan attn_plan(const mtp_kv_cache* c, int B, int M, int n_q_heads, bool tc, int sms) {
    AttnPlan p;
    p.tc = tc;
    const int rows = M * (n_q_heads / c->n_kv_heads);
    p.RT = tc ? tc_rows(c->kv_dtype == MTP_DTYPE_E4M3, rows, c->head_dim, B) : kCcRows;
    const int most = tc ? tc_rows_max(rows, c->head_dim) : kCcRows;
    p.tile_log2 = tc ? kTcTileLog2 : kCcTileLog2;
    p.grid = tc ? sms : 2 * sms;
    size_t off = sizeof(WsHeader);
    p.status = off; off = al256(off + (size_t)p.grid * sizeof(int));
    p.split = off;  off = al256(off + (size_t)p.grid * sizeof(int4));
    p.part = off;   off = al256(off + 2 * (size_t)p.grid * part_floats(most, c->head_dim) * sizeof(float));
    p.end = off;
    return p;
}

bool heads_ok(const mtp_kv_cache* c, int n_q_heads, int* rc) {
    *rc = n_q_heads < 1 || n_q_heads % c->n_kv_heads ? MTP_ERR_ARG : n_q_heads / c->n_kv_heads > 16 ? MTP_ERR_UNSUPPORTED : MTP_OK;
    return *rc == MTP_OK;
}

// prompts and shared prefixes: what both calls check and fill alike
// (on the tensor cores if the queries are bf16)
bool rows_tc(const mtp_kv_cache* c) {
    return c->kv_dtype != MTP_DTYPE_F32 && (c->head_dim == 64 || c->head_dim == 128 || c->head_dim == 256);
}
// (the tiles of shared prefixes' sequences are counted in 31 bits)
bool prefix_fits(const mtp_kv_cache* c, int B, int M, int n_q_heads) {
    const int64_t tiles = B * ((int64_t)c->max_pages * c->page_size / kPosTile + 2);
    return (int64_t)B * M * n_q_heads < 1ll << 31 && tiles < 1ll << 31;
}
struct RowsSpace {
    size_t status, note, row_parts, head, worker, blocks, items, cum, cumt, lens, staged, q_scale, odd, part, part_ml, dense, dense_ml, end;
    int workers;
};
// (every field grows with B, M and T, so that a workspace sized for more serves less)
RowsSpace rows_space(const mtp_kv_cache* c, int B, int M, int64_t T, int n_q_heads, int sms) {
    RowsSpace p = {};
    const int hd = c->head_dim;
    size_t off = sizeof(WsHeader);
    auto take = [&](size_t n) {
        const size_t at = off;
        off = al256(off + n);
        return at;
    };
    if (rows_tc(c)) {
        const size_t rows = (size_t)T * n_q_heads;
        p.workers = sms / rows_pair(hd);
        p.status = take(((size_t)sms + 1) * sizeof(int));
        p.note = take((size_t)p.workers * sizeof(RowNote));
        p.head = take(sizeof(PlanHead));
        p.worker = take((size_t)p.workers * sizeof(WorkerRec));
        p.blocks = take((M > 0 ? 3 : 1) * (size_t)B * sizeof(BlockRec));
        if (M > 0) {
            p.items = take(((size_t)B * M * (n_q_heads / c->n_kv_heads) / kRowTile + B + 2) * sizeof(long long));
            p.cum = take(((size_t)B + 1) * sizeof(int));
            p.cumt = take(((size_t)B + 1) * sizeof(int));
            p.lens = take((size_t)B * sizeof(int));
        }
        p.part_ml = take(2 * (size_t)p.workers * kRowTile * sizeof(float2));
        p.part = take(2 * (size_t)p.workers * kRowTile * hd * sizeof(float));
        p.staged = take(rows * hd * 2);
        p.q_scale = take(rows * sizeof(float));
        if (M > 0) {
            p.row_parts = take(2 * rows * sizeof(RowPart));
            p.dense_ml = take(2 * rows * sizeof(float2));
            p.dense = take(2 * rows * hd * sizeof(float));
        } else {
            p.odd = take(2 * ((rows + 4095) / 4096 * 4096));
        }
    }
    p.end = off;
    return p;
}
size_t rows_workspace(const mtp_kv_cache* c, int B, int M, int64_t T, int n_q_heads) {
    int sms = num_sms();
    if (sms <= 0) sms = 152;   // no device (a host-side size query)
    return rows_space(c, B, M, T, n_q_heads, sms).end;
}
int rows_call(const mtp_kv_cache* c, int B, int n_q_heads, const int32_t* kv_len, const void* q, int dtype, int64_t sb, int64_t sm,
              int64_t sh, const float* q_norm, float rms_eps, float attn_scale, const void* out) {
    int rc = check_cache(c, true);
    if (rc != MTP_OK) return rc;
    if (B < 1 || B > MTP_MAX_PAGED_BATCH) return MTP_ERR_ARG;
    if (!heads_ok(c, n_q_heads, &rc)) return rc;
    if (dtype != MTP_DTYPE_F32 && dtype != MTP_DTYPE_BF16) return MTP_ERR_UNSUPPORTED;
    if (!kv_len || misaligned(kv_len, 4) || misaligned(q_norm, 4)) return MTP_ERR_ARG;
    if (!(rms_eps >= 0.f) || !(attn_scale >= 0.f) || isinf(attn_scale)) return MTP_ERR_ARG;
    if ((rc = check_rows(q, dtype, sb, sm, sh)) != MTP_OK) return rc;
    return !out || misaligned(out, 16) ? MTP_ERR_ARG : MTP_OK;
}

RowsArgs rows_args(const mtp_kv_cache* c, int B, int n_q_heads, const int32_t* kv_len, const void* q, int64_t sb, int64_t sm,
                   int64_t sh, const float* q_norm, float rms_eps, float attn_scale, void* out, void* ws) {
    RowsArgs a;
    a.c = device_cache(c);
    a.hd = c->head_dim; a.B = B; a.Hq = n_q_heads; a.G = n_q_heads / c->n_kv_heads;
    a.M = 0; a.T = 0; a.n_groups = 0;
    a.kv_len = kv_len; a.n_new = nullptr; a.row_start = nullptr; a.group_start = nullptr; a.prefix_len = nullptr;
    a.q = q; a.sb = sb; a.sm = sm; a.sh = sh;
    a.q_norm = q_norm; a.eps = rms_eps;
    a.scale = (float)((attn_scale > 0.f ? (double)attn_scale : 1.0 / sqrt((double)c->head_dim)) * 1.4426950408889634074);
    a.out = out;
    a.hdr = static_cast<WsHeader*>(ws);
    fill_rope(&a.rope, c->rope_theta, c->head_dim);
    return a;
}

int launch_rows(const mtp_kv_cache* c, const RowsArgs& a, int dtype, int64_t T, void* ws, int sms, cudaStream_t s) {
    if (dtype != MTP_DTYPE_BF16 || !rows_tc(c)) return launch_rows_cc(a, dtype, c->kv_dtype, s) == cudaSuccess ? MTP_OK : MTP_ERR_CUDA;
    const RowsSpace p = rows_space(c, a.B, a.M, T, a.Hq, sms);
    char* base = static_cast<char*>(ws);
    RowsTcParams pp;
    RowsTcArgs& t = pp.t;
    t.a = a;
    t.workers = p.workers;
    const long long U = (long long)kPosTile * a.G;
    // (in 64 bits: a window or a sink may be as long as an int goes)
    t.window_units = U * ((a.c.sink + (long long)kPosTile - 1) / kPosTile + (a.c.window + (long long)(kRowTile - 1) / a.G) / kPosTile + 2);
    t.cta_status = reinterpret_cast<int*>(base + p.status);
    t.note = reinterpret_cast<RowNote*>(base + p.note);
    t.row_parts = reinterpret_cast<RowPart*>(base + p.row_parts);
    t.head = reinterpret_cast<PlanHead*>(base + p.head);
    t.worker = reinterpret_cast<WorkerRec*>(base + p.worker);
    t.blocks = reinterpret_cast<BlockRec*>(base + p.blocks);
    t.items = reinterpret_cast<long long*>(base + p.items);
    t.cum = reinterpret_cast<int*>(base + p.cum);
    t.cumt = reinterpret_cast<int*>(base + p.cumt);
    t.lens = reinterpret_cast<int*>(base + p.lens);
    t.staged = reinterpret_cast<uint16_t*>(base + p.staged);
    t.q_scale = reinterpret_cast<float*>(base + p.q_scale);
    t.part = reinterpret_cast<float*>(base + p.part);
    t.part_ml = reinterpret_cast<float2*>(base + p.part_ml);
    t.odd = reinterpret_cast<uint8_t*>(base + p.odd);
    t.odd_plane = (T * a.Hq + 4095) / 4096 * 4096;
    t.dense = reinterpret_cast<float*>(base + p.dense);
    t.dense_ml = reinterpret_cast<float2*>(base + p.dense_ml);
    t.timeout_ns = kWaitLimitNs;
    // (a stride beyond 2^40 bytes has no map)
    if (!encode_pages(&pp.tk, c->k, c, kPosTile / rows_pair(c->head_dim)) || !encode_pages(&pp.tv, c->v, c, kPosTile) ||
        !encode_rows(&pp.tq, t.staged, c->head_dim, T * a.Hq))
        return MTP_ERR_UNSUPPORTED;
    const bool e4m3 = c->kv_dtype == MTP_DTYPE_E4M3;
    if (launch_rows_prepare(t, c->kv_dtype, sms, s) != cudaSuccess) return MTP_ERR_CUDA;
    const auto launch = a.M > 0 ? (e4m3 ? launch_rows_tc_e4m3_shared : launch_rows_tc_bf16_shared) : (e4m3 ? launch_rows_tc_e4m3 : launch_rows_tc_bf16);
    if (launch(pp, s) != cudaSuccess) return MTP_ERR_CUDA;
    return launch_rows_merge(t, c->kv_dtype, s) == cudaSuccess ? MTP_OK : MTP_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t mtp_kv_workspace_size(const mtp_kv_cache* c, int B, int M, int n_q_heads) {
    if (check_cache(c, false) != MTP_OK || B < 1 || B > MTP_MAX_PAGED_BATCH || M < 1 || M > MTP_MAX_APPEND_ROWS) return 0;
    int rc;
    if (!heads_ok(c, n_q_heads, &rc)) return 0;
    int sms = num_sms();
    if (sms <= 0) sms = 152;   // no device (a host-side size query)
    if (M > MTP_MAX_ATTN_ROWS) M = MTP_MAX_ATTN_ROWS;
    const size_t cc = attn_plan(c, B, M, n_q_heads, false, sms).end, tc = attn_plan(c, B, M, n_q_heads, true, sms).end;
    return cc > tc ? cc : tc;
}

int mtp_kv_append(const mtp_kv_cache* c, int B, int M, const int32_t* kv_len, const int32_t* n_new, const void* k,
                  const void* v, int in_dtype, int64_t in_stride_b, int64_t in_stride_m, int64_t in_stride_h,
                  const float* k_norm, float rms_eps, void* ws, size_t ws_bytes, mtp_stream_t stream) {
    int rc = check_cache(c, true);
    if (rc != MTP_OK) return rc;
    if (B < 1 || B > MTP_MAX_PAGED_BATCH || M < 1 || M > MTP_MAX_APPEND_ROWS) return MTP_ERR_ARG;
    if (in_dtype != MTP_DTYPE_F32 && in_dtype != MTP_DTYPE_BF16) return MTP_ERR_UNSUPPORTED;
    if (!kv_len || misaligned(kv_len, 4) || misaligned(n_new, 4) || misaligned(k_norm, 4)) return MTP_ERR_ARG;
    if (!(rms_eps >= 0.f)) return MTP_ERR_ARG;
    for (const void* p : {k, v})
        if ((rc = check_rows(p, in_dtype, in_stride_b, in_stride_m, in_stride_h)) != MTP_OK) return rc;
    if (!ws || misaligned(ws, 256) || ws_bytes < sizeof(WsHeader)) return MTP_ERR_WORKSPACE;
    const int sms = num_sms();
    if (sms <= 0) return MTP_ERR_CUDA;
    AppendArgs a;
    a.c = device_cache(c);
    a.hd = c->head_dim; a.B = B; a.M = M;
    a.kv_len = kv_len; a.n_new = n_new;
    a.k = k; a.v = v;
    a.sb = in_stride_b; a.sm = in_stride_m; a.sh = in_stride_h;
    a.k_norm = k_norm; a.eps = rms_eps;
    a.hdr = static_cast<WsHeader*>(ws);
    a.hpt = 1;
    fill_rope(&a.rope, c->rope_theta, c->head_dim);
    return launch_kv_append(a, in_dtype, c->kv_dtype, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MTP_OK
                                                                                                                   : MTP_ERR_CUDA;
}

int mtp_paged_attention(const mtp_kv_cache* c, int B, int M, int n_q_heads, const int32_t* kv_len, const int32_t* n_new,
                        const void* q, int dtype, int64_t q_stride_b, int64_t q_stride_m, int64_t q_stride_h,
                        const float* q_norm, float rms_eps, float attn_scale, void* out, void* ws, size_t ws_bytes,
                        mtp_stream_t stream) {
    int rc = check_cache(c, true);
    if (rc != MTP_OK) return rc;
    if (B < 1 || B > MTP_MAX_PAGED_BATCH || M < 1 || M > MTP_MAX_ATTN_ROWS) return MTP_ERR_ARG;
    if (!heads_ok(c, n_q_heads, &rc)) return rc;
    if (dtype != MTP_DTYPE_F32 && dtype != MTP_DTYPE_BF16) return MTP_ERR_UNSUPPORTED;
    if (!kv_len || misaligned(kv_len, 4) || misaligned(n_new, 4) || misaligned(q_norm, 4)) return MTP_ERR_ARG;
    if (!(rms_eps >= 0.f) || !(attn_scale >= 0.f) || isinf(attn_scale)) return MTP_ERR_ARG;
    if ((rc = check_rows(q, dtype, q_stride_b, q_stride_m, q_stride_h)) != MTP_OK) return rc;
    if (!out || misaligned(out, 16)) return MTP_ERR_ARG;
    const int sms = num_sms();
    if (sms <= 0) return MTP_ERR_CUDA;
    const AttnPlan p = attn_plan(c, B, M, n_q_heads, tc_path(c, dtype), sms);
    if (!ws || misaligned(ws, 256) || ws_bytes < p.end) return MTP_ERR_WORKSPACE;
    char* base = static_cast<char*>(ws);
    PagedTcArgs t;
    PagedAttnArgs& a = t.a;
    a.c = device_cache(c);
    a.hd = c->head_dim; a.B = B; a.M = M; a.Hq = n_q_heads; a.G = n_q_heads / c->n_kv_heads;
    a.kv_len = kv_len; a.n_new = n_new;
    a.q = q; a.sb = q_stride_b; a.sm = q_stride_m; a.sh = q_stride_h;
    a.q_norm = q_norm; a.eps = rms_eps;
    a.scale = (float)((attn_scale > 0.f ? (double)attn_scale : 1.0 / sqrt((double)c->head_dim)) * 1.4426950408889634074);
    a.out = out;
    a.hdr = static_cast<WsHeader*>(ws);
    a.cta_status = reinterpret_cast<int*>(base + p.status);
    a.split = reinterpret_cast<int4*>(base + p.split);
    a.part = reinterpret_cast<float*>(base + p.part);
    a.RT = p.RT; a.rt_log2 = 0;
    while ((1 << a.rt_log2) < p.RT) ++a.rt_log2;
    const long long items = (long long)B * c->n_kv_heads * ((M * a.G + p.RT - 1) / p.RT);
    a.by_item = items <= p.grid;   // one merge CTA per row of an item, instead of per row of every CTA's
    a.rows_max = M * a.G < p.RT ? M * a.G : p.RT;
    a.tile_log2 = p.tile_log2; a.grid = p.grid; a.open_max = p.tc ? kTcOpen : 0;
    a.timeout_ns = kWaitLimitNs;
    fill_rope(&a.rope, c->rope_theta, c->head_dim);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (p.tc) {
        const bool e4m3 = c->kv_dtype == MTP_DTYPE_E4M3;
        t.slots = tc_slots(e4m3, c->head_dim, p.RT, B);
        if (t.slots < (c->head_dim + 127) / 128) return MTP_ERR_UNSUPPORTED;   // a value tile must fit the ring
        if (!encode_pages(&t.tk, c->k, c) || !encode_pages(&t.tv, c->v, c)) return MTP_ERR_UNSUPPORTED;   // a stride beyond 2^40 bytes
        e = e4m3 ? launch_paged_attn_tc_e4m3(t, s) : launch_paged_attn_tc_bf16(t, s);
    } else {
        e = launch_paged_attn_cc(a, dtype, c->kv_dtype, s);
    }
    if (e != cudaSuccess) return MTP_ERR_CUDA;
    return launch_paged_merge(a, dtype, s) == cudaSuccess ? MTP_OK : MTP_ERR_CUDA;
}

size_t mtp_prompt_workspace_size(const mtp_kv_cache* c, int B, int64_t T, int n_q_heads) {
    int rc;
    if (check_cache(c, false) != MTP_OK || B < 1 || B > MTP_MAX_PAGED_BATCH || T < 1 || T > MTP_MAX_PROMPT_ROWS) return 0;
    if (!heads_ok(c, n_q_heads, &rc) || T * n_q_heads >= 1ll << 31) return 0;
    return rows_workspace(c, B, 0, T, n_q_heads);
}

size_t mtp_prefix_workspace_size(const mtp_kv_cache* c, int B, int M, int n_q_heads) {
    int rc;
    if (check_cache(c, false) != MTP_OK || B < 1 || B > MTP_MAX_PAGED_BATCH || M < 1 || M > MTP_MAX_ATTN_ROWS) return 0;
    if (!heads_ok(c, n_q_heads, &rc) || !prefix_fits(c, B, M, n_q_heads)) return 0;
    return rows_workspace(c, B, M, (int64_t)B * M, n_q_heads);
}

int mtp_prompt_attention(const mtp_kv_cache* c, int B, int64_t T, int n_q_heads, const int32_t* kv_len, const int32_t* row_start,
                         const void* q, int dtype, int64_t q_stride_m, int64_t q_stride_h, const float* q_norm, float rms_eps,
                         float attn_scale, void* out, void* ws, size_t ws_bytes, mtp_stream_t stream) {
    const int rc = rows_call(c, B, n_q_heads, kv_len, q, dtype, 0, q_stride_m, q_stride_h, q_norm, rms_eps, attn_scale, out);
    if (rc != MTP_OK) return rc;
    if (T < 1 || T > MTP_MAX_PROMPT_ROWS || !row_start || misaligned(row_start, 4)) return MTP_ERR_ARG;
    if (T * n_q_heads >= 1ll << 31) return MTP_ERR_UNSUPPORTED;
    if (!ws || misaligned(ws, 256) || ws_bytes < rows_workspace(c, B, 0, T, n_q_heads)) return MTP_ERR_WORKSPACE;
    const int sms = num_sms();
    if (sms <= 0) return MTP_ERR_CUDA;
    RowsArgs a = rows_args(c, B, n_q_heads, kv_len, q, 0, q_stride_m, q_stride_h, q_norm, rms_eps, attn_scale, out, ws);
    a.T = (int)T;
    a.row_start = row_start;
    return launch_rows(c, a, dtype, T, ws, sms, reinterpret_cast<cudaStream_t>(stream));
}

int mtp_prefix_attention(const mtp_kv_cache* c, int B, int M, int n_q_heads, const int32_t* kv_len, const int32_t* n_new, int n_groups,
                         const int32_t* group_start, const int32_t* prefix_len, const void* q, int dtype, int64_t q_stride_b,
                         int64_t q_stride_m, int64_t q_stride_h, const float* q_norm, float rms_eps, float attn_scale, void* out,
                         void* ws, size_t ws_bytes, mtp_stream_t stream) {
    const int rc = rows_call(c, B, n_q_heads, kv_len, q, dtype, q_stride_b, q_stride_m, q_stride_h, q_norm, rms_eps, attn_scale, out);
    if (rc != MTP_OK) return rc;
    if (M < 1 || M > MTP_MAX_ATTN_ROWS || misaligned(n_new, 4) || n_groups < 0 || n_groups > B) return MTP_ERR_ARG;
    if (n_groups > 0 && (!group_start || !prefix_len || misaligned(group_start, 4) || misaligned(prefix_len, 4))) return MTP_ERR_ARG;
    if (c->window > 0 || !prefix_fits(c, B, M, n_q_heads)) return MTP_ERR_UNSUPPORTED;
    if (!ws || misaligned(ws, 256) || ws_bytes < rows_workspace(c, B, M, (int64_t)B * M, n_q_heads)) return MTP_ERR_WORKSPACE;
    const int sms = num_sms();
    if (sms <= 0) return MTP_ERR_CUDA;
    RowsArgs a = rows_args(c, B, n_q_heads, kv_len, q, q_stride_b, q_stride_m, q_stride_h, q_norm, rms_eps, attn_scale, out, ws);
    a.M = M;
    a.n_new = n_new;
    a.n_groups = n_groups; a.group_start = group_start; a.prefix_len = prefix_len;
    return launch_rows(c, a, dtype, (int64_t)B * M, ws, sms, reinterpret_cast<cudaStream_t>(stream));
}

int mtp_rotate_axes(int64_t rows, int n_axes, const int32_t* positions, const int32_t* sections, int interleaved, float theta,
                    int head_dim, int dtype, const void* q, int n_q_heads, int64_t q_stride_m, int64_t q_stride_h, const void* k,
                    int n_k_heads, int64_t k_stride_m, int64_t k_stride_h, const float* q_norm, const float* k_norm, float rms_eps,
                    void* out_q, int64_t out_q_stride_m, int64_t out_q_stride_h, void* out_k, int64_t out_k_stride_m,
                    int64_t out_k_stride_h, mtp_stream_t stream) {
    if (rows < 1 || rows > MTP_MAX_PROMPT_ROWS || n_axes < 1 || n_axes > MTP_MAX_AXES || !sections) return MTP_ERR_ARG;
    const int hd = head_dim;
    if (hd != 32 && hd != 64 && hd != 128 && hd != 256 && hd != 512) return MTP_ERR_UNSUPPORTED;
    if (dtype != MTP_DTYPE_F32 && dtype != MTP_DTYPE_BF16) return MTP_ERR_UNSUPPORTED;
    if (!positions || misaligned(positions, 4) || misaligned(q_norm, 4) || misaligned(k_norm, 4)) return MTP_ERR_ARG;
    if (!(theta > 0.f) || isinf(theta) || !(rms_eps >= 0.f)) return MTP_ERR_ARG;
    int64_t pairs = 0;
    for (int i = 0; i < n_axes; ++i) {
        if (sections[i] < 0) return MTP_ERR_ARG;
        pairs += sections[i];
    }
    if (pairs < 1 || 2 * pairs > hd) return MTP_ERR_ARG;
    if (pairs % 8) return MTP_ERR_UNSUPPORTED;
    if (n_q_heads < 1 || n_q_heads > 16384 || (k && (n_k_heads < 1 || n_k_heads > 16384))) return MTP_ERR_ARG;
    int rc;
    if ((rc = check_rows(q, dtype, 0, q_stride_m, q_stride_h)) != MTP_OK) return rc;
    if ((rc = check_rows(out_q, dtype, 0, out_q_stride_m, out_q_stride_h)) != MTP_OK) return rc;
    if (k && ((rc = check_rows(k, dtype, 0, k_stride_m, k_stride_h)) != MTP_OK ||
              (rc = check_rows(out_k, dtype, 0, out_k_stride_m, out_k_stride_h)) != MTP_OK))
        return rc;
    if (rows * (n_q_heads + (k ? n_k_heads : 0)) >= 1ll << 31) return MTP_ERR_UNSUPPORTED;
    const int sms = num_sms();
    if (sms <= 0) return MTP_ERR_CUDA;
    RotateArgs a;
    a.in[0] = q; a.in[1] = k; a.out[0] = out_q; a.out[1] = out_k;
    a.in_sm[0] = q_stride_m; a.in_sh[0] = q_stride_h; a.in_sm[1] = k_stride_m; a.in_sh[1] = k_stride_h;
    a.out_sm[0] = out_q_stride_m; a.out_sh[0] = out_q_stride_h; a.out_sm[1] = out_k_stride_m; a.out_sh[1] = out_k_stride_h;
    a.norm[0] = q_norm; a.norm[1] = k_norm;
    a.heads[0] = n_q_heads; a.heads[1] = k ? n_k_heads : 0;
    a.pos = positions;
    a.axes = n_axes; a.rows = (int)rows; a.hd = hd; a.pairs = (int)pairs;
    a.eps = rms_eps;
    fill_rope(&a.rope, theta, 2 * (int)pairs);
    for (int i = 0, at = 0, end = sections[0]; i < (int)pairs; ++i) {
        while (i >= end) end += sections[++at];
        const int turn = i % n_axes;
        a.axis[i] = (uint8_t)(interleaved ? (i < (int64_t)n_axes * sections[turn] ? turn : 0) : at);
    }
    return launch_rotate_axes(a, dtype, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MTP_OK : MTP_ERR_CUDA;
}

int mtp_token_logprobs(const void* logits, int ldtype, int64_t rows, int V, int64_t row_stride, const int32_t* tokens,
                       int top_k, float* out_logprob, float* out_entropy, int32_t* out_top_ids, float* out_top_logprobs,
                       mtp_stream_t stream) {
    if (!logits) return MTP_ERR_ARG;
    if (ldtype != MTP_DTYPE_F32 && ldtype != MTP_DTYPE_BF16) return MTP_ERR_UNSUPPORTED;
    if (misaligned(logits, ldtype == MTP_DTYPE_BF16 ? 2 : 4)) return MTP_ERR_ARG;
    if (rows < 1 || rows > 17ll * MTP_MAX_VERIFY_BATCH || V < 1 || row_stride < V) return MTP_ERR_ARG;
    if (top_k < 0 || top_k > MTP_MAX_TOP) return MTP_ERR_ARG;
    for (const void* p : {(const void*)tokens, (const void*)out_logprob, (const void*)out_entropy, (const void*)out_top_ids,
                          (const void*)out_top_logprobs})
        if (misaligned(p, 4)) return MTP_ERR_ARG;
    const int sms = num_sms();
    if (sms <= 0) return MTP_ERR_CUDA;
    LogprobArgs a;
    a.logits = logits; a.rows = rows; a.V = V; a.stride = row_stride;
    a.tokens = tokens; a.K = out_top_ids || out_top_logprobs ? top_k : 0;
    a.logprob = tokens ? out_logprob : nullptr; a.entropy = out_entropy;
    a.top_ids = out_top_ids; a.top_logprobs = out_top_logprobs;
    a.timeout_ns = kWaitLimitNs;
    return launch_logprobs(a, ldtype, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MTP_OK : MTP_ERR_CUDA;
}

}  // extern "C"
