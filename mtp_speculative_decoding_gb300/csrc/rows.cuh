// rows.cuh -- argument block and row helpers of the attention of many rows over
// the paged cache: whole prompts, and batches that share prefixes (internal).
#pragma once

#include "paged.cuh"

namespace mtp {

struct RowsArgs {
    PagedKV c;
    int hd, B, Hq, G;
    int M;                          // shared prefixes: rows of a sequence at most; prompts: 0
    int T;                          // prompts: packed rows
    int n_groups;                   // shared prefixes
    const int32_t *kv_len, *n_new;  // n_new: shared prefixes only (null: all M)
    const int32_t* row_start;       // prompts: [B + 1]
    const int32_t *group_start, *prefix_len;   // [n_groups + 1], [n_groups]
    const void* q;
    long long sb, sm, sh;           // (prompts: sb 0)
    const float* q_norm;
    float eps, scale;               // scale: attn_scale * log2(e) (scores are in bits)
    void* out;
    WsHeader* hdr;
    RopeTab rope;
};

// A sequence of the call: its rows are tokens [0, n), token j at position len +
// j; positions below P lie on the pages of sequence `first`.
struct Seq {
    int len, n, P, first, group;    // group: -1 without a shared prefix
    long long q0;                   // element of its first row in q
    long long row0;                 // its first token's place in out (in tokens)
};
// the last i in [0, n) with start[i] <= x, 0 if there is none
__device__ __forceinline__ int last_at_most(const int32_t* start, int n, int x) {
    int lo = 0;
    for (int hi = n - 1; lo < hi;) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}
// Prompts: sequence b's rows are its alone.  No bound in front of them lies behind their
// start, none behind them in front of their end; the last bound that is not above one of
// its rows is then its own.  Of bounds that ascend that holds for every sequence.
__device__ __forceinline__ bool bound_agrees(const int32_t* row_start, int b, int i) {
    return i <= b ? row_start[i] <= row_start[b] : row_start[i] >= row_start[b + 1];
}
// false: its lengths, rows or group are out of range (s.n is 0 then).  starts,
// lengths: copies of group_start and prefix_len.  (Whether bound_agrees is the caller's
// to find out.)
__device__ __forceinline__ bool seq_at(const RowsArgs& a, int b, Seq& s, const int32_t* starts, const int32_t* lengths) {
    s.len = a.kv_len[b];
    s.P = 0;
    s.first = b;
    s.group = -1;
    bool ok = true;
    if (a.M > 0) {
        s.n = a.n_new ? a.n_new[b] : a.M;
        s.row0 = (long long)b * a.M;
        s.q0 = b * a.sb;
        ok = s.n >= 0 && s.n <= a.M;
        if (a.n_groups > 0) {
            const int i = last_at_most(starts, a.n_groups, b), g0 = starts[i], g1 = starts[i + 1];
            if (g0 >= 0 && g0 <= b && b < g1 && g1 <= a.B) {
                s.P = lengths[i];
                s.first = g0;
                s.group = i;
                ok = ok && s.P >= 0 && s.P <= s.len;
            } else {
                // outside every group where the bounds ascend: before the first or behind the last
                ok = ok && (b < starts[0] || (i == a.n_groups - 1 && g0 <= g1 && b >= g1));
            }
        }
    } else {
        const int r0 = a.row_start[b], r1 = a.row_start[b + 1];
        ok = r0 >= 0 && r0 <= r1 && r1 <= a.T;
        s.n = r1 - r0;
        s.row0 = r0;
        s.q0 = r0 * a.sm;
    }
    ok = ok && s.len >= 0 && (long long)s.len + s.n <= (long long)a.c.max_pages << a.c.ps_log2;
    if (!ok) s.n = 0;
    return ok;
}

__device__ __forceinline__ bool seq_at(const RowsArgs& a, int b, Seq& s) { return seq_at(a, b, s, a.group_start, a.prefix_len); }

cudaError_t launch_rows_cc(const RowsArgs& a, int dtype, int kv_dtype, cudaStream_t s);

// ---------------------------------------------------------------------------
// rotation by several positions
// ---------------------------------------------------------------------------
struct RotateArgs {
    const void* in[2];              // query rows, key rows (null: none)
    void* out[2];
    long long in_sm[2], in_sh[2], out_sm[2], out_sh[2];   // strides of row and head (elements)
    const float* norm[2];
    int heads[2];
    const int32_t* pos;             // [axes, rows]
    int axes, rows, hd, pairs;
    float eps;
    int hpt, groups[2];             // heads a thread; thread groups of the queries and of the keys
    RopeTab rope;
    uint8_t axis[256];              // a pair's axis
};
cudaError_t launch_rotate_axes(RotateArgs a, int dtype, int sms, cudaStream_t s);

}  // namespace mtp
