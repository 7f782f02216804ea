// rows_attn_tc.cuh -- attention of many rows on the tensor cores: the plan of a
// call, shared by the attention and by the merge of what it left in parts
// (internal).
#pragma once

#include <cuda.h>

#include "rows.cuh"

namespace mtp {

constexpr int kRowTile = 256;         // rows of an item
constexpr int kPosTile = 128;         // positions of a tile
// What beginning an item costs, in tiles (queries, an epilogue, and a pipeline
// that fills anew).
constexpr int kRowsOpen = 2;

// A block is a sequence's rows against its own positions, or, in front of the
// sequences, a group's rows against the group's prefix.  An item is (block, KV
// head, row tile): kRowTile of the block's n * G rows (row r: token r / G, query
// head r % G of the group) against the tiles that any of them attends.
//
// Items lie end to end on a line, block by block, KV head by KV head.  A tile
// takes U = kPosTile * G units of it, so that the tiles of a causal row tile grow
// by kRowTile units from one to the next and everything before an item is a
// closed form: row tile i of a sequence has at most
//   (kRowTile i + len G + kRowTile - 1) / U + 1 - (first / kPosTile)
// tiles (rounded down), which its kRowTile i + C units cover, with half a tile more on
// average for what the rounding takes; under a window a constant bounds it.  Worker
// w (a CTA, or a pair) takes the tiles that begin in its share of the line, so ragged
// lengths and causal triangles cost every worker the same.  A share holds U units
// at least: every worker between an item's first and last one has a tile of it.
struct RowsPlan {
    int open, workers;                // units before an item's tiles / U; workers with a share
    const long long* pre;             // [blocks + 1] units before a block
    const int* cum;                   // shared prefixes: [B + 1] tokens before a sequence
};
struct RowsTcArgs {
    RowsArgs a;
    int workers;                      // of the launch
    long long window_units;           // most units of a row tile under a window
    int* cta_status;                  // [CTAs]
    int4* note;                       // prompts, [workers]: the item that begins in a worker's share and ends behind it
    int2* plan_head;                  // open, workers of the plan; then its arrays
    long long* plan_pre;
    int* plan_cum;
    float* part;                      // [2 workers][kRowTile][hd] and, behind them, their (m, l)
    float2* part_ml;
    uint8_t* odd;                     // prompts, [T * Hq]: the row's result is not finite
    float* dense;                     // shared prefixes, [2][B * M * Hq][hd]: a row's prefix and own part, where one worker had it whole
    float2* dense_ml;
    unsigned long long timeout_ns;
};
struct RowsTcParams {
    CUtensorMap tk, tv;               // (dimension, slot, KV head, page)
    RowsTcArgs t;
};

__host__ __device__ __forceinline__ int rows_blocks(const RowsArgs& a) { return a.n_groups + a.B; }

struct Block {
    int b0, b1;                       // its sequences; table row b0
    int n, len;                       // tokens; position of token 0 (sequences)
    int lo, hi;                       // positions [lo, hi) of it at most
    int group;                        // 1: a group's prefix
    int valid;                        // 0: out of range
    long long q0, row0;               // a sequence's (see Seq)
};
__device__ __forceinline__ Block block_at(const RowsArgs& a, const int* cum, int blk) {
    Block k = {};
    k.valid = 1;
    if (blk < a.n_groups) {
        const int g0 = a.group_start[blk], g1 = a.group_start[blk + 1], P = a.prefix_len[blk];
        k.group = 1;
        k.valid = g0 >= 0 && g0 <= g1 && g1 <= a.B && P >= 0 && P <= (long long)a.c.max_pages << a.c.ps_log2;
        if (k.valid) {
            k.b0 = g0;
            k.b1 = g1;
            k.hi = P;
            k.n = P > 0 ? cum[g1] - cum[g0] : 0;
        }
        return k;
    }
    Seq s;
    const int b = blk - a.n_groups;
    k.valid = seq_at(a, b, s);
    k.b0 = b;
    k.b1 = b + 1;
    k.n = s.n;
    k.len = s.len;
    k.lo = s.n > 0 ? s.P : 0;
    k.hi = s.n > 0 ? s.len + s.n : 0;
    k.q0 = s.q0;
    k.row0 = s.row0;
    return k;
}
__device__ __forceinline__ int row_tiles_of(const RowsArgs& a, const Block& k) { return (k.n * a.G + kRowTile - 1) / kRowTile; }
// units of the tiles of the row tiles before i (without what opening them costs)
__device__ __forceinline__ long long tile_units(const RowsTcArgs& t, const Block& k, long long i) {
    const RowsArgs& a = t.a;
    const long long U = (long long)kPosTile * a.G;
    if (k.group) return i * ((k.hi + kPosTile - 1) / kPosTile) * U;
    const long long C = (long long)k.len * a.G + kRowTile - (k.lo / kPosTile) * U + U / 2;
    long long grow = i;               // row tiles that the window does not bound
    if (a.c.window > 0) {
        const long long room = t.window_units - C;
        const long long most = room <= 0 ? 0 : (room + kRowTile - 1) / kRowTile;
        grow = most < i ? most : i;
    }
    return kRowTile * (grow * (grow - 1) / 2) + C * grow + (i - grow) * t.window_units;
}
__device__ __forceinline__ long long units_before(const RowsTcArgs& t, const Block& k, int open, long long i) {
    return tile_units(t, k, i) + i * open * (long long)kPosTile * t.a.G;
}
// worker w's share of T units begins at share_at(T, w); the worker that has unit x
__device__ __forceinline__ long long share_at(long long T, int workers, int w) {
    const long long base = T / workers, rem = T - base * workers;
    return base * w + (w < rem ? w : rem);
}
__device__ __forceinline__ int worker_of(long long T, int workers, long long x) {
    const long long base = T / workers, rem = T - base * workers;
    return (int)(x < rem * (base + 1) ? x / (base + 1) : rem + (x - rem * (base + 1)) / base);
}

// Where an item's tiles lie.
struct Item {
    long long begin, tiles_at, end;   // its units: [begin, end), the tiles' from tiles_at
    int st, lt, n;                    // tiles [0, st) (the sink) and [lt, lt + n - st)
    int r0, rows;                     // its rows [r0, r0 + rows) of the block
    int p_first, p_last;              // positions of its first and last row (a group: behind the prefix)
};
__device__ __forceinline__ Item item_of(const RowsTcArgs& t, const RowsPlan& plan, const Block& k, int blk, int g, int rt) {
    const RowsArgs& a = t.a;
    const long long U = (long long)kPosTile * a.G;
    const long long before = units_before(t, k, plan.open, rt), head = units_before(t, k, plan.open, row_tiles_of(a, k));
    Item it;
    it.begin = plan.pre[blk] + g * head + before;
    it.tiles_at = it.begin + plan.open * U;
    it.end = plan.pre[blk] + g * head + units_before(t, k, plan.open, rt + 1);
    it.r0 = rt * kRowTile;
    const int left = k.n * a.G - it.r0;
    it.rows = left < kRowTile ? left : kRowTile;
    it.st = 0;
    if (k.group) {
        it.p_first = it.p_last = k.hi;
        it.lt = 0;
        it.n = (k.hi + kPosTile - 1) / kPosTile;
        return it;
    }
    it.p_first = k.len + it.r0 / a.G;
    it.p_last = k.len + (it.r0 + it.rows - 1) / a.G;
    int lo = k.lo;
    if (a.c.window > 0) {
        const int w = it.p_first + 1 > a.c.window ? it.p_first + 1 - a.c.window : 0;
        if (w > lo) lo = w;
        const int far = it.p_last + 1 > a.c.window ? it.p_last + 1 - a.c.window : 0;
        const int sink = a.c.sink < far ? a.c.sink : far;
        it.st = (sink + kPosTile - 1) / kPosTile;
    }
    it.lt = lo / kPosTile;
    if (it.st > it.lt) it.st = it.lt;
    it.n = it.st + it.p_last / kPosTile + 1 - it.lt;
    return it;
}

// A worker's part of an item.
struct Piece {
    Block k;
    Item it;
    int blk, g, rt;
    int t0, n;                        // tiles [t0, t0 + n) of the item
    int slot;                         // 0: the whole item; 1: it began before; 2: it ends behind
    long long next;                   // where the item behind it begins
};
// The piece at unit x of a share that ends at xe; n <= 0 where no tile of the item
// begins in the share.
__device__ __forceinline__ Piece piece_at(const RowsTcArgs& t, const RowsPlan& plan, long long x, long long xs, long long xe) {
    const RowsArgs& a = t.a;
    Piece p;
    int b = 0;
    for (int hi = rows_blocks(a) - 1; b < hi;) {   // the last block that begins at x or before
        const int mid = (b + hi + 1) >> 1;
        if (plan.pre[mid] <= x) b = mid;
        else hi = mid - 1;
    }
    p.blk = b;
    p.k = block_at(a, plan.cum, b);
    const int nrt = row_tiles_of(a, p.k);
    const long long head = units_before(t, p.k, plan.open, nrt);
    long long rel = x - plan.pre[b];
    p.g = head > 0 ? (int)(rel / head) : 0;
    rel -= p.g * head;
    int rt = 0;
    for (int hi = nrt - 1; rt < hi;) {
        const int mid = (rt + hi + 1) >> 1;
        if (units_before(t, p.k, plan.open, mid) <= rel) rt = mid;
        else hi = mid - 1;
    }
    p.rt = rt;
    p.it = item_of(t, plan, p.k, b, p.g, rt);
    const long long U = (long long)kPosTile * a.G;
    // tiles that begin in [xs, xe)
    const long long from = xs - p.it.tiles_at, to = xe - p.it.tiles_at;
    const long long t0 = from <= 0 ? 0 : (from + U - 1) / U, t1 = to <= 0 ? 0 : (to + U - 1) / U;
    p.t0 = (int)(t0 < p.it.n ? t0 : p.it.n);
    p.n = (int)(t1 < p.it.n ? t1 : p.it.n) - p.t0;
    p.slot = p.t0 > 0 ? 1 : p.n < p.it.n ? 2 : 0;
    p.next = p.it.end;
    return p;
}
__device__ __forceinline__ int tile_of(const Item& it, int k) { return k < it.st ? k : it.lt + (k - it.st); }

// Bytes of the plan in shared memory.
__host__ __device__ constexpr int rows_plan_bytes(int B, int n_groups) { return (B + n_groups + 1) * 8 + (B + 2) * 4 + 2 * 32 * 8; }

// Fills the plan (shared memory: pre, cum, 64 words of scratch); the whole CTA,
// THREADS threads.  False for this thread if it saw something out of range.
template <int THREADS>
__device__ __forceinline__ bool make_plan(const RowsTcArgs& t, RowsPlan& plan, long long* pre, int* cum, long long* tmp) {
    static_assert(THREADS % 32 == 0 && THREADS <= 1024, "scratch");
    const RowsArgs& a = t.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    bool good = true;
    // sums over the threads in front of this one, and over all
    auto scan = [&](long long v, long long* s, long long& total) {
        long long inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += u;
        }
        __syncthreads();
        if (lane == 31) s[warp] = inc;
        __syncthreads();
        long long base = inc - v;
        total = 0;
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) base += s[w];
            total += s[w];
        }
        return base;
    };
    long long all;
    if (a.n_groups > 0) {   // tokens before every sequence
        const int per = (a.B + THREADS - 1) / THREADS, b0 = tid * per, b1 = b0 + per < a.B ? b0 + per : a.B;
        int sum = 0;
        for (int b = b0; b < b1; ++b) {
            Seq s;
            seq_at(a, b, s);
            sum += s.n;
        }
        int at = (int)scan(sum, tmp, all);
        for (int b = b0; b < b1; ++b) {
            Seq s;
            seq_at(a, b, s);
            cum[b] = at;
            at += s.n;
        }
        if (tid == 0) cum[a.B] = (int)all;
        __syncthreads();
    }
    const int nb = rows_blocks(a), per = (nb + THREADS - 1) / THREADS, k0 = tid * per, k1 = k0 + per < nb ? k0 + per : nb;
    const long long U = (long long)kPosTile * a.G;
    long long tiles = 0, items = 0;
    for (int i = k0; i < k1; ++i) {
        const Block k = block_at(a, cum, i);
        good = good && k.valid;
        const int nrt = row_tiles_of(a, k);
        tiles += a.c.Hkv * tile_units(t, k, nrt);
        items += (long long)a.c.Hkv * nrt;
    }
    long long units, n_items;
    long long at = scan(tiles, tmp, units);
    const long long it = scan(items, tmp + 32, n_items);
    // where a share is few tiles, how they spread counts for more
    plan.open = kRowsOpen;
    while (plan.open > 0 && 2ll * plan.open * U * t.workers > units) --plan.open;
    at += it * plan.open * U;
    for (int i = k0; i < k1; ++i) {
        pre[i] = at;
        const Block k = block_at(a, cum, i);
        at += a.c.Hkv * units_before(t, k, plan.open, row_tiles_of(a, k));
    }
    const long long T = units + n_items * plan.open * U;
    if (tid == 0) pre[nb] = T;
    const long long most = T / U;
    plan.workers = most < t.workers ? (most > 1 ? (int)most : 1) : t.workers;
    plan.pre = pre;
    plan.cum = cum;
    __syncthreads();
    return good;
}

// The place of row r (of a block's rows) of KV head g.
struct RowPlace {
    int b, j;                         // sequence, token
    int pos;                          // its position
    long long q;                      // element of q
    long long out;                    // row of out (in heads)
};
__device__ __forceinline__ RowPlace row_place(const RowsArgs& a, const int* cum, const Block& k, int g, int r) {
    RowPlace p;
    int tok = (int)udiv((unsigned)r, (unsigned)a.G);
    const int h = g * a.G + r - tok * a.G;
    p.b = k.b0;
    if (k.group) {
        const int x = cum[k.b0] + tok;
        p.b = k.b0 + last_at_most(cum + k.b0, k.b1 - k.b0, x);
        tok = x - cum[p.b];
        p.pos = a.kv_len[p.b] + tok;
        p.q = p.b * a.sb + tok * a.sm + h * a.sh;
        p.out = ((long long)p.b * a.M + tok) * a.Hq + h;
    } else {
        p.pos = k.len + tok;
        p.q = k.q0 + tok * a.sm + h * a.sh;
        p.out = (k.row0 + tok) * a.Hq + h;
    }
    p.j = tok;
    return p;
}

// shared memory of the attention kernel
__host__ __device__ constexpr int rows_pair(int hd) { return hd == 256 ? 2 : 1; }        // CTAs of a worker
__host__ __device__ constexpr int rows_q_bytes(int hd) { return kRowTile / rows_pair(hd) * hd * 2; }
__host__ __device__ constexpr int rows_slot_bytes(int hd) { return kPosTile * hd * 2 / rows_pair(hd); }
constexpr int kRowsMeta = 16;         // tiles whose masks and scales the producer may be ahead
constexpr int kRowsSlots = 8, kRowsRaw = 4;   // ring slots at most
constexpr int kRowsSmemLimit = 227 * 1024 - 64;
__host__ __device__ constexpr int rows_other(int hd, int B, int n_groups) {
    return 1024 + kRowsMeta * (16 + 64 + 16) + (3 * kRowsSlots + 2 * kRowsRaw + kRowsMeta + 16) * 8 + hd * 4 + 2 * kRowTile * 4 + rows_plan_bytes(B, n_groups) + 64;
}
// 8-bit caches: codes as they come in take half a slot each
__host__ __device__ constexpr int rows_raw(bool e4m3, int hd) { return e4m3 ? (hd == 64 ? 4 : 3) : 0; }
__host__ __device__ constexpr int rows_slots(bool e4m3, int hd, int B, int n_groups) {
    int n = (kRowsSmemLimit - rows_other(hd, B, n_groups) - rows_q_bytes(hd) - rows_raw(e4m3, hd) * rows_slot_bytes(hd) / 2) / rows_slot_bytes(hd);
    return n < kRowsSlots ? n : kRowsSlots;
}

// one translation unit each (rows_attn_tc.cu)
cudaError_t launch_rows_tc_bf16(const RowsTcParams& p, cudaStream_t s);
cudaError_t launch_rows_tc_e4m3(const RowsTcParams& p, cudaStream_t s);
cudaError_t launch_rows_merge(const RowsTcArgs& t, int kv_dtype, cudaStream_t s);

}  // namespace mtp
