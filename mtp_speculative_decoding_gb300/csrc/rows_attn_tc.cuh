// rows_attn_tc.cuh -- attention of many rows on the tensor cores: the plan of a
// call, shared by the kernel that makes it, the attention, and the merge of what
// that left in parts (internal).
#pragma once

#include <cuda.h>

#include "rows.cuh"

namespace mtp {

constexpr int kRowTile = 256;         // rows of an item
constexpr int kPosTile = 128;         // positions of a tile
// What beginning an item costs, in tiles (an epilogue, and a pipeline that fills
// anew).  Measured with 0, 1, 2, 3, 4, 6: 13 packed prompts of up to 2048 tokens take 186,
// 175, 175, 181, 181, 190 us, one of 8192 at head dimension 256 396, 373, 366, 369, 373,
// 379.
constexpr int kRowsOpen = 2;

// A block is rows and positions: a sequence's rows against its positions (prompts,
// and sequences of no group), a group's rows against the group's prefix, or a group's
// rows against their sequences' own positions, the tiles of one sequence after those
// of the other: few rows of many sequences then share their queries' copy and the
// accumulator, and a tile's other rows have weights of zero.  (An item a sequence costs
// 5 us for one or two tiles.)  An item is (block, KV head, row tile): kRowTile of the
// block's n * G rows (row r: token r / G, query head r % G of the KV head) against the
// tiles that any of them attends.
//
// Items lie end to end on a line, block by block, KV head by KV head.  A tile
// takes U = kPosTile * G units of it, so that the tiles of a causal row tile grow
// by kRowTile units from one to the next and everything before an item is a
// closed form: row tile i of a sequence has at most
//   (kRowTile i + len G + kRowTile - 1) / U + 1 - first / kPosTile
// tiles (rounded down), which its kRowTile i + C units cover, with half a tile more on
// average for what the rounding takes; under a window a constant bounds it.  (The
// tiles of a group's own positions are counted item by item.)  Worker
// w (a CTA, or a pair) takes the tiles that begin in its share of the line, so ragged
// lengths and causal triangles cost every worker the same.  A share holds U units
// at least: every worker between an item's first and last one has a tile of it.
enum { kSequence = 0, kPrefix = 1, kOwn = 2 };
struct __align__(16) BlockRec {
    int n, len;                       // tokens; position of token 0 (sequences), end of the sequences (a group's own positions)
    int lo, hi;                       // positions [lo, hi) of it at most (a group's own positions: from lo on)
    int table;                        // row of the page table: the sequence, or the group's first
    int kind;                         // kSequence, kPrefix, kOwn
    int q_stride;                     // rows of a KV head in the staged queries
    int row0;                         // sequences: its first token in out; a group's own positions: its first entry in `items`
    long long q_row;                  // its first row there (KV head 0)
    long long pre;                    // units before the block
};
static_assert(sizeof(BlockRec) == 48, "three 16-byte loads");
// where a worker's share begins: its first item, and where that begins
struct __align__(16) WorkerRec {
    long long xs, xe;                 // share of the line
    long long begin;                  // the item's first unit
    int blk, g, rt;
    int open;                         // units before an item's tiles / U
    BlockRec k;                       // the item's block
};
// an item that begins in a worker's share and ends behind it
struct __align__(16) RowNote {
    int last;                         // worker with its last tile (-1: there is no such item)
    int rows, r0, g;                  // rows [r0, r0 + rows) of the block, KV head
    int row0;                         // the sequence's first token in out
    int pad_[3];
};
// a part of a row's result with shared prefixes: in `dense`, or in slots of workers
struct __align__(16) RowPart {
    static constexpr uint32_t kSlots = ~0u;
    uint32_t dense;                   // the row's place in `dense`
    uint16_t w0, w1;                  // first and last worker that has a tile of it
    uint16_t first;                   // worker in whose share its item begins
    uint16_t r;                       // row of the slots
    int there;                        // 0: no such part
};
static_assert(sizeof(RowPart) == 16, "one load");
struct PlanHead {
    long long T;                      // units in all
    int open, workers;                // units before an item's tiles / U; workers with a share
};

// Rows are staged as operands first (rows_prepare.cu): normed, rotated and rounded
// once, the rows of a group (or of a sequence of no group) KV head by KV head, a
// KV head's rows token by token, so that the rows of an item lie one after another.
struct RowsTcArgs {
    RowsArgs a;
    int workers;                      // of the launch
    long long window_units;           // most units of a row tile under a window
    PlanHead* head;
    BlockRec* blocks;                 // [2 n_groups + B]
    WorkerRec* worker;                // [workers]
    long long* items;                 // tiles of the groups' own items before each of them (a sequence's tiles count once an
                                      // item that its rows reach into: more than 31 bits)
    int *cum, *cumt, *lens;           // shared prefixes: tokens and own tiles before a sequence [B + 1], its cached positions [B]
    uint16_t* staged;                 // [rows][hd]
    float* q_scale;                   // e4m3: [rows] a staged row's power of two times the softmax scale
    int* cta_status;                  // [CTAs], and behind them the plan's
    RowNote* note;                    // prompts, [workers]
    RowPart* row_parts;               // shared prefixes, [B * M * Hq][2]: a row's own part and its prefix's
    float* part;                      // [2 workers][kRowTile][hd]
    float2* part_ml;                  // their maxima and sums
    uint8_t* odd;                     // prompts, [2][odd_plane]: the row's result is not finite, by each thread that has a share of it
    long long odd_plane;              // T * Hq, rounded up
    float* dense;                     // shared prefixes, [2][rows][hd] by staged rows: a row's prefix and own part, where one worker had it whole
    float2* dense_ml;
    unsigned long long timeout_ns;
};
struct RowsTcParams {
    CUtensorMap tk, tv, tq;           // (dimension, slot, KV head, page) of k and v; (dimension, row) of the staged queries
    RowsTcArgs t;
};

// groups' prefixes, groups' own positions, sequences (of a group: nothing)
__host__ __device__ __forceinline__ int rows_blocks(const RowsArgs& a) { return 2 * a.n_groups + a.B; }
__device__ __forceinline__ int row_tiles_of(const RowsArgs& a, const BlockRec& k) { return (k.n * a.G + kRowTile - 1) / kRowTile; }
// units of row tile i's tiles: kRowTile i + C, bounded under a window; all alike for a prefix
__device__ __forceinline__ long long grow_units(const RowsTcArgs& t, const BlockRec& k) {
    const long long U = (long long)kPosTile * t.a.G;
    return (long long)k.len * t.a.G + kRowTile - (k.lo / kPosTile) * U + U / 2;
}
__device__ __forceinline__ long long item_units(const RowsTcArgs& t, const BlockRec& k, int i) {
    if (k.kind == kPrefix) return (k.hi + kPosTile - 1) / kPosTile * (long long)(kPosTile * t.a.G);
    const long long u = (long long)kRowTile * i + grow_units(t, k);
    return t.a.c.window > 0 && u > t.window_units ? t.window_units : u;
}
// units of the row tiles before i (without what opening them costs)
__device__ __forceinline__ long long tile_units(const RowsTcArgs& t, const BlockRec& k, long long i) {
    if (k.kind == kPrefix) return i * item_units(t, k, 0);
    if (k.kind == kOwn) return (t.items[k.row0 + i] - t.items[k.row0]) * (kPosTile * t.a.G);
    const long long C = grow_units(t, k);
    long long grow = i;               // row tiles that the window does not bound
    if (t.a.c.window > 0) {
        const long long room = t.window_units - C;
        const long long most = room <= 0 ? 0 : (room + kRowTile - 1) / kRowTile;
        grow = most < i ? most : i;
    }
    return kRowTile * (grow * (grow - 1) / 2) + C * grow + (i - grow) * t.window_units;
}
__device__ __forceinline__ long long units_before(const RowsTcArgs& t, const BlockRec& k, int open, long long i) {
    return tile_units(t, k, i) + i * open * (long long)(kPosTile * t.a.G);
}
__device__ __forceinline__ long long quotient(long long a, long long b) {   // a / b, neither negative
    return (unsigned long long)(a | b) >> 32 ? a / b : (long long)((unsigned)a / (unsigned)b);
}
// Shares of T units are even, the first T mod workers of them one longer: the worker that
// has unit x
__device__ __forceinline__ int worker_of(long long T, int workers, long long x) {
    const long long base = quotient(T, workers), rem = T - base * workers;
    return (int)(x < rem * (base + 1) ? quotient(x, base + 1) : rem + quotient(x - rem * (base + 1), base));
}

// The sequences of the call with shared prefixes: tokens and own tiles before each,
// cached positions (shared memory or the workspace's).
struct Sequences { const int *cum, *cumt, *lens; };

// Where an item's tiles lie.
struct Item {
    int st, lt, n;                    // tiles [0, st) (the sink) and [lt, lt + n - st); a group's own: from tile lt of all on
    int r0, rows;                     // its rows [r0, r0 + rows) of the block
    int p_first, p_last;              // positions of its first and last row (a group: behind the prefix)
};
// (SHARED false: prompts, whose blocks are sequences)
template <bool SHARED>
__device__ __forceinline__ Item item_of(const RowsArgs& a, const Sequences& sq, const BlockRec& k, int rt) {
    Item it;
    it.r0 = rt * kRowTile;
    const int left = k.n * a.G - it.r0;
    it.rows = left < kRowTile ? left : kRowTile;
    it.st = 0;
    if (SHARED && k.kind == kPrefix) {
        it.p_first = it.p_last = k.hi;
        it.lt = 0;
        it.n = (k.hi + kPosTile - 1) / kPosTile;
        return it;
    }
    const int j0 = (int)udiv((unsigned)it.r0, (unsigned)a.G), j1 = (int)udiv((unsigned)(it.r0 + it.rows - 1), (unsigned)a.G);
    if (SHARED && k.kind == kOwn) {
        const int m = k.len - k.table, x = sq.cum[k.table];
        it.p_first = it.p_last = 0;
        it.lt = sq.cumt[k.table + last_at_most(sq.cum + k.table, m, x + j0)];
        it.n = sq.cumt[k.table + last_at_most(sq.cum + k.table, m, x + j1) + 1] - it.lt;
        return it;
    }
    it.p_first = k.len + j0;
    it.p_last = k.len + j1;
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
// Tile k of an item: sequence whose pages it lies on, first position, where the
// positions that anyone attends end, and which of the item's row tiles of 128 attend it
// (bits).
struct Tile { int seq, pos, end, rows; };
template <bool SHARED>
__device__ __forceinline__ Tile tile_of(const RowsArgs& a, const Sequences& sq, const BlockRec& k, const Item& it, int i) {
    Tile t;
    if (SHARED && k.kind == kOwn) {
        const int x = it.lt + i;
        t.seq = k.table + last_at_most(sq.cumt + k.table, k.len - k.table, x);
        t.pos = (k.lo / kPosTile + x - sq.cumt[t.seq]) * kPosTile;
        const int c0 = sq.cum[t.seq], c1 = sq.cum[t.seq + 1], base = sq.cum[k.table];
        t.end = sq.lens[t.seq] + c1 - c0;
        const int ra = (c0 - base) * a.G - it.r0, rb = (c1 - base) * a.G - it.r0;
        t.rows = (ra < 128 && rb > 0 ? 1 : 0) | (rb > 128 && it.rows > 128 && ra < it.rows ? 2 : 0);
        return t;
    }
    t.seq = k.table;
    t.pos = (i < it.st ? i : it.lt + (i - it.st)) * kPosTile;
    t.end = SHARED && k.kind == kPrefix ? k.hi : it.p_last + 1;
    t.rows = it.rows > 128 ? 3 : 1;
    return t;
}

// The pieces of items that a worker takes, one after another.
template <bool SHARED>
struct Walk {
    BlockRec k;
    Item it;
    long long at, xs, xe;             // where the next item begins; the share
    long long tiles_at;               // where this item's tiles begin
    int blk, g, rt;                   // of this piece
    int nb, ng, nr;                   // of the next item
    int t0, n;                        // tiles [t0, t0 + n) of the item
    int slot;                         // 0: the whole item; 1: it began before; 2: it ends behind
    int open, held;                   // units before an item's tiles / U; block that k is
    Sequences sq;

    __device__ __forceinline__ void start(const WorkerRec& w, const Sequences& s) {
        sq = s;
        at = w.begin;
        xs = w.xs;
        xe = w.xe;
        held = nb = w.blk;
        ng = w.g;
        nr = w.rt;
        open = w.open;
        k = w.k;
    }
    __device__ __forceinline__ bool next(const RowsTcArgs& t) {
        const int U = kPosTile * t.a.G;
        while (at < xe) {
            if (held != nb) {
                k = t.blocks[nb];
                held = nb;
            }
            const int nrt = row_tiles_of(t.a, k);
            if (nr >= nrt) {          // the next KV head, or the next block
                nr = 0;
                if (nrt == 0 || ++ng >= t.a.c.Hkv) {
                    ng = 0;
                    ++nb;
                }
                continue;
            }
            blk = nb;
            g = ng;
            rt = nr++;
            it = item_of<SHARED>(t.a, sq, k, rt);
            tiles_at = at + (long long)open * U;
            at = tiles_at + (SHARED && k.kind == kOwn ? (long long)it.n * U : item_units(t, k, rt));
            const long long from = xs - tiles_at + U - 1, to = xe - tiles_at + U - 1;   // tiles that begin in [xs, xe)
            const long long f = from < U ? 0 : quotient(from, U), e = to < U ? 0 : quotient(to, U);
            t0 = (int)(f < it.n ? f : it.n);
            n = (int)(e < it.n ? e : it.n) - t0;
            slot = t0 > 0 ? 1 : n < it.n ? 2 : 0;
            if (n > 0) return true;
        }
        return false;
    }
};

// shared memory of the attention kernel
__host__ __device__ constexpr int rows_pair(int hd) { return hd == 256 ? 2 : 1; }        // CTAs of a worker
__host__ __device__ constexpr int rows_q_bytes(int hd) { return kRowTile / rows_pair(hd) * hd * 2; }
__host__ __device__ constexpr int rows_slot_bytes(int hd) { return kPosTile * hd * 2 / rows_pair(hd); }
constexpr int kRowsMeta = 16;         // tiles whose masks and scales may be there at a time
constexpr int kRowsSlots = 8, kRowsRaw = 4;   // ring slots at most
constexpr int kRowsSmemLimit = 227 * 1024 - 64;
// threads that share a row of a tile in the softmax: a pair of CTAs has one row tile each and
// registers for two (one CTA with two row tiles was slower so: 351 against 276 us for 8192
// tokens at head dimension 128)
__host__ __device__ constexpr int rows_halves(int hd) { return rows_pair(hd); }
constexpr int kRowsOther = 1024 + 2 * kRowTile * 4 + kRowsMeta * (16 + 64 + 16) + (3 * kRowsSlots + 2 * kRowsRaw + 2 * kRowsMeta + 16) * 8;
// the sequences' tables, behind the rest
__host__ __device__ constexpr int rows_tables(int B) { return (3 * B + 2) * 4; }
// 8-bit caches: codes as they come in take half a slot each
__host__ __device__ constexpr int rows_raw(bool e4m3, int hd) { return e4m3 ? (hd == 64 ? 4 : 3) : 0; }
__host__ __device__ constexpr int rows_slots(bool e4m3, int hd) {
    const int n = (kRowsSmemLimit - kRowsOther - rows_tables(MTP_MAX_PAGED_BATCH) - rows_q_bytes(hd) - rows_raw(e4m3, hd) * rows_slot_bytes(hd) / 2) / rows_slot_bytes(hd);
    return n < kRowsSlots ? n : kRowsSlots;
}

cudaError_t launch_rows_prepare(const RowsTcArgs& t, int kv_dtype, int sms, cudaStream_t s);
// one translation unit each (rows_attn_tc.cu)
cudaError_t launch_rows_tc_bf16(const RowsTcParams& p, cudaStream_t s);
cudaError_t launch_rows_tc_e4m3(const RowsTcParams& p, cudaStream_t s);
cudaError_t launch_rows_tc_bf16_shared(const RowsTcParams& p, cudaStream_t s);
cudaError_t launch_rows_tc_e4m3_shared(const RowsTcParams& p, cudaStream_t s);
cudaError_t launch_rows_merge(const RowsTcArgs& t, int kv_dtype, cudaStream_t s);

}  // namespace mtp
