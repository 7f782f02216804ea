// paged_attn_tc.cuh -- attention over the paged cache on the tensor cores:
// sizes shared by the kernel and the host's plan (internal).
#pragma once

#include <cuda.h>

#include "paged.cuh"

namespace mtp {

constexpr int kTcTileLog2 = 7, kTcTile = 1 << kTcTileLog2;          // positions of a tile: the MMA's M side
constexpr int kTcSlotsMax = 24;       // ring slots of a CTA at most
constexpr int kTcMeta = 16;           // tiles of page scales the producer may be ahead
// What beginning an item costs a CTA, in tiles.  16 sequences of 2k to 32k
// positions in e4m3 / 64 sequences of 4096 / 64 windows of 1024 in bf16 (head
// dimension 256, 4 KV heads) take 105.6 / 97.2 / 44.8 us with 0, 99.2 / 96.8 /
// 43.0 with 3 and 98.6 / 98.3 / 43.5 with 5.
constexpr int kTcOpen = 3;
constexpr int kTcFix = 256;           // positions listed as not finite
constexpr int kTcSmemLimit = 227 * 1024 - 64;   // beside the static words

struct PagedTcArgs {
    CUtensorMap tk, tv;               // (dimension, slot, KV head, page) of k and v
    PagedAttnArgs a;
    int slots;                        // ring slots
};

// tiles of P in shared memory: one where two would leave the ring too little
__host__ __device__ constexpr int tc_p_bufs(bool e4m3, int hd, int RT) { return !e4m3 && RT * hd > 32 * 256 ? 1 : 2; }
// bytes of shared memory besides the ring
__host__ __device__ constexpr int tc_other(bool e4m3, int hd, int RT, int B) {
    return (e4m3 ? 3 : 2 * 2) * RT * hd                          // Q, in parts
           + tc_p_bufs(e4m3, hd, RT) * (e4m3 ? 3 : 2 * 2) * RT * 128 // P, in parts
           + kTcMeta * 8 * 2 * 4 + kTcMeta * 4                   // page scales
           + RT * 4 * (4 + 3 + 4) + 2 * kTcFix * 4 + hd * 4          // row tables, list, rotation table
           + (2 * kTcSlotsMax + kTcMeta + 16) * 8 + kPlanTmp * 8 + 64 + plan_bytes(B) + 1024;
}
__host__ __device__ constexpr int tc_slot_bytes(bool e4m3, int hd) { return kTcTile * (hd < 128 ? hd : 128) * (e4m3 ? 1 : 2); }
__host__ __device__ constexpr int tc_slots(bool e4m3, int hd, int RT, int B) {
    int n = (kTcSmemLimit - tc_other(e4m3, hd, RT, B)) / tc_slot_bytes(e4m3, hd);
    if (n > kTcSlotsMax) n = kTcSlotsMax;
    return n;
}

// Rows of a row tile: the smallest of 16, 32, 64 that holds all rows (at head
// dimension 512 at most 32: the queries of more leave no ring), fewer where a
// value tile would not fit the ring beside a large batch's plan.
inline int tc_rows_max(int rows, int hd) { return rows <= 16 ? 16 : rows <= 32 || hd == 512 ? 32 : 64; }
inline int tc_rows(bool e4m3, int rows, int hd, int B) {
    int RT = tc_rows_max(rows, hd);
    while (RT > 16 && tc_slots(e4m3, hd, RT, B) < (hd + 127) / 128) RT /= 2;
    return RT;
}

// one translation unit each (paged_attn_tc.cu)
cudaError_t launch_paged_attn_tc_bf16(const PagedTcArgs& p, cudaStream_t s);
cudaError_t launch_paged_attn_tc_e4m3(const PagedTcArgs& p, cudaStream_t s);

}  // namespace mtp
