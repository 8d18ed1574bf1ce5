// sv_chunk_tc.cu -- attention of chunks of new tokens over a paged KV cache
// (prompt chunks of any length, mixed with single tokens) on the
// 5th-generation tensor cores.
//
// Source: the paged KV of "Chapitre 9", section "Ce que prépare le Chapitre
// 9"; "Chapitre 9" §9.1 (the prefix's K/V is reused, the new positions attend
// to it and causally to each other in one pass).
//
// Row i of sequence b sits at position p = L_b + i and sees the slots
// max(0, p - window + 1) .. p.  An item is a run of consecutive rows of one
// sequence and one KV head: the G = Hq/Hkv heads of a token share K/V, so a
// Q tile holds tpt = 128 / G tokens (128 MMA rows), and an item one or two
// tiles.  For each 128-slot tile of K/V an item runs one step a Q tile:
//     S = Q K^T (128 x 128, f32 in tensor memory)
//     P = 2^(scale * log2 e * S - m), written over S as bf16
//     O += P V (f32 in tensor memory)
// with a running row maximum m that moves only when it grows by more than
// 2^8 (O is then rescaled) and the row sums of the f32 P.
//
// Two streams of steps alternate, so that the tensor core works on one
// stream's products while the softmax warps of the other turn S into P: the
// steps of a CTA are one list, step g belongs to stream g & 1 (its own S/P
// and O columns and its own four softmax warps).  An item of two Q tiles puts
// a tile on each stream and both read every K/V tile; an item of one Q tile
// (single tokens, short chunks) gives the streams its K/V tiles in turn, and
// their (O, m, sum) are merged at the end.
//
// The work list is every (sequence, KV head, item, K/V tile).  A persistent
// grid takes equal contiguous ranges of it, weighed by what tiles and items take
// (sv_chunk_list.h), so the load is even whatever the lengths;
// an item cut by a range's end leaves partials in the workspace, merged by the
// warp that arrives last, in index order.
//
// Warps: 0-3 and 4-7 softmax of streams 0 and 1 (one thread a row); 8 and 11
// load K and V tiles by TMA through the page table; 9 issues the products; 10
// walks the work list, publishes the items, loads Q and at the end checks the
// page table and writes seq_status.  Every wait is bounded.
//
// What bounds it (32 query over 8 KV heads of 128, one GB300): long chunks the
// tensor core and the power cap -- 4096 rows after 28672 slots 1.19 ms (1.73
// PFLOP/s) after a pause, 1.31-1.38 ms back to back; large batches of single
// tokens HBM -- 128 after 4096 slots 316-321 us, 6.8 TB/s.  In between, a step's chain: S product, softmax of one row a thread
// (about 1400 cycles a tile), PV product; and for short items the instructions
// themselves: the roles' code is fetched through one instruction cache, and
// every shortening of it (loops kept rolled, rare parts out of line) gained
// several per cent.  Tried without gain: P released in two halves; the softmax
// in two or four rounds of columns read twice from tensor memory; with D = 64,
// P in columns of its own so that the next S is made during the softmax;
// products of 64 rows for few rows; the two streams finishing items in turn.
#include "sv_chunk_tc.cuh"

namespace sv {
namespace chunk {

const void *kernel_fn(int D) {
    return D == 128 ? reinterpret_cast<const void *>(&chunk_attention_kernel<128, false>)
                    : reinterpret_cast<const void *>(&chunk_attention_kernel<64, false>);
}

static_assert((kStagesOf<128, false> + 2) * kTileBytes<128> + sizeof(Shared) <= 227 * 1024, "shared memory");

int smem_bytes(int D) {
    return (D == 128 ? (kStagesOf<128, false> + 2) * kTileBytes<128> : (kStagesOf<64, false> + 2) * kTileBytes<64>) + (int)sizeof(Shared);
}

}  // namespace chunk
}  // namespace sv
