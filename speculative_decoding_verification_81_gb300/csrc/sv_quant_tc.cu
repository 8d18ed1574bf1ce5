// sv_quant_tc.cu -- the chunk attention over pages held in 4 bits: the kernel of
// sv_chunk_tc.cuh with sixteen warps.
//
// Source: as sv_chunk_tc.cu, which says how the steps, items and warps go
// together.  What differs: warps 8 and 11 copy the codes and parameters of K and
// V tiles to a ring of their own (8.5 KB a tile at D = 128 for 32), and warps
// 12-15, a thread a slot, turn each into 16-bit operands in the swizzled tiles that
// the products read:
//     S = Q (codes_k - 8)^T               (bf16 products; the codes are exact)
//     x = step_k S + middle_k sum(q)      (f32, log2 units; middle = minimum + 8 steps)
//     P = 2^(x + e - m), rounded to f16;  l += 2^(x - m)
//     O += P V 2^-e                       (f16 products)
// where m is 7 below the largest x + e (up to 15 while it lags), so that P stays below 2^15
// and is rounded by at most 2^-11 of itself down to 2^-21 of the largest -- beside one slot
// with most of a row's weight the others' P are small, and l, which is f32, has them
// all -- and e is the exponent of the largest value of V in a warp's 32 slots, fourteen
// less: V 2^-e stays below 2^15, and its middle and then its values are rounded by at
// most 2^-11 of themselves each, down to 2^-28 of that largest value (its steps not at
// all).  K is not rounded -- a score's error would be in the log-sum-exp, which is
// f32 -- and what P and V lose is a third of what the output's own rounding to bf16
// takes (error against 64 bits 1.7e-3 of the output's size, which is that rounding,
// with a slot of weight 0.99 or 0.999 among 16384 too; with P and V in bf16 it was
// 3.4e-3; with the largest P at 2^0 those two 5.7e-3 and 5.7e-2).  A slot that no row
// of the item sees is zeros.  A row may be a node of a draft tree: it then sees
// the slots before its sequence's rows and its own path's, a 64-bit set that each
// softmax thread makes of the parents.
//
// Why not the values of K in 16 bits: two parts of them are needed for the scores'
// last bits, which makes three products of two.  Why queries as the rows of S although
// every thread then reads every slot's step and middle (64 reads of 16 bytes a tile):
// with slots as the rows a thread has its own, but a tile does 48 columns' work
// instead of 128 or 256 and its barriers cost what they cost here (2048 rows after
// 14336 slots 1390 us against 538, trees of 26 80 against 34; chains of 9 97 and 85).
//
// What bounds it (32 query over 8 KV heads of 128): the chain of a step's parts and
// the one instruction cache that all roles are fetched through, not the tensor core
// (2048 rows after 14336 slots 538-544 us, 0.5 of the measured rate; a prompt of 4096
// 181 us, 0.40) nor memory (chains of 9 after 2048-4096 slots for 32 requests 85 us,
// 0.19 of the measured bandwidth, and the same for 8 to 40 columns a sequence).  A
// step's softmax takes 2600 cycles, a tile's expansion 900 for K and 900 for V.
// Ablations of the latter: without the scores' constants 490 us, without exponentials
// 485, without the operands' stores 470, without the three 340.
// Tried without gain: the expansion by eight warps, four for K and four for V (fewer
// registers for the softmax); tiles copied by each expanding warp in 16-byte pieces
// (chains 133 us) or loaded to registers a tile ahead (121); three places for tiles
// and six for codes; 152 or 144 registers for the softmax; up to 64 rows twice in
// their Q tile, so that two threads share a row's slots (chains 90 us, prompts 567).
#include "sv_chunk_tc.cuh"

namespace sv {
namespace chunk {

const void *quant_kernel_fn(int D) {
    return D == 128 ? reinterpret_cast<const void *>(&chunk_attention_kernel<128, true>)
                    : reinterpret_cast<const void *>(&chunk_attention_kernel<64, true>);
}

template <int D>
constexpr int kQuantSmem = (kStagesOf<D, true> + 2) * kTileBytes<D> + kRawBytes<D, true> + (int)sizeof(QuantShared);
static_assert(kQuantSmem<128> <= 227 * 1024 && kQuantSmem<64> <= 227 * 1024, "shared memory");

int quant_smem_bytes(int D) { return D == 128 ? kQuantSmem<128> : kQuantSmem<64>; }

}  // namespace chunk
}  // namespace sv
