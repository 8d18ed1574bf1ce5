// sv_quant_tc.cu -- the chunk attention over pages held in 4 bits: the kernel of
// sv_chunk_tc.cuh with sixteen warps.
//
// Source: as sv_chunk_tc.cu, which says how the steps, items and warps go
// together.  What differs: warps 8 and 11 copy the codes and parameters of K and
// V tiles to a ring of their own (8.5 KB a tile at D = 128 for 32), and warps
// 12-15, a thread a slot, turn each into bf16 values in the swizzled tiles that
// the products read.  A value is minimum + step * code rounded once to bf16, what
// a cache in bf16 would hold of it; a slot that no row of the item sees is zeros.
// A row may be a node of a draft tree: it then sees the slots before its sequence's
// rows and its own path's, a 64-bit set that each softmax thread makes of the
// parents.
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
