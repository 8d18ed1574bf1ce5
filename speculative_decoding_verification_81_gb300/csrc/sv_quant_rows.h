// sv_quant_rows.h -- parameters and entry of the form for few rows a sequence of
// the attention over pages held in 4 bits (sv_quant_rows.cu).
#pragma once

#include "sv_chunk.cuh"
#include "sv_quant_list.h"

namespace sv {
namespace chunk {

constexpr int kRowsCols = 16;      // columns (rows times heads) of an item at most
constexpr int kRowsMaxGrid = 512;  // CTAs of a call at most: the workspace's shares and counters
// Columns of a mean sequence up to which a call takes this form.  Both measured, us, this one first, for 32
// requests after 2048-4096 slots: 4 columns 43 and 117, 8 columns 44 and 85, 16 columns 57 and 84; 24 columns
// (two items of this form a head) 99 and 84.  A form of 40 columns took 106 for 36, where the other takes 85.
// Uneven batches, n single tokens after 1000 slots beside a chunk of m rows after 2000 (n, m, the mean's columns: this
// form, the other): 64, 512, 36: 173, 115; 64, 2048, 132: 700, 203; 256, 512, 12: 263, 346; 256, 2048, 36: 793, 453;
// 700, 512, 8: 470, 861; 700, 2048, 16: 1009, 978.  The mean takes the quicker form or one 3% behind; the two parts in a
// call each would take 79, 170, 153, 243, 321 and 412, but the lengths are on the device.
constexpr int kRowsMost = 16;
constexpr float kUnset = -3.4028234663852886e38f;  // u of a column that has seen no slot: no finite score is less
constexpr float kRoom = 15.f;      // log2 of the largest P; kTop as u moves
constexpr float kLeast = -80.f;    // log2 of a step below which it counts as this much for u (l stays below 2^(15 + 80) a slot)

struct RowsParams : QuantParams {
    const uint16_t *q;
    long long q_stride;  // elements between rows of q
    RowsShape rows;
};

// The counter of an item shared from CTA `cta` on, in the set of the given call.
SV_CALL_HD int rows_counter(unsigned long long call, int cta) { return (int)(call & 1) * kRowsMaxGrid + cta; }

// The form for the call's rows; -1 where it has too many.
int rows_form(const ChunkArgs &args);
sv_status launch_rows(const ChunkArgs &args, const QuantParams &params, int form, cudaStream_t stream);

}  // namespace chunk
}  // namespace sv
