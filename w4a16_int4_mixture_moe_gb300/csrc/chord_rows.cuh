// A few weight rows times many activation rows on the tcgen05 tensor cores:
//   D[r, j] = sum_k W[w0 + r, k] * x[row(j), k]
// for the router's logits (the experts' rows, a tile of consecutive tokens) and for the first half of
// an adapter (the slot's rows, the block's gathered rows).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace chord {

struct RowsArgs {
    const void* x;
    int64_t x_rows, x_stride;
    const void* W;           // bf16 [w_rows, K] dense
    int64_t w_rows;
    int K;
    int parts, part_rows;    // the sum over `parts` weight matrices, part_rows rows apart (logits)
    int R;                   // weight rows of an item
    int nb;                  // rows of x an item holds at most: a multiple of 16, at most 128
    int splits;              // K slices, a cluster of CTAs: 1, 2, 4 or 8
    int64_t items;
    // logits: item = (tile of nb tokens, group of R experts); out [x_rows, E]
    int E, groups;
    float* out;
    // adapters (nblocks not null): item = block of the plan, out [P, R]
    const int32_t* nblocks;
    const int32_t* block_slot;
    const int32_t* rows;     // [blocks, block_rows], a prefix; -1: none
    int block_rows;          // a multiple of nb: an item is nb of a block's rows
    int div;
    int* err;
};

// Rows of x that an item of R weight rows (at most 512) may hold.
int rows_block(int R);
// The largest split of K whose join fits the shared memory, at most `want`; wanted where items are few.
int rows_splits(int R, int nb, int steps, int64_t items, int want);
cudaError_t launch_rows(const RowsArgs& a, bool pdl, cudaStream_t st);

}  // namespace chord
