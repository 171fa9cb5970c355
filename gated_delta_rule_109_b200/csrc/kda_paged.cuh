// Attention of one new token per sequence over a paged key-value cache: declarations and
// the split of the work shared by its kernels (internal header).
//
//     o = softmax(scale q K^T) V
// over the keys and values that a sequence's pages hold, the new token's own included when
// the call carries them (they are written to the cache as well).  Query heads h of one
// group h / (H / Hkv) share a key-value head.
//
// Split: a unit is 64 / HW consecutive keys of HW neighbouring key-value heads of one
// sequence, for one block of their query heads, and all units lie on one line ordered by
// sequence, heads, block and position.  HW is 2 where the number of key-value heads is even,
// else 1: neighbouring heads are neighbours in memory, and a reader of two takes 512 B (bf16,
// D = 128) of every position where a reader of one takes 256 B.  Of the U units CTA c of G (at
// most U of them) takes [c U / G, (c + 1) U / G), whatever sequence they belong to, so the
// CTAs' shares differ by at most one unit for every mix of lengths.  A stretch of units with
// one owner is written out at once; one that several CTAs share leaves each owner's running
// maximum, sum and unnormalised output in the workspace, and a second kernel joins them.
// The lengths are read on the device: nothing of that split depends on what the host knows.
// Where the rows are short, or many, every row has one owner for each group of heads and block
// instead; if already the table's bounds tell that, there is no second kernel.
#pragma once

#include "kda_internal.cuh"

namespace kda {

struct PagedArgs {
    const void *q, *k, *v;          // [B, H, D], [B, Hkv, D] or null, ditto
    void *k_cache, *v_cache;        // [num_pages, page_size, Hkv, D]
    const int *block_table;         // [B, max_pages]
    const int *lengths;             // [B] keys in the cache before the call; negative: idle row
    void *out;                      // [B, H, D]
    int B, H, Hkv, D, num_pages, page_size, max_pages;
    kda_dtype dtype;
    float scale;
    float *ws;
};

size_t paged_workspace_bytes(int H, int Hkv, int D, kda_dtype dtype);
cudaError_t launch_paged_decode(const PagedArgs &a, cudaStream_t stream);
// Reads and clears the status word: bit 0: a row named a page outside the cache or a length
// beyond its table.  Synchronous.
cudaError_t take_paged_device_status(unsigned int *status);

}  // namespace kda
