// efla_pages.cuh -- the state cache's block, and a row's pages in the paged steps (internal).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "efla_common.cuh"
#include "efla_scan.cuh"

namespace efla {

// The block, in int32 words: a header of 64 (word 0: errors, 1 and 2: the running call's),
// the table (slot -> page), the owners (page -> slot), then scratch: a claim per slot (zero
// between calls) and the list of page moves.
constexpr int kPagesHeader = 64;
enum : uint32_t { kPagesBadSlot = 4u, kPagesFull = 8u };   // error word bits
struct PagesBlock {
    uint32_t* err;
    int* moves;
    uint32_t* tickets;     // blocks of the running call that are done; zero between calls
    int* table;
    int* owner;
    int* claim;
    int* src;
    int* dst;
    int n_pages, n_slots;
};
inline size_t pages_words(int n_pages, int n_slots) {
    return (size_t)kPagesHeader + 2 * (size_t)n_slots + 3 * (size_t)n_pages;
}
inline PagesBlock pages_block(void* p, int n_pages, int n_slots) {
    int* w = static_cast<int*>(p);
    PagesBlock b;
    b.err = reinterpret_cast<uint32_t*>(w);
    b.moves = w + 1;
    b.tickets = reinterpret_cast<uint32_t*>(w + 2);
    b.table = w + kPagesHeader;
    b.owner = b.table + n_slots;
    b.claim = b.owner + n_pages;
    b.src = b.claim + n_slots;
    b.dst = b.src + n_pages;
    b.n_pages = n_pages;
    b.n_slots = n_slots;
    return b;
}

// Row n's pages, computed by a whole block (every thread calls it).  A row is refused, with the
// error recorded, where it would be wrong or race: a slot out of range or without a page, a slot
// that an earlier row has too, or another source slot that some row of this call writes.  The
// answer depends on the lists alone, never on the order in which blocks run.
struct RowPages {
    bool active;
    long write, read;      // pages; read < 0: from a zero state
};
__device__ __forceinline__ RowPages row_pages(const PagedRows& P, int slot, int src, bool* bad) {
    RowPages r{true, -1, -1};
    if (slot < 0 || slot >= P.n_slots) *bad = true;
    else r.write = P.table[slot];
    if (src == slot) r.read = r.write;
    else if (src != -1) {
        if (src < 0 || src >= P.n_slots) *bad = true;
        else r.read = P.table[src];
        *bad |= r.read < 0 || r.read >= P.n_pages;
    }
    *bad |= r.write < 0 || r.write >= P.n_pages;
    return r;
}
__device__ __forceinline__ RowPages paged_row(const PagedRows& P, int N, int n) {
    const int slot = P.slots[n];
    if (slot == -1) return RowPages{false, -1, -1};
    const int src = P.source ? P.source[n] : slot;
    bool bad = false;
    for (int m = threadIdx.x; m < n; m += blockDim.x) bad |= P.slots[m] == slot;
    if (src != slot && src != -1)
        for (int m = threadIdx.x; m < N; m += blockDim.x) bad |= P.slots[m] == src;
    RowPages r = row_pages(P, slot, src, &bad);
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) atomicOr(P.err, kPagesBadSlot);
        r.active = false;
    }
    return r;
}

cudaError_t launch_pages_init(const PagesBlock& b, cudaStream_t stream);
cudaError_t launch_pages_free(const PagesBlock& b, const int* slots, int n, cudaStream_t stream);
cudaError_t launch_pages_fork(const PagesBlock& b, void* pool, size_t page_bytes, size_t data_bytes, const int* source,
                              const int* dest, int n, cudaStream_t stream);
cudaError_t launch_pages_copy(const PagesBlock& b, void* pool, size_t page_bytes, size_t data_bytes, const int* source,
                              const int* dest, int n, cudaStream_t stream);
cudaError_t launch_pages_compact(const PagesBlock& b, void* pool, size_t page_bytes, size_t data_bytes,
                                 cudaStream_t stream);
cudaError_t launch_pages_rows(const PagesBlock& b, void* pool, size_t page_bytes, void* rows, size_t row_bytes,
                              const int* slots, int n, bool write, cudaStream_t stream);
// pairs of one copy: 16 bytes of every source page have to fit a CTA's shared memory
constexpr int kPagesCopyMax = 8192;

}  // namespace efla
