// efla_pages.cu -- pages of the state cache: init, free, fork, copy, compact, rows in and out.
//
// A page holds the whole recurrent state of one sequence; a slot names a sequence.  A plan (which
// page goes where) follows from the lists, the table and the owners alone, so it is the same on
// every run; the data then moves with every byte read once and written once.
//
// For caches of up to 4096 pages and lists of up to 256 entries one launch does both: every block
// makes the whole plan for itself in shared memory, moves its share, and the last one to finish writes
// the new table and owners, which the others have by then read (48 pairs of 8 KiB copied: 3.9 us; with two
// launches the call took twice as long; free, compact and fork of 24 of 256 pages of 1 MiB: 26.6 us, with two launches each 11
// more).
// Larger ones take a launch of one block for the plan.
#include "efla_kernels.h"
#include "efla_pages.cuh"

namespace efla {
namespace {

constexpr int kPlanThreads = 1024;

// Exclusive prefix sum of a 0/1 flag over the block, in thread order; *total: the block's sum.
__device__ __forceinline__ int block_rank(bool flag, int* total) {
    __shared__ int warps[33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned mask = __ballot_sync(0xffffffffu, flag);
    __syncthreads();
    if (lane == 0) warps[warp] = __popc(mask);
    __syncthreads();
    if (warp == 0) {
        const int own = warps[lane];
        int sum = own;
        for (int off = 1; off < 32; off <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, sum, off);
            if (lane >= off) sum += up;
        }
        warps[lane] = sum - own;
        if (lane == 31) warps[32] = sum;
    }
    __syncthreads();
    *total = warps[32];
    return warps[warp] + __popc(mask & ((1u << lane) - 1u));
}

__global__ void pages_init_kernel(PagesBlock b) {
    after_previous();
    const int words = b.n_slots + b.n_pages;
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < kPagesHeader) reinterpret_cast<int*>(b.err)[i] = 0;
    if (i < words) b.table[i] = -1;                              // table and owners are adjacent
    if (i < b.n_slots + 2 * b.n_pages) b.claim[i] = 0;           // claims and the move list too
}

__global__ void pages_free_kernel(PagesBlock b, const int* slots, int n) {
    after_previous();
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n) return;
    const int s = slots[i];
    if (s == -1) return;
    // a slot listed twice gives its page back once; the second time it is empty, an error
    const int page = s < 0 || s >= b.n_slots ? -1 : atomicExch(&b.table[s], -1);
    if (page < 0 || page >= b.n_pages) atomicOr(b.err, kPagesBadSlot);
    else b.owner[page] = -1;
}

// The lowest of the entries that name a slot claims it (entry i claims with n - i, so the
// largest claim wins and an unclaimed slot is zero).
__device__ __forceinline__ void claim_slots(const PagesBlock& b, const int* dest, int n) {
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int s = dest[i];
        if (s >= 0 && s < b.n_slots) atomicMax(&b.claim[s], n - i);
    }
    __syncthreads();
}
__device__ __forceinline__ void release_claims(const PagesBlock& b, const int* dest, int n) {
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int s = dest[i];
        if (s >= 0 && s < b.n_slots) b.claim[s] = 0;
    }
}

// Entry i of a fork (fresh: the destination has no page yet) or a copy (it has one) in order.
// *page: the source's page, -1 for a zeroed one.
__device__ __forceinline__ bool plan_entry(const PagesBlock& b, const int* source, const int* dest, int n, int i,
                                           bool fresh, int* page) {
    if (i >= n) return false;
    const int s = dest[i];
    if (s == -1) return false;
    bool ok = s >= 0 && s < b.n_slots && b.claim[s] == n - i;
    if (ok) {
        const int has = b.table[s];
        ok = fresh ? has == -1 : has >= 0 && has < b.n_pages;
    }
    const int from = source[i];
    *page = -1;
    if (ok && from != -1) {
        ok = from >= 0 && from < b.n_slots;
        if (ok) *page = b.table[from];
        ok = ok && *page >= 0 && *page < b.n_pages;
    }
    if (!ok) atomicOr(b.err, kPagesBadSlot);
    return ok;
}

__global__ void __launch_bounds__(kPlanThreads) pages_fork_plan(PagesBlock b, const int* source, const int* dest,
                                                                int n) {
    after_previous();
    claim_slots(b, dest, n);
    int count = 0;
    for (int base = 0; base < n; base += kPlanThreads) {
        const int i = base + threadIdx.x;
        int page, total;
        const bool ok = plan_entry(b, source, dest, n, i, true, &page);
        const int r = count + block_rank(ok, &total);
        if (ok && r < b.n_pages) {
            b.src[r] = page;
            b.dst[r] = dest[i];          // the slot, until it has a page
        }
        count += total;
    }
    const int wanted = count;
    count = min(count, b.n_pages);
    release_claims(b, dest, n);
    // the r-th entry gets the r-th free page
    int free_pages = 0;
    for (int base = 0; base < b.n_pages && free_pages < count; base += kPlanThreads) {
        const int p = base + threadIdx.x;
        int total;
        const bool is_free = p < b.n_pages && b.owner[p] == -1;
        const int r = free_pages + block_rank(is_free, &total);
        if (is_free && r < count) {
            const int s = b.dst[r];
            b.owner[p] = s;
            b.table[s] = p;
            b.dst[r] = p;
        }
        free_pages += total;
    }
    if (threadIdx.x == 0) {
        if (free_pages < wanted) atomicOr(b.err, kPagesFull);
        *b.moves = min(free_pages, count);
    }
}

__global__ void __launch_bounds__(kPlanThreads) pages_copy_plan(PagesBlock b, const int* source, const int* dest,
                                                                int n) {
    after_previous();
    claim_slots(b, dest, n);
    int count = 0;
    for (int base = 0; base < n; base += kPlanThreads) {
        const int i = base + threadIdx.x;
        int page, total;
        bool ok = plan_entry(b, source, dest, n, i, false, &page);
        ok = ok && source[i] != dest[i];
        const int r = count + block_rank(ok, &total);
        if (ok && r < b.n_pages) {
            b.src[r] = page;
            b.dst[r] = b.table[dest[i]];
        }
        count += total;
    }
    release_claims(b, dest, n);
    if (threadIdx.x == 0) *b.moves = min(count, b.n_pages);
}

__global__ void __launch_bounds__(kPlanThreads) pages_compact_plan(PagesBlock b) {
    after_previous();
    int live = 0;
    for (int base = 0; base < b.n_pages; base += kPlanThreads) {
        const int p = base + threadIdx.x;
        int total;
        block_rank(p < b.n_pages && b.owner[p] >= 0, &total);
        live += total;
    }
    // the r-th page in use from `live` on goes into the r-th free page before it
    int holes = 0, late = 0;
    for (int base = 0; base < b.n_pages; base += kPlanThreads) {
        const int p = base + threadIdx.x;
        const bool used = p < b.n_pages && b.owner[p] >= 0;
        int total;
        const bool hole = p < live && !used, move = p >= live && used;
        int r = holes + block_rank(hole, &total);
        if (hole) b.dst[r] = p;
        holes += total;
        r = late + block_rank(move, &total);
        if (move) b.src[r] = p;
        late += total;
    }
    __syncthreads();
    for (int r = threadIdx.x; r < late; r += kPlanThreads) {
        const int from = b.src[r], to = b.dst[r], s = b.owner[from];
        b.owner[to] = s;
        b.owner[from] = -1;
        if (s < b.n_slots) b.table[s] = to;
        else atomicOr(b.err, kPagesBadSlot);
    }
    if (threadIdx.x == 0) *b.moves = late;
}

// ---------------------------------------------------------------- moves
// 250 pages of 1 MiB: 96 us (5.5 TB/s read and written, 84% of the measured copy rate); 24 pages: 9 us.
// Bulk copies through shared memory instead took 102 and 11 us, four vectors a thread and eight
// blocks per SM 100 and 10.
constexpr int kMoveThreads = 256, kUnit = 8 * kMoveThreads;      // 16-byte vectors of a block's piece: 32 KiB

// The block's share of the moves src[m] -> dst[m] (src < 0: zeros), where no page is both.
__device__ __forceinline__ void move_pages(const int* src, const int* dst, int moves, char* pool, size_t page_bytes,
                                           long vecs) {
    const long pieces = (vecs + kUnit - 1) / kUnit, total = moves * pieces;
    for (long u = blockIdx.x; u < total; u += gridDim.x) {
        const int m = (int)(u / pieces);
        const long v0 = (u % pieces) * kUnit + threadIdx.x;
        const int from = src[m];
        const uint4* in = reinterpret_cast<const uint4*>(pool + (size_t)(from < 0 ? 0 : from) * page_bytes);
        uint4* out = reinterpret_cast<uint4*>(pool + (size_t)dst[m] * page_bytes);
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = make_uint4(0, 0, 0, 0);
            if (from >= 0 && v0 + i * kMoveThreads < vecs) v[i] = in[v0 + i * kMoveThreads];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (v0 + i * kMoveThreads < vecs) out[v0 + i * kMoveThreads] = v[i];
    }
}

__global__ void __launch_bounds__(kMoveThreads) pages_move_kernel(PagesBlock b, char* pool, size_t page_bytes, long vecs) {
    after_previous();
    move_pages(b.src, b.dst, *b.moves, pool, page_bytes, vecs);
}

// Exclusive prefix sum over the block's threads; *total: the block's sum.
__device__ __forceinline__ int block_sum(int value, int* total) {
    __shared__ int warps[kMoveThreads / 32 + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int sum = value;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, off);
        if (lane >= off) sum += up;
    }
    __syncthreads();
    if (lane == 31) warps[warp] = sum;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kMoveThreads / 32; ++w) {
        if (w == warp) before = all;
        all += warps[w];
    }
    *total = all;
    return before + sum - value;
}

// Whether entry i (source `from`, destination `to`) may run: as plan_entry, with the list in
// shared memory instead of claims.
__device__ __forceinline__ bool list_entry(const PagesBlock& b, const int* dests, int i, int from, int to, bool fresh,
                                           int* page, int* has) {
    bool ok = to >= 0 && to < b.n_slots;
    if (ok) {
        *has = b.table[to];
        ok = fresh ? *has == -1 : *has >= 0 && *has < b.n_pages;
    }
    *page = -1;
    if (from != -1) {
        ok = ok && from >= 0 && from < b.n_slots;
        if (ok) *page = b.table[from];
        ok = ok && *page >= 0 && *page < b.n_pages;
    }
    for (int m = 0; m < i; ++m) ok = ok && dests[m] != to;
    if (!ok) atomicOr(b.err, kPagesBadSlot);
    return ok;
}

constexpr int kFusedList = 256, kFusedPages = 4096, kPer = kFusedPages / kMoveThreads;
struct FusedPlan {
    int dests[kFusedList], slots[kFusedList];
    int src[kFusedPages / 2], dst[kFusedPages / 2];
};

// True in the last block that gets here: the others have read all that it may now overwrite.
__device__ __forceinline__ bool last_block(const PagesBlock& b) {
    __shared__ bool last;
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(b.tickets, 1u) == gridDim.x - 1;
        if (last) *b.tickets = 0;
    }
    __syncthreads();
    return last;
}

__global__ void __launch_bounds__(kMoveThreads) pages_fork_kernel(PagesBlock b, const int* source,
                                                                  const int* dest, int n, char* pool,
                                                                  size_t page_bytes, long vecs) {
    __shared__ FusedPlan plan;
    after_previous();
    const int i = threadIdx.x, to = i < n ? dest[i] : -1, from = i < n ? source[i] : -1;
    // the free pages of this thread's stretch
    const int per = (b.n_pages + kMoveThreads - 1) / kMoveThreads, p0 = i * per;
    uint32_t open = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        if (k < per && p0 + k < b.n_pages && b.owner[p0 + k] == -1) open |= 1u << k;
    plan.dests[i] = to;
    __syncthreads();
    int page, has, count, open_all;
    const bool ok = to != -1 && list_entry(b, plan.dests, i, from, to, true, &page, &has);
    const int r = block_sum(ok, &count);
    if (ok) {
        plan.src[r] = page;
        plan.slots[r] = to;
    }
    int f = block_sum(__popc(open), &open_all);
    const int moves = min(count, open_all);
    for (; open && f < moves; open &= open - 1) plan.dst[f++] = p0 + __ffs(open) - 1;
    __syncthreads();
    if (pool) move_pages(plan.src, plan.dst, moves, pool, page_bytes, vecs);
    if (!last_block(b)) return;
    if (i < moves) {
        b.table[plan.slots[i]] = plan.dst[i];
        b.owner[plan.dst[i]] = plan.slots[i];
    }
    if (i == 0 && moves < count) atomicOr(b.err, kPagesFull);
}

__global__ void __launch_bounds__(kMoveThreads) pages_compact_kernel(PagesBlock b, char* pool, size_t page_bytes, long vecs) {
    __shared__ FusedPlan plan;
    after_previous();
    const int per = (b.n_pages + kMoveThreads - 1) / kMoveThreads, p0 = threadIdx.x * per;
    uint32_t used = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        if (k < per && p0 + k < b.n_pages && b.owner[p0 + k] >= 0) used |= 1u << k;
    int live, holes, late;
    block_sum(__popc(used), &live);
    const int here = min(max(b.n_pages - p0, 0), per);                     // pages of the stretch
    const int low = min(max(live - p0, 0), here);                          // those before `live`
    const uint32_t low_bits = (1u << low) - 1u;
    uint32_t hole = ~used & low_bits, move = used & ~low_bits;
    int h = block_sum(__popc(hole), &holes), l = block_sum(__popc(move), &late);
    for (; hole; hole &= hole - 1) plan.dst[h++] = p0 + __ffs(hole) - 1;
    for (; move; move &= move - 1) plan.src[l++] = p0 + __ffs(move) - 1;
    __syncthreads();
    move_pages(plan.src, plan.dst, late, pool, page_bytes, vecs);
    if (!last_block(b)) return;
    for (int r = threadIdx.x; r < late; r += kMoveThreads) {
        const int from = plan.src[r], to = plan.dst[r], slot = b.owner[from];
        b.owner[to] = slot;
        b.owner[from] = -1;
        if (slot < b.n_slots) b.table[slot] = to;
        else atomicOr(b.err, kPagesBadSlot);
    }
}

// Moves as if all at once: a block owns a strip of `width` 16-byte columns of every page, reads it
// for all moves into shared memory, then writes it.
__device__ __forceinline__ void move_strip(const int* src, const int* dst, int moves, char* pool, size_t page_bytes,
                                           long vecs, int width, uint4* held) {
    const long c0 = (long)blockIdx.x * width;
    const int w = (int)min((long)width, vecs - c0), total = moves * w;
#pragma unroll 4
    for (int i = threadIdx.x; i < total; i += kMoveThreads) {
        const int from = src[i / w];
        held[i] = from < 0 ? make_uint4(0, 0, 0, 0)
                           : *reinterpret_cast<const uint4*>(pool + (size_t)from * page_bytes + (c0 + i % w) * 16);
    }
    __syncthreads();
#pragma unroll 4
    for (int i = threadIdx.x; i < total; i += kMoveThreads)
        *reinterpret_cast<uint4*>(pool + (size_t)dst[i / w] * page_bytes + (c0 + i % w) * 16) = held[i];
}

__global__ void __launch_bounds__(kMoveThreads) pages_strip_kernel(PagesBlock b, char* pool, size_t page_bytes, long vecs,
                                                                   int width) {
    extern __shared__ uint4 held[];
    after_previous();
    move_strip(b.src, b.dst, *b.moves, pool, page_bytes, vecs, width, held);
}

__global__ void __launch_bounds__(kMoveThreads) pages_copy_kernel(PagesBlock b, const int* source,
                                                                  const int* dest, int n, char* pool,
                                                                  size_t page_bytes, long vecs, int width) {
    extern __shared__ uint4 held[];
    __shared__ int dests[kFusedList], src[kFusedList], dst[kFusedList];
    after_previous();
    const int i = threadIdx.x, to = i < n ? dest[i] : -1, from = i < n ? source[i] : -1;
    dests[i] = to;
    __syncthreads();
    int page, has, moves;
    bool ok = to != -1 && list_entry(b, dests, i, from, to, false, &page, &has);
    ok = ok && from != to;
    const int r = block_sum(ok, &moves);
    if (ok) {
        src[r] = page;
        dst[r] = has;
    }
    __syncthreads();
    move_strip(src, dst, moves, pool, page_bytes, vecs, width, held);
}

// Rows into the pages of their slots (write) or out of them; one block per 4 KiB of a row.
__global__ void __launch_bounds__(256) pages_rows_kernel(PagesBlock b, char* pool, size_t page_bytes, char* rows,
                                                         size_t row_bytes, const int* slots, int n,
                                                         int pieces, bool write) {
    after_previous();
    const int i = blockIdx.x / pieces;
    const size_t at = ((size_t)(blockIdx.x % pieces) * 256 + threadIdx.x) * 16;
    const int s = slots[i];
    if (s == -1) return;
    bool bad = s < 0 || s >= b.n_slots;
    const int page = bad ? -1 : b.table[s];
    bad |= page < 0 || page >= b.n_pages;
    if (write)                                   // of rows for one slot the first is taken
        for (int m = threadIdx.x; m < i; m += 256) bad |= slots[m] == s;
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) atomicOr(b.err, kPagesBadSlot);
        return;
    }
    if (at >= row_bytes) return;
    uint4* cached = reinterpret_cast<uint4*>(pool + (size_t)page * page_bytes + at);
    uint4* row = reinterpret_cast<uint4*>(rows + (size_t)i * row_bytes + at);
    if (write) *cached = *row;
    else *row = *cached;
}

int move_grid() {
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms * 2;
}

}  // namespace

cudaError_t launch_pages_init(const PagesBlock& b, cudaStream_t stream) {
    const int words = b.n_slots + 2 * b.n_pages + kPagesHeader;
    return launch_after(pages_init_kernel, (words + 255) / 256, 256, 0, stream, b);
}

cudaError_t launch_pages_free(const PagesBlock& b, const int* slots, int n, cudaStream_t stream) {
    return launch_after(pages_free_kernel, (n + 255) / 256, 256, 0, stream, b, slots, n);
}

static cudaError_t launch_moves(const PagesBlock& b, void* pool, size_t page_bytes, size_t data_bytes,
                                cudaStream_t stream) {
    return launch_after(pages_move_kernel, move_grid(), kMoveThreads, 0, stream, b, static_cast<char*>(pool),
                        page_bytes, (long)(data_bytes / 16));
}

// A fused call's blocks: what its largest possible number of moves keeps busy.
static unsigned fused_grid(long moves, long vecs) {
    const long pieces = moves * ((vecs + kUnit - 1) / kUnit), most = move_grid();
    return (unsigned)(pieces < 1 ? 1 : pieces < most ? pieces : most);
}

cudaError_t launch_pages_fork(const PagesBlock& b, void* pool, size_t page_bytes, size_t data_bytes, const int* source,
                              const int* dest, int n, cudaStream_t stream) {
    const long vecs = pool ? (long)(data_bytes / 16) : 0;
    if (n <= kFusedList && b.n_pages <= kFusedPages) {
        return launch_after(pages_fork_kernel, fused_grid(n, vecs), kMoveThreads, 0, stream, b, source, dest, n,
                            static_cast<char*>(pool), page_bytes, vecs);
    }
    const cudaError_t e = launch_after(pages_fork_plan, 1, kPlanThreads, 0, stream, b, source, dest, n);
    if (e != cudaSuccess || !pool) return e;
    return launch_moves(b, pool, page_bytes, data_bytes, stream);
}

cudaError_t launch_pages_compact(const PagesBlock& b, void* pool, size_t page_bytes, size_t data_bytes,
                                 cudaStream_t stream) {
    if (b.n_pages <= kFusedPages) {
        const long vecs = (long)(data_bytes / 16);
        return launch_after(pages_compact_kernel, fused_grid(b.n_pages / 2, vecs), kMoveThreads, 0, stream, b,
                            static_cast<char*>(pool), page_bytes, vecs);
    }
    const cudaError_t e = launch_after(pages_compact_plan, 1, kPlanThreads, 0, stream, b);
    if (e != cudaSuccess) return e;
    return launch_moves(b, pool, page_bytes, data_bytes, stream);
}

cudaError_t launch_pages_copy(const PagesBlock& b, void* pool, size_t page_bytes, size_t data_bytes, const int* source,
                              const int* dest, int n, cudaStream_t stream) {
    // strips as wide as shared memory allows, but enough of them for every SM (down to 128 bytes)
    const long vecs = (long)(data_bytes / 16), spread = (vecs + 295) / 296;
    long width = kPagesCopyMax / n;
    if (width > (spread > 8 ? spread : 8)) width = spread > 8 ? spread : 8;
    if (width > vecs) width = vecs;
    const unsigned grid = (unsigned)((vecs + width - 1) / width);
    const size_t held = (size_t)n * width * 16;
    constexpr int kHeld = kPagesCopyMax * 16;
    static std::atomic<uint64_t> done{0}, done_list{0};
    cudaError_t e;
    if (n <= kFusedList) {
        if ((e = set_smem_limit_once(pages_copy_kernel, kHeld, done_list)) != cudaSuccess) return e;
        return launch_after(pages_copy_kernel, grid, kMoveThreads, held, stream, b, source, dest, n,
                            static_cast<char*>(pool), page_bytes, vecs, (int)width);
    }
    e = launch_after(pages_copy_plan, 1, kPlanThreads, 0, stream, b, source, dest, n);
    if (e != cudaSuccess) return e;
    if ((e = set_smem_limit_once(pages_strip_kernel, kHeld, done)) != cudaSuccess) return e;
    return launch_after(pages_strip_kernel, grid, kMoveThreads, held, stream, b, static_cast<char*>(pool),
                        page_bytes, vecs, (int)width);
}

cudaError_t launch_pages_rows(const PagesBlock& b, void* pool, size_t page_bytes, void* rows, size_t row_bytes,
                              const int* slots, int n, bool write, cudaStream_t stream) {
    const int pieces = (int)((row_bytes + 4095) / 4096);
    return launch_after(pages_rows_kernel, (unsigned)((long)n * pieces), 256, 0, stream, b, static_cast<char*>(pool),
                        page_bytes, static_cast<char*>(rows), row_bytes, slots, n, pieces, write);
}

}  // namespace efla
