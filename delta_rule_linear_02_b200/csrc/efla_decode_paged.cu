// efla_decode_paged.cu -- one recurrent (decode) token for the rows of a batch whose states lie in
// the pages of a state cache: the update of the dense step (the exact flow, gated or not),
//     r = k^T S, p = q^T S, c = q.k,  w = d alpha r - abar v,  S <- d S - k w^T,  o = d p - c w,
// d = e^g (1 without g), with S read from one page and written to the same or another one.
// Bound by memory: the state is read once and written once, 8 bytes for four flops.  Column j of the new
// state needs column j of the old one alone: in the first kernel a block owns 32 columns of one head and passes
// them through registers once, every load of it in flight at the start.  For few rows that is the
// shortest way (9 rows of 16 heads of 128: 6.3 us for 19 MB); for many the second kernel is
// better, as blocks of one short life each leave memory idle between them.
#include "efla_kernels.h"
#include "efla_pages.cuh"
#include "efla_scan.cuh"
#include "sm100.cuh"

namespace efla {
using namespace sm100;
namespace {
constexpr int kCols = 32;
constexpr int kThreads = 256;

template <typename Tin, int D>
__global__ void __launch_bounds__(kThreads) decode_paged_kernel(const Tin* q, const Tin* k,
                                                                const Tin* v,
                                                                const Tin* beta,
                                                                const float* g, char* pool,
                                                                Tin* o, int N, int H, int rule,
                                                                PagedRows P) {
    constexpr int RPT = D / 32;
    constexpr int SLICES = D / kCols;
    after_previous();
    const int t = threadIdx.x, cq = t & 7, rg = t >> 3, warp = t >> 5, lane = t & 31;
    const long head = blockIdx.x / SLICES;
    const int n = (int)(head / H), hh = (int)(head % H);
    const int j0 = (blockIdx.x % SLICES) * kCols + cq * 4;
    const RowPages pg = paged_row(P, N, n);
    if (!pg.active) return;
    float* to = reinterpret_cast<float*>(pool + pg.write * P.page_bytes) + (long)hh * D * D;
    const float* from = reinterpret_cast<const float*>(pool + (pg.read < 0 ? 0 : pg.read) * P.page_bytes) + (long)hh * D * D;
    float4 s[RPT];
#pragma unroll
    for (int m = 0; m < RPT; ++m)
        s[m] = pg.read < 0 ? make_float4(0.f, 0.f, 0.f, 0.f)
                           : __ldcs(reinterpret_cast<const float4*>(from + (long)(rg + 32 * m) * D + j0));
    const Tin* qh = q + head * D;
    const Tin* kh = k + head * D;
    float kr[RPT], qr[RPT];
#pragma unroll
    for (int m = 0; m < RPT; ++m) {
        kr[m] = Elem<Tin>::to_f(kh[rg + 32 * m]);
        qr[m] = Elem<Tin>::to_f(qh[rg + 32 * m]);
    }
    const float4 vv = load4(v + head * D + j0);

    __shared__ float4 red_r[8][8], red_p[8][8];
    __shared__ float sh_alpha, sh_c, sh_abar, sh_dec;
    if (warp == 0) {
        float lam = 0.f, c = 0.f;
#pragma unroll
        for (int i = lane; i < D; i += 32) {
            const float ki = Elem<Tin>::to_f(kh[i]);
            lam = fmaf(ki, ki, lam);
            c = fmaf(Elem<Tin>::to_f(qh[i]), ki, c);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            lam += __shfl_xor_sync(0xffffffffu, lam, off);
            c += __shfl_xor_sync(0xffffffffu, c, off);
        }
        if (lane == 0) {
            const float bt = Elem<Tin>::to_f(beta[head]);
            const float al = rule_alpha(rule, bt, lam), gh = g ? g[head] : 0.f;
            sh_alpha = al;
            sh_c = c;
            sh_abar = g ? rule_write_gate(rule, bt, lam, gh) : al;
            sh_dec = g ? expf(gh) : 1.f;
        }
    }
    float4 r = make_float4(0.f, 0.f, 0.f, 0.f), p = r;
#pragma unroll
    for (int m = 0; m < RPT; ++m) {
        r.x = fmaf(kr[m], s[m].x, r.x); r.y = fmaf(kr[m], s[m].y, r.y);
        r.z = fmaf(kr[m], s[m].z, r.z); r.w = fmaf(kr[m], s[m].w, r.w);
        p.x = fmaf(qr[m], s[m].x, p.x); p.y = fmaf(qr[m], s[m].y, p.y);
        p.z = fmaf(qr[m], s[m].z, p.z); p.w = fmaf(qr[m], s[m].w, p.w);
    }
#pragma unroll
    for (int off = 8; off < 32; off <<= 1) {
        r.x += __shfl_xor_sync(0xffffffffu, r.x, off); r.y += __shfl_xor_sync(0xffffffffu, r.y, off);
        r.z += __shfl_xor_sync(0xffffffffu, r.z, off); r.w += __shfl_xor_sync(0xffffffffu, r.w, off);
        p.x += __shfl_xor_sync(0xffffffffu, p.x, off); p.y += __shfl_xor_sync(0xffffffffu, p.y, off);
        p.z += __shfl_xor_sync(0xffffffffu, p.z, off); p.w += __shfl_xor_sync(0xffffffffu, p.w, off);
    }
    if (lane < 8) {
        red_r[warp][lane] = r;
        red_p[warp][lane] = p;
    }
    __syncthreads();
    r = red_r[0][cq];
    p = red_p[0][cq];
#pragma unroll
    for (int w = 1; w < 8; ++w) {
        const float4 a = red_r[w][cq], b = red_p[w][cq];
        r.x += a.x; r.y += a.y; r.z += a.z; r.w += a.w;
        p.x += b.x; p.y += b.y; p.z += b.z; p.w += b.w;
    }
    const float dec = sh_dec, da = sh_dec * sh_alpha, ab = sh_abar, c = sh_c;
    const float4 w = make_float4(fmaf(da, r.x, -ab * vv.x), fmaf(da, r.y, -ab * vv.y), fmaf(da, r.z, -ab * vv.z),
                                 fmaf(da, r.w, -ab * vv.w));
#pragma unroll
    for (int m = 0; m < RPT; ++m) {
        const float km = kr[m];
        float4 u = s[m];
        u.x = fmaf(-km, w.x, dec * u.x); u.y = fmaf(-km, w.y, dec * u.y);
        u.z = fmaf(-km, w.z, dec * u.z); u.w = fmaf(-km, w.w, dec * u.w);
        __stcs(reinterpret_cast<float4*>(to + (long)(rg + 32 * m) * D + j0), u);
    }
    if (rg == 0)
        store4(o + head * D + j0, make_float4(fmaf(-c, w.x, dec * p.x), fmaf(-c, w.y, dec * p.y),
                                              fmaf(-c, w.z, dec * p.z), fmaf(-c, w.w, dec * p.w)));
}

// The same step for many heads.  A head's state is contiguous in its page, so a producer warp moves
// 64 KiB jobs (one head of 128, four of 64) by bulk copies through a ring of three buffers, in and
// out, and looks the rows up ahead; eight warps keep a job's state in registers from the first
// product to the update and write it back in place.  256 rows of 16 heads of 128: 98 us, 5.6 TB/s read
// and written (85% of the measured copy rate; the same state updated in place without pages: 95.6).
constexpr int kJobFloats = 16384, kRing = 3, kWorkers = 256, kStreamThreads = kWorkers + 32;
constexpr uint64_t kWaitNs = 2000000000ull;

struct Job {
    int n, h0, heads;      // row, first head, heads; n < 0: no more
    bool zero;             // from a zero state
    long out;              // its place in the pool, in floats
};
template <typename Tin, int D>
struct StreamSmem {
    static constexpr int kHeads = kJobFloats / (D * D);
    static constexpr int kRow = kHeads * D * (int)sizeof(Tin);       // q, k or v of a job
    static constexpr int kRed = 8 * 32 * 16;                          // one sum of every warp
    static constexpr int kBytes = kRing * kJobFloats * 4 + kRing * 3 * kRow + 4 * kRed + kRing * (int)sizeof(Job) + 8 * 8;
};

// All but the last N of the thread's bulk stores have read their source.
template <int N>
__device__ __forceinline__ void wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }

// A row's pages as paged_row gives them, by one warp.
__device__ __forceinline__ RowPages paged_row_warp(const PagedRows& P, int N, int n) {
    const int lane = threadIdx.x & 31, slot = P.slots[n];
    if (slot == -1) return RowPages{false, -1, -1};
    const int src = P.source ? P.source[n] : slot;
    bool bad = false;
    for (int m = lane; m < n; m += 32) bad |= P.slots[m] == slot;
    if (src != slot && src != -1)
        for (int m = lane; m < N; m += 32) bad |= P.slots[m] == src;
    RowPages r = row_pages(P, slot, src, &bad);
    r.active = !__any_sync(0xffffffffu, bad);
    if (!r.active && lane == 0) atomicOr(P.err, kPagesBadSlot);
    return r;
}

template <typename Tin, int D>
__global__ void __launch_bounds__(kStreamThreads, 1) decode_stream_kernel(const Tin* q, const Tin* k,
                                                                          const Tin* v,
                                                                          const Tin* beta,
                                                                          const float* g, char* pool,
                                                                          Tin* o, int N, int H, int rule,
                                                                          PagedRows P) {
    using M = StreamSmem<Tin, D>;
    extern __shared__ __align__(128) char smem[];
    float* ring = reinterpret_cast<float*>(smem);
    char* rows = smem + kRing * kJobFloats * 4;                                      // [ring][q, k, v]
    float4* red = reinterpret_cast<float4*>(rows + kRing * 3 * M::kRow);             // [2][r, p][warp][32]
    Job* jobs = reinterpret_cast<Job*>(red + 4 * 8 * 32);
    uint64_t* full = reinterpret_cast<uint64_t*>(jobs + kRing);
    uint64_t* done = full + kRing;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kRing; ++i) mbar_init(full + i, 1), mbar_init(done + i, kWorkers / 32);
        fence_mbar_init();
    }
    __syncthreads();
    after_previous();

    if (warp == kWorkers / 32) {          // the producer
        const int per_row = (H + M::kHeads - 1) / M::kHeads;
        const long total = (long)N * per_row;
        long job = total * blockIdx.x / gridDim.x;
        const long end = total * (blockIdx.x + 1) / gridDim.x;
        RowPages pg{false, -1, -1};
        int row = -1, sent = 0;
        bool ok = true;
        // Job j is done: its state leaves the buffer in quarters, and as soon as a quarter has been read
        // the next job's may take its place (`load(quarter)`).
        auto write_back = [&](int j, auto load) {
            const int b = j % kRing;
            ok = ok && __all_sync(0xffffffffu, mbar_wait(done + b, j / kRing & 1, kWaitNs));
            if (ok && lane == 0) {
                const int quarter = jobs[b].heads * D * D / 4;
                float* to = reinterpret_cast<float*>(pool) + jobs[b].out;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    bulk_store(to + i * quarter, ring + b * kJobFloats + i * quarter, quarter * 4);
                load(b);
            }
            __syncwarp();
        };
        for (; job < end && ok; ++job) {
            const int n = (int)(job / per_row), h0 = (int)(job % per_row) * M::kHeads, heads = min(M::kHeads, H - h0);
            if (n != row) {
                pg = paged_row_warp(P, N, n);
                row = n;
            }
            if (!pg.active) continue;
            const int b = sent % kRing, bytes = heads * D * (int)sizeof(Tin), quarter = heads * D * D;      // in bytes
            const long at = ((long)n * H + h0) * D;
            const char* from = pool + (pg.read < 0 ? 0 : pg.read) * (long)P.page_bytes + (long)h0 * D * D * 4;
            char* to = reinterpret_cast<char*>(ring + b * kJobFloats);
            auto begin = [&]() {
                jobs[b] = Job{n, h0, heads, pg.read < 0, pg.write * (long)(P.page_bytes / 4) + (long)h0 * D * D};
                mbar_arrive_expect_tx(full + b, 3 * bytes + (pg.read < 0 ? 0 : 4 * quarter));
                bulk_load(rows + (b * 3 + 0) * M::kRow, q + at, bytes, full + b);
                bulk_load(rows + (b * 3 + 1) * M::kRow, k + at, bytes, full + b);
                bulk_load(rows + (b * 3 + 2) * M::kRow, v + at, bytes, full + b);
            };
            auto load = [&](int i) {
                if (pg.read >= 0) bulk_load(to + i * quarter, from + i * quarter, quarter, full + b);
            };
            if (sent < kRing) {
                if (lane == 0) {
                    begin();
                    for (int i = 0; i < 4; ++i) load(i);
                }
                __syncwarp();
            } else {
                // A last job of fewer heads is shorter: then its quarters are not where the next one's go.  A
                // job from a zero state loads none, and the workers may write theirs as soon as it begins.
                const bool whole = jobs[b].heads != heads || pg.read < 0;
                write_back(sent - kRing, [&](int) {
                    if (whole) wait_read<0>();
                    begin();
                    wait_read<3>();
                    load(0);
                    wait_read<2>();
                    load(1);
                    wait_read<1>();
                    load(2);
                    wait_read<0>();
                    load(3);
                });
            }
            ++sent;
        }
        if (sent >= kRing) write_back(sent - kRing, [](int) {});
        if (ok && lane == 0) {            // the end, in the next buffer
            jobs[sent % kRing].n = -1;
            mbar_arrive(full + sent % kRing);
        }
        for (int j = max(0, sent - kRing + 1); j < sent; ++j) write_back(j, [](int) {});
        if (!ok && lane == 0) atomicOr(P.err, kDevTimeout);
        tma_store_wait_all();
        return;
    }

    constexpr int kQuads = D / 4, kSide = 32 / kQuads;                // rows that a warp reads at once
    constexpr int kWarpsPerHead = 8 / M::kHeads, kRows = D / (kWarpsPerHead * kSide);      // rows of a thread: 16
    const int hw = warp / kWarpsPerHead, part = warp % kWarpsPerHead;
    const int quad = lane % kQuads, row0 = (part * kSide + lane / kQuads) * kRows;
    for (int j = 0;; ++j) {
        const int b = j % kRing;
        if (!mbar_wait(full + b, j / kRing & 1, kWaitNs)) {
            if (threadIdx.x == 0) atomicOr(P.err, kDevTimeout);
            break;
        }
        const Job job = jobs[b];
        if (job.n < 0) break;
        const bool on = hw < job.heads;
        const long head = (long)job.n * H + job.h0 + hw;
        float* S = ring + b * kJobFloats + hw * D * D;
        const Tin* qs = reinterpret_cast<const Tin*>(rows + (b * 3 + 0) * M::kRow) + hw * D;
        const Tin* ks = reinterpret_cast<const Tin*>(rows + (b * 3 + 1) * M::kRow) + hw * D;
        const Tin* vs = reinterpret_cast<const Tin*>(rows + (b * 3 + 2) * M::kRow) + hw * D;
        float4* red_r = red + (j & 1) * 2 * 8 * 32;
        float4* red_p = red_r + 8 * 32;
        float4 s[kRows], r = make_float4(0.f, 0.f, 0.f, 0.f), p = r;
        float kr[kRows], alpha = 0.f, c = 0.f, abar = 0.f, dec = 1.f;
        if (on) {
            const float bt = Elem<Tin>::to_f(beta[head]), gh = g ? g[head] : 0.f;
            float lam = 0.f;
#pragma unroll
            for (int i = lane; i < D; i += 32) {
                const float ki = Elem<Tin>::to_f(ks[i]);
                lam = fmaf(ki, ki, lam);
                c = fmaf(Elem<Tin>::to_f(qs[i]), ki, c);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
                lam += __shfl_xor_sync(0xffffffffu, lam, off);
                c += __shfl_xor_sync(0xffffffffu, c, off);
            }
            alpha = rule_alpha(rule, bt, lam);
            abar = g ? rule_write_gate(rule, bt, lam, gh) : alpha;
            dec = g ? expf(gh) : 1.f;
#pragma unroll
            for (int m = 0; m < kRows; ++m) {
                s[m] = job.zero ? make_float4(0.f, 0.f, 0.f, 0.f) : *reinterpret_cast<const float4*>(S + (row0 + m) * D + quad * 4);
                kr[m] = Elem<Tin>::to_f(ks[row0 + m]);
                const float qm = Elem<Tin>::to_f(qs[row0 + m]);
                r.x = fmaf(kr[m], s[m].x, r.x); r.y = fmaf(kr[m], s[m].y, r.y);
                r.z = fmaf(kr[m], s[m].z, r.z); r.w = fmaf(kr[m], s[m].w, r.w);
                p.x = fmaf(qm, s[m].x, p.x); p.y = fmaf(qm, s[m].y, p.y);
                p.z = fmaf(qm, s[m].z, p.z); p.w = fmaf(qm, s[m].w, p.w);
            }
        }
        red_r[warp * 32 + lane] = r;
        red_p[warp * 32 + lane] = p;
        bar_sync(1, kWorkers);
        if (on) {
            r = p = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kWarpsPerHead * kSide; ++i) {
                const int at = (hw * kWarpsPerHead + i / kSide) * 32 + (i % kSide) * kQuads + quad;
                const float4 a = red_r[at], e = red_p[at];
                r.x += a.x; r.y += a.y; r.z += a.z; r.w += a.w;
                p.x += e.x; p.y += e.y; p.z += e.z; p.w += e.w;
            }
            const float4 vv = load4(vs + quad * 4);
            const float da = dec * alpha;
            const float4 w = make_float4(fmaf(da, r.x, -abar * vv.x), fmaf(da, r.y, -abar * vv.y), fmaf(da, r.z, -abar * vv.z),
                                         fmaf(da, r.w, -abar * vv.w));
#pragma unroll
            for (int m = 0; m < kRows; ++m) {
                float4 u = s[m];
                u.x = fmaf(-kr[m], w.x, dec * u.x); u.y = fmaf(-kr[m], w.y, dec * u.y);
                u.z = fmaf(-kr[m], w.z, dec * u.z); u.w = fmaf(-kr[m], w.w, dec * u.w);
                *reinterpret_cast<float4*>(S + (row0 + m) * D + quad * 4) = u;
            }
            if (part == 0 && lane < kQuads)
                store4(o + head * D + quad * 4, make_float4(fmaf(-c, w.x, dec * p.x), fmaf(-c, w.y, dec * p.y),
                                                            fmaf(-c, w.z, dec * p.z), fmaf(-c, w.w, dec * p.w)));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(done + b);
    }
}

template <typename Tin, int D>
cudaError_t launch_t(const void* q, const void* k, const void* v, const void* beta, const float* g, float* pool,
                     void* o, int N, int H, int rule, const PagedRows& paged, cudaStream_t stream) {
    using M = StreamSmem<Tin, D>;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const long jobs = (long)N * ((H + M::kHeads - 1) / M::kHeads);
    // Slices against the stream, fp32, device us.  d = 128: 304 jobs 11.8 and 12.8, 592 19.4 and 17.7,
    // 4096 113 and 100; d = 64, whose slices are half as high: 76 jobs 5.6 and 7.6, 148 8.8 and 8.6,
    // 296 14.1 and 11.6, 1024 40.8 and 28.3.
    if (jobs >= (D == 64 ? 1 : 3) * sms) {
        static std::atomic<uint64_t> limit{0};
        if ((e = set_smem_limit_once(decode_stream_kernel<Tin, D>, M::kBytes, limit)) != cudaSuccess) return e;
        return launch_after(decode_stream_kernel<Tin, D>, sms, kStreamThreads, M::kBytes, stream, (const Tin*)q,
                            (const Tin*)k, (const Tin*)v, (const Tin*)beta, g, reinterpret_cast<char*>(pool),
                            (Tin*)o, N, H, rule, paged);
    }
    const long blocks = (long)N * H * (D / kCols);
    return launch_after(decode_paged_kernel<Tin, D>, (unsigned)blocks, kThreads, 0, stream, (const Tin*)q,
                        (const Tin*)k, (const Tin*)v, (const Tin*)beta, g, reinterpret_cast<char*>(pool), (Tin*)o, N,
                        H, rule, paged);
}
}  // namespace

cudaError_t launch_decode_paged(const void* q, const void* k, const void* v, const void* beta, const float* g,
                                float* pool, void* o, int N, int H, int D, bool bf16, int rule,
                                const PagedRows& paged, cudaStream_t stream) {
    if (bf16)
        return D == 128 ? launch_t<__nv_bfloat16, 128>(q, k, v, beta, g, pool, o, N, H, rule, paged, stream)
                        : launch_t<__nv_bfloat16, 64>(q, k, v, beta, g, pool, o, N, H, rule, paged, stream);
    return D == 128 ? launch_t<float, 128>(q, k, v, beta, g, pool, o, N, H, rule, paged, stream)
                    : launch_t<float, 64>(q, k, v, beta, g, pool, o, N, H, rule, paged, stream);
}

}  // namespace efla
