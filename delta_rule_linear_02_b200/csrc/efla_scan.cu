// efla_scan.cu -- the per-channel gated linear recurrence: forward, backward, one token.
//
// The recurrence is affine in the state: over any run of tokens h_out = A h_in + B, and runs
// compose.  A tile is 32 tokens x 128 channels (a "strip").  A cluster of blocks takes one strip
// along time: in each turn its blocks hold consecutive tiles, and
//   1. the eight compute warps reduce four tokens each (a lane holds four channels) to (A, B);
//   2. the two chain warps (a thread holds two channels) fold these to the tile's (A, B), write it
//      into the shared memory of every block of the cluster, and fold what all blocks sent onto
//      the state the turn began with: the state entering the block's own tile, the one entering
//      each of its runs, and the one that the next turn begins with, which is thus known to every
//      block without another exchange;
//   3. the compute warps continue their runs from there and write the outputs.
// Inputs are staged by bulk copies some turns ahead and read from memory once.  Everything is
// folded in token order, so the results are the same bits on every run.
#include "efla_kernels.h"
#include "efla_pages.cuh"
#include "efla_scan.cuh"
#include "sm100.cuh"

namespace efla {
using namespace sm100;
namespace {

struct P4 {          // four channels
    float2 lo, hi;
};
__device__ __forceinline__ P4 all4(float x) { return P4{both(x), both(x)}; }
__device__ __forceinline__ P4 fma4(const P4& a, const P4& b, const P4& c) {
    return P4{fma2(a.lo, b.lo, c.lo), fma2(a.hi, b.hi, c.hi)};
}
__device__ __forceinline__ P4 mul4(const P4& a, const P4& b) { return P4{mul2(a.lo, b.lo), mul2(a.hi, b.hi)}; }
__device__ __forceinline__ P4 add4(const P4& a, const P4& b) { return P4{add2(a.lo, b.lo), add2(a.hi, b.hi)}; }
template <typename T>
__device__ __forceinline__ P4 ld4(const T* p) {
    const float4 f = load4(p);
    return P4{make_float2(f.x, f.y), make_float2(f.z, f.w)};
}
template <typename T>
__device__ __forceinline__ void st4(T* p, const P4& v) {
    store4(p, make_float4(v.lo.x, v.lo.y, v.hi.x, v.hi.y));
}

constexpr int kTok = kScanChunk, kWarps = 8, kRun = kTok / kWarps, kCh = 128;
constexpr int kComputeThreads = kWarps * 32, kChainThreads = kCh / 2, kThreads = kComputeThreads + kChainThreads;
constexpr int kCluster = 16;       // most blocks of a cluster
constexpr int kMarks = 8;          // chunks whose marks are kept
constexpr uint64_t kWaitNs = 2000000000ull;

// How lanes map to (stream, channel): heads of d channels with 32 % (d / 4) == 0 are packed
// side by side into a strip; other widths up to 128 take a strip each, wider ones several.
struct Strips {
    int dv;          // vectors of four channels per head
    int heads;       // heads per strip
    int per_head;    // strips per head
    int count;       // strips
    __host__ __device__ Strips(long Z, int d) {
        dv = d / 4;
        heads = dv <= 32 && 32 % dv == 0 ? 32 / dv : 1;
        per_head = (dv + 31) / 32;
        count = (int)(heads > 1 ? (Z + heads - 1) / heads : Z * per_head);
    }
};

// What a lane holds of any strip.
struct Lane {
    int c, smem, row;     // channel within the head or its part; offset of token 0 in a staged tile; elements between tokens
    int p, heads, per_head, d;
    long Z;
    __device__ __forceinline__ Lane(const Strips& S, long Z_, int d_, int lane)
        : heads(S.heads), per_head(S.per_head), d(d_), Z(Z_) {
        p = S.heads > 1 ? lane / S.dv : 0;
        c = S.heads > 1 ? (lane % S.dv) * 4 : lane * 4;
        row = S.per_head > 1 ? kCh : d_;
        smem = S.heads > 1 ? p * kTok * d_ + c : c < row ? c : 0;       // off lanes: something that is there
    }
};
struct Spot {
    long z;
    int c;
    bool on;
};
__device__ __forceinline__ Spot spot_of(const Lane& L, int strip) {
    Spot s;
    if (L.per_head == 1) {
        s.z = (long)strip * L.heads + L.p;
        s.c = L.c;
    } else {
        s.z = strip / L.per_head;
        s.c = (strip % L.per_head) * kCh + L.c;
    }
    s.on = s.z < L.Z && s.c < L.d;
    return s;
}

// Stage one tensor's tile (one warp calls it; the barrier already expects the bytes).  A strip
// that holds whole heads is `rows` x d contiguous elements per head; a part of a wide head is
// copied token by token.  All addresses and sizes are multiples of 16 bytes, because d elements are.
template <typename T>
__device__ __forceinline__ void stage(T* dst, const T* src, const Strips& S, long Z, int Ttot, int d, int strip, int t0,
                                      int rows, uint64_t* bar) {
    const int lane = threadIdx.x & 31;
    if (S.per_head == 1) {
        const long z = (long)strip * S.heads + lane;
        if (lane < S.heads && z < Z)
            bulk_load(dst + lane * kTok * d, src + (z * Ttot + t0) * d, rows * d * (int)sizeof(T), bar);
    } else {
        const long z = strip / S.per_head;
        const int c0 = (strip % S.per_head) * kCh;
        for (int t = lane; t < rows; t += 32)
            bulk_load(dst + t * kCh, src + (z * Ttot + t0 + t) * d + c0, min(kCh, d - c0) * (int)sizeof(T), bar);
    }
}
__device__ __forceinline__ int strip_channels(const Strips& S, long Z, int d, int strip) {
    if (S.heads > 1) return (int)min((long)S.heads, Z - (long)strip * S.heads) * d;
    return S.per_head == 1 ? d : min(kCh, d - (strip % S.per_head) * kCh);
}

// The packed sequence that holds token t: the largest n with cu[n] <= t.
__device__ __forceinline__ int seq_of(const ScanArgs& P, int t) {
    if (!P.cu) return 0;
    int lo = 0, hi = P.nseq;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (P.cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Which of a chunk's tokens begin or end a sequence (bit l: token l).  One warp calls it.
__device__ __forceinline__ uint2 chunk_marks(const ScanArgs& P, int chunk) {
    const int t0 = chunk * kTok;
    if (!P.cu) return make_uint2(chunk == 0 ? 1u : 0u, P.T - t0 <= kTok ? 1u << (P.T - t0 - 1) : 0u);
    static_assert(kTok == 32, "one lane per token");
    const int t = t0 + (threadIdx.x & 31), n = t < P.T ? seq_of(P, t) : 0;
    return make_uint2(__ballot_sync(0xffffffffu, t < P.T && P.cu[n] == t),
                      __ballot_sync(0xffffffffu, t < P.T && P.cu[n + 1] == t + 1));
}
__device__ __forceinline__ uint32_t run_bits(uint32_t marks, int warp) {
    return marks >> (warp * kRun) & ((1u << kRun) - 1u);
}

// Sequences without tokens pass their states through.
__device__ __forceinline__ void pass_empty(const ScanArgs& P, const float* in, float* out) {
    if (!P.cu || !out) return;
    for (int n = blockIdx.x; n < P.nseq; n += gridDim.x)
        if (P.cu[n] == P.cu[n + 1])
            for (long i = threadIdx.x; i < P.Z * P.d; i += kThreads)
                out[n * P.Z * P.d + i] = in ? in[n * P.Z * P.d + i] : 0.f;
}

// A of a run with a sequence's begin in it: what came before does not matter, not even a NaN.
// (No product of decays is -0.)  A cut is one for all channels.
constexpr float kCut = -0.0f;
__device__ __forceinline__ float2 run_on(float2 A, float2 h, float2 B) {
    return __float_as_uint(A.x) == 0x80000000u ? B : fma2(A, h, B);
}
__device__ __forceinline__ float2 ld2(const float* p) { return *reinterpret_cast<const float2*>(p); }

// The state entering each run takes the place of its B.
template <bool kReverse>
__device__ __forceinline__ void enter_runs(const float* runA, float* runB, float2 h) {
    float2 A[kWarps], B[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) A[w] = ld2(runA + w * kCh), B[w] = ld2(runB + w * kCh);
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        const int w = kReverse ? kWarps - 1 - i : i;
        *reinterpret_cast<float2*>(runB + w * kCh) = h;
        h = run_on(A[w], h, B[w]);
    }
}

// ---------------------------------------------------------------- the cluster
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t in_block(uint32_t smem_addr, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr), "r"(rank));
    return a;
}
// 16 bytes into a block's shared memory, counted there by a barrier
__device__ __forceinline__ void send(uint32_t to, uint32_t bar, float2 A, float2 B) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
                 "r"(__float_as_uint(A.x)), "r"(__float_as_uint(A.y)), "r"(__float_as_uint(B.x)),
                 "r"(__float_as_uint(B.y)), "r"(bar)
                 : "memory");
}

// One warp's arrival (its earlier shared-memory accesses are done).
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
__device__ __forceinline__ void wait_or_give_up(uint64_t* bar, int parity, bool* dead, uint32_t* err) {
    if (!mbar_wait(bar, parity, *dead ? 0 : kWaitNs)) {
        if (!*dead && (threadIdx.x & 31) == 0) atomicOr(err, kDevTimeout);
        *dead = true;
    }
}

// A chain thread's part of one turn: the tile's (A, B) from its runs (kReverse: last run first; no
// tile: nothing changes), the exchange, the state entering the tile; `carry` goes from this turn's
// first state to the next one's.  sent: [2][rank][64] x {A, B of two channels}.
template <bool kReverse>
__device__ __forceinline__ float2 chain_turn(const float* runA, const float* runB, bool tile, int blocks, uint32_t rank,
                                             int n, float4* sent, uint64_t* got, float2* carry, bool* dead,
                                             uint32_t* err) {
    float2 A = both(1.f), B = both(0.f);
    if (tile) {
        bool cut = false;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            const int w = kReverse ? kWarps - 1 - i : i;
            const float2 a = ld2(runA + w * kCh);
            cut |= __float_as_uint(a.x) == 0x80000000u;
            B = run_on(a, B, ld2(runB + w * kCh));
            A = mul2(A, a);
        }
        if (cut) A = both(kCut);
    }
    float2 h = *carry;
    if (blocks == 1) {
        *carry = run_on(A, h, B);
        return h;
    }
    const int k = threadIdx.x - kComputeThreads, buf = n & 1;
    const uint32_t to = smem_u32(sent + (buf * blocks + rank) * kChainThreads + k), bar = smem_u32(got + buf);
    for (int q = 0; q < blocks; ++q) send(in_block(to, q), in_block(bar, q), A, B);
    if (k == 0) mbar_arrive_expect_tx(got + buf, blocks * kChainThreads * 16);
    wait_or_give_up(got + buf, n >> 1 & 1, dead, err);
    float2 mine = h;
    const float4* all = sent + buf * blocks * kChainThreads + k;
    for (int q = 0; q < blocks; ++q) {
        const float4 v = all[q * kChainThreads];
        if (q == (int)rank) mine = h;
        h = run_on(make_float2(v.x, v.y), h, make_float2(v.z, v.w));
    }
    *carry = h;
    return mine;
}

// The gates of one token: of a channel each, or one for all.
template <bool kShared>
struct Gate {
    P4 v[kRun];
    __device__ __forceinline__ P4 at(int i) const { return v[i]; }
    __device__ __forceinline__ void set(int i, const P4& x) { v[i] = x; }
};
template <>
struct Gate<true> {
    float v[kRun];
    __device__ __forceinline__ P4 at(int i) const { return all4(v[i]); }
    __device__ __forceinline__ void set(int i, const P4& x) { v[i] = x.lo.x; }
};
template <bool kShared, bool kSlope>
__device__ __forceinline__ void token_gates(int rule, const float* gt, float gs, P4* a, P4* w, P4* dw) {
    if constexpr (kShared) {
        float2 a2, w2, d2 = both(0.f);
        scan_gates2<kSlope>(rule, both(gs), &a2, &w2, &d2);
        *a = all4(a2.x);
        *w = all4(w2.x);
        *dw = all4(d2.x);
    } else {
        const P4 g = ld4(gt);
        scan_gates2<kSlope>(rule, g.lo, &a->lo, &w->lo, &dw->lo);
        scan_gates2<kSlope>(rule, g.hi, &a->hi, &w->hi, &dw->hi);
    }
}

template <typename Tin, bool kShared>
struct FwdSmem {
    static constexpr int kX = kTok * kCh * sizeof(Tin), kG = kShared ? 0 : kTok * kCh * 4;
    static constexpr int kStage = kX + kG, kStages = 2;
    static constexpr int kRuns = kWarps * kCh;                  // floats of one value of all runs
    static constexpr int bytes(int blocks) { return kStages * kStage + 2 * kRuns * 4 + 2 * blocks * kChainThreads * 16 + 256; }
};

template <typename Tin, bool kShared>
__global__ void __launch_bounds__(kThreads, 3) scan_fwd_kernel(ScanArgs P, int blocks, int steps) {
    using M = FwdSmem<Tin, kShared>;
    extern __shared__ __align__(128) char smem[];
    float* runs = reinterpret_cast<float*>(smem + M::kStages * M::kStage);     // [A, B (then: entering)][warp][128]
    float4* sent = reinterpret_cast<float4*>(runs + 2 * M::kRuns);
    uint64_t* full = reinterpret_cast<uint64_t*>(sent + 2 * blocks * kChainThreads);
    uint64_t* ready = full + M::kStages;      // the tile's (A, B) of all runs are there
    uint64_t* entered = ready + 1;            // the states entering them are
    uint64_t* got = entered + 1;              // [2] all blocks' (A, B) are
    uint2* marks = reinterpret_cast<uint2*>(got + 2);
    const Strips S(P.Z, P.d);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = blocks > 1 ? cluster_rank() : 0;
    const int strip = blockIdx.x / blocks, turns = (steps + blocks - 1) / blocks;
    const Tin* x = static_cast<const Tin*>(P.x);
    Tin* o = static_cast<Tin*>(P.o);
    if (threadIdx.x == 0) {
        for (int i = 0; i < M::kStages; ++i) mbar_init(full + i, 1);
        mbar_init(ready, kWarps);
        mbar_init(entered, kChainThreads / 32);
        mbar_init(got, 1);
        mbar_init(got + 1, 1);
        fence_mbar_init();
    }
    __syncthreads();
    auto prefetch = [&](int n) {      // by the last warp
        const int chunk = n * blocks + rank;
        if (chunk >= steps) return;
        const int st = n % M::kStages, t0 = chunk * kTok, rows = min(kTok, P.T - t0);
        const uint2 m = chunk_marks(P, chunk);
        if (lane == 0) {
            marks[n % kMarks] = m;
            mbar_arrive_expect_tx(full + st, rows * strip_channels(S, P.Z, P.d, strip) * (int)(sizeof(Tin) + (kShared ? 0 : 4)));
        }
        __syncwarp();
        char* dst = smem + st * M::kStage;
        stage(reinterpret_cast<Tin*>(dst), x, S, P.Z, P.T, P.d, strip, t0, rows, full + st);
        if (!kShared) stage(reinterpret_cast<float*>(dst + M::kX), P.g, S, P.Z, P.T, P.d, strip, t0, rows, full + st);
    };
    if (warp == kThreads / 32 - 1)
        for (int i = 0; i < M::kStages; ++i) prefetch(i);
    pass_empty(P, P.S0, P.S_T);
    if (blocks > 1) cluster_sync();       // every block's barriers are set up
    bool dead = false;

    if (warp >= kWarps) {                 // the chain
        const int k = (threadIdx.x - kComputeThreads) * 2;
        float2 carry = both(0.f);
        for (int n = 0; n < turns; ++n) {
            const int chunk = n * blocks + rank;
            const bool tile = chunk < steps;
            if (tile) {
                wait_or_give_up(ready, n & 1, &dead, P.err);
                if (warp == kThreads / 32 - 1) prefetch(n + M::kStages);      // the stage has been read
            }
            const float2 h = chain_turn<false>(runs + k, runs + M::kRuns + k, tile, blocks, rank, n, sent, got, &carry,
                                               &dead, P.err);
            if (tile) {
                enter_runs<false>(runs + k, runs + M::kRuns + k, h);
                warp_arrive(entered);
                if (P.E) *reinterpret_cast<float2*>(P.E + ((size_t)chunk * S.count + strip) * kCh + k) = h;
            }
        }
    } else {
        const Lane lanes(S, P.Z, P.d, lane);
        const Spot L = spot_of(lanes, strip);
        const int mine = lanes.smem + warp * kRun * lanes.row;
        float* run = runs + warp * kCh + lane * 4;
        for (int n = 0; n < turns; ++n) {
            const int chunk = n * blocks + rank;
            if (chunk >= steps) break;
            const int tw = chunk * kTok + warp * kRun, st = n % M::kStages;
            float gs[kRun];
            if (kShared) {
#pragma unroll
                for (int i = 0; i < kRun; ++i) gs[i] = L.on && tw + i < P.T ? P.g[L.z * P.T + tw + i] : 0.f;
            }
            wait_or_give_up(full + st, n / M::kStages & 1, &dead, P.err);
            const uint2 m = marks[n % kMarks];
            const uint32_t first = run_bits(m.x, warp);
            const Tin* xs = reinterpret_cast<const Tin*>(smem + st * M::kStage) + mine;
            const float* gt = reinterpret_cast<const float*>(smem + st * M::kStage + M::kX) + mine;
            // 1. the run's tokens as h = a h' + b, and the run's (A, B)
            Gate<kShared> a;
            P4 b[kRun];
#pragma unroll
            for (int i = 0; i < kRun; ++i) {
                P4 a1, w, dw;
                token_gates<kShared, false>(P.rule, gt + i * lanes.row, gs[i], &a1, &w, &dw);
                a.set(i, a1);
                b[i] = mul4(w, ld4(xs + i * lanes.row));
            }
            if (tw + kRun > P.T) {            // behind the end: tokens that change nothing
#pragma unroll
                for (int i = 0; i < kRun; ++i)
                    if (tw + i >= P.T) {
                        a.set(i, all4(1.f));
                        b[i] = all4(0.f);
                    }
            }
            for (uint32_t bits = first; bits; bits &= bits - 1) {     // a sequence begins: its own state enters
                const int from = __ffs(bits) - 1;
                const P4 s0 = P.S0 && L.on ? ld4(P.S0 + ((long)seq_of(P, tw + from) * P.Z + L.z) * P.d + L.c) : all4(0.f);
#pragma unroll
                for (int i = 0; i < kRun; ++i)
                    if (i == from) {
                        b[i] = fma4(a.at(i), s0, b[i]);
                        a.set(i, all4(0.f));
                    }
            }
            P4 ra = all4(1.f), rb = all4(0.f);
#pragma unroll
            for (int i = 0; i < kRun; ++i) {
                if (first >> i & 1u) rb = all4(0.f);
                ra = mul4(ra, a.at(i));
                rb = fma4(a.at(i), rb, b[i]);
            }
            if (first) ra = all4(kCut);
            st4(run, ra);
            st4(run + M::kRuns, rb);
            warp_arrive(ready);
            // 3. the outputs
            wait_or_give_up(entered, n & 1, &dead, P.err);
            P4 h = ld4(run + M::kRuns);
            const uint32_t last = P.S_T ? run_bits(m.y, warp) : 0u;
            const int live = L.on ? P.T - tw : 0;
            if (!o && !last) continue;
            Tin* out = o + (L.z * P.T + tw) * P.d + L.c;
#pragma unroll
            for (int i = 0; i < kRun; ++i) {
                if (first >> i & 1u) h = all4(0.f);          // its state is in b
                h = fma4(a.at(i), h, b[i]);
                if (o && i < live) st4(out + i * P.d, h);
                if (last >> i & 1u) {                        // a sequence ends
                    if (L.on) st4(P.S_T + ((long)seq_of(P, tw + i) * P.Z + L.z) * P.d + L.c, h);
                }
            }
        }
    }
    if (blocks > 1) cluster_sync();       // no block leaves while another may still send to it
}

// The reverse pass.  c = e^{g_t} G_t flows from token t into t - 1 (dS_T into a sequence's last
// token), G_t = dO_t + c: affine again, c_out = A c_in + R over a run, and the tiles are taken
// from the last to the first.  A tile's own states are put together again from the state that
// the forward kept for it, so no state but one of 32 tokens is ever stored.
template <typename Tin, bool kShared>
struct BwdSmem {
    static constexpr int kX = kTok * kCh * sizeof(Tin), kG = kShared ? 0 : kTok * kCh * 4;
    static constexpr int kStage = 2 * kX + kG, kStages = 2;
    static constexpr int kRuns = kWarps * kCh;
    static constexpr int bytes(int blocks) { return kStages * kStage + 4 * kRuns * 4 + 2 * blocks * kChainThreads * 16 + 256; }
};

template <typename Tin, bool kShared>
__global__ void __launch_bounds__(kThreads, 2) scan_bwd_kernel(ScanArgs P, const float* states, float* parts, int blocks,
                                                               int steps) {
    using M = BwdSmem<Tin, kShared>;
    extern __shared__ __align__(128) char smem[];
    // [A, B (then: the state entering), reverse A, R (then: the flow entering)][warp][128]
    float* runs = reinterpret_cast<float*>(smem + M::kStages * M::kStage);
    float4* sent = reinterpret_cast<float4*>(runs + 4 * M::kRuns);
    uint64_t* full = reinterpret_cast<uint64_t*>(sent + 2 * blocks * kChainThreads);
    uint64_t* spent = full + M::kStages;      // a stage has been read to its end
    uint64_t* ready = spent + M::kStages;
    uint64_t* entered = ready + 1;
    uint64_t* got = entered + 1;
    uint2* marks = reinterpret_cast<uint2*>(got + 2);
    const Strips S(P.Z, P.d);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = blocks > 1 ? cluster_rank() : 0;
    const int strip = blockIdx.x / blocks, turns = (steps + blocks - 1) / blocks;
    const Tin* x = static_cast<const Tin*>(P.x);
    const Tin* dO = static_cast<const Tin*>(P.dO);
    if (threadIdx.x == 0) {
        for (int i = 0; i < M::kStages; ++i) mbar_init(full + i, 1), mbar_init(spent + i, kWarps);
        mbar_init(ready, kWarps);
        mbar_init(entered, kChainThreads / 32);
        mbar_init(got, 1);
        mbar_init(got + 1, 1);
        fence_mbar_init();
    }
    __syncthreads();
    auto prefetch = [&](int n) {
        const int chunk = steps - 1 - (n * blocks + (int)rank);
        if (chunk < 0) return;
        const int st = n % M::kStages, t0 = chunk * kTok, rows = min(kTok, P.T - t0);
        const uint2 m = chunk_marks(P, chunk);
        if (lane == 0) {
            marks[n % kMarks] = m;
            mbar_arrive_expect_tx(full + st,
                                  rows * strip_channels(S, P.Z, P.d, strip) * (int)(2 * sizeof(Tin) + (kShared ? 0 : 4)));
        }
        __syncwarp();
        char* dst = smem + st * M::kStage;
        stage(reinterpret_cast<Tin*>(dst), x, S, P.Z, P.T, P.d, strip, t0, rows, full + st);
        stage(reinterpret_cast<Tin*>(dst + M::kX), dO, S, P.Z, P.T, P.d, strip, t0, rows, full + st);
        if (!kShared) stage(reinterpret_cast<float*>(dst + 2 * M::kX), P.g, S, P.Z, P.T, P.d, strip, t0, rows, full + st);
    };
    if (warp == kThreads / 32 - 1)
        for (int i = 0; i < M::kStages; ++i) prefetch(i);
    pass_empty(P, P.dST, P.dS0);
    if (blocks > 1) cluster_sync();
    bool dead = false;

    if (warp >= kWarps) {             // the chain
        const int k = (threadIdx.x - kComputeThreads) * 2;
        float2 carry = both(0.f);
        for (int n = 0; n < turns; ++n) {
            const int chunk = steps - 1 - (n * blocks + (int)rank);
            const bool tile = chunk >= 0;
            float2 h = both(0.f);
            if (tile) {
                if (chunk > 0) h = ld2(states + ((size_t)chunk * S.count + strip) * kCh + k);
                wait_or_give_up(ready, n & 1, &dead, P.err);
            }
            const float2 c = chain_turn<true>(runs + 2 * M::kRuns + k, runs + 3 * M::kRuns + k, tile, blocks, rank, n, sent,
                                              got, &carry, &dead, P.err);
            if (tile) {
                enter_runs<true>(runs + 2 * M::kRuns + k, runs + 3 * M::kRuns + k, c);
                enter_runs<false>(runs + k, runs + M::kRuns + k, h);
                warp_arrive(entered);
                if (warp == kThreads / 32 - 1 && chunk - M::kStages * blocks >= 0) {
                    wait_or_give_up(spent + n % M::kStages, n / M::kStages & 1, &dead, P.err);
                    prefetch(n + M::kStages);
                }
            }
        }
    } else {
        const Lane lanes(S, P.Z, P.d, lane);
        const Spot L = spot_of(lanes, strip);
        const int mine = lanes.smem + warp * kRun * lanes.row;
        for (int n = 0; n < turns; ++n) {
            const int chunk = steps - 1 - (n * blocks + (int)rank);
            if (chunk < 0) break;
            const int tw = chunk * kTok + warp * kRun, st = n % M::kStages;
            const bool ragged = tw + kRun > P.T;
            float gs[kRun];
            if (kShared) {
    #pragma unroll
                for (int i = 0; i < kRun; ++i) gs[i] = L.on && tw + i < P.T ? P.g[L.z * P.T + tw + i] : 0.f;
            }
            wait_or_give_up(full + st, n / M::kStages & 1, &dead, P.err);
            const uint2 m = marks[n % kMarks];
            const uint32_t first = run_bits(m.x, warp), last = run_bits(m.y, warp);
            const int off = mine;
            const Tin* xs = reinterpret_cast<const Tin*>(smem + st * M::kStage) + off;
            const Tin* us = reinterpret_cast<const Tin*>(smem + st * M::kStage + M::kX) + off;
            const float* gt = reinterpret_cast<const float*>(smem + st * M::kStage + 2 * M::kX) + off;
            auto row_of = [&](int i) { return ((long)seq_of(P, tw + i) * P.Z + L.z) * P.d + L.c; };
            auto row = [&](const float* from, int i) { return from && L.on ? ld4(from + row_of(i)) : all4(0.f); };
            // 1. the gates, and the run's (A, B) forward and in reverse
            Gate<kShared> a, w, dw;
    #pragma unroll
            for (int i = 0; i < kRun; ++i) {
                P4 a1, w1, dw1;
                token_gates<kShared, true>(P.rule, gt + i * lanes.row, gs[i], &a1, &w1, &dw1);
                if (ragged && tw + i >= P.T) a1 = all4(1.f), w1 = dw1 = all4(0.f);
                a.set(i, a1);
                w.set(i, w1);
                dw.set(i, dw1);
            }
            // (tokens behind the end are staged as whatever the stage held)
            auto x_at = [&](int i) { return ragged && tw + i >= P.T ? all4(0.f) : ld4(xs + i * lanes.row); };
            auto u_at = [&](int i) { return ragged && tw + i >= P.T ? all4(0.f) : ld4(us + i * lanes.row); };
            const int cut = 31 - __clz(first);         // the last begin in the run; -1: none
            P4 ra = all4(1.f), rb = all4(0.f), edge = all4(0.f);
            if (first) edge = row(P.S0, cut);
    #pragma unroll
            for (int i = 0; i < kRun; ++i) {
                if (i == cut) rb = edge;
                ra = mul4(ra, a.at(i));
                rb = fma4(a.at(i), rb, mul4(w.at(i), x_at(i)));
            }
            if (first) ra = all4(kCut);
            float* out = runs + warp * kCh + lane * 4;
            st4(out, ra);
            st4(out + M::kRuns, rb);
            ra = all4(1.f);
            rb = all4(0.f);
            const int stop = __ffs(last) - 1;          // the first end in the run
            if (last) edge = row(P.dST, stop);
    #pragma unroll
            for (int i = kRun - 1; i >= 0; --i) {
                if (i == stop) rb = edge;
                ra = mul4(ra, a.at(i));
                rb = mul4(a.at(i), add4(u_at(i), rb));
            }
            if (last) ra = all4(kCut);
            st4(out + 2 * M::kRuns, ra);
            st4(out + 3 * M::kRuns, rb);
            warp_arrive(ready);
            wait_or_give_up(entered, n & 1, &dead, P.err);
            // 2. the states before the run's tokens: e = a h' + w' x
            P4 e[kRun], G[kRun];
            P4 h = ld4(out + M::kRuns);
    #pragma unroll
            for (int i = 0; i < kRun; ++i) {
                const P4 xv = x_at(i);
                e[i] = fma4(a.at(i), h, mul4(dw.at(i), xv));
                h = fma4(a.at(i), h, mul4(w.at(i), xv));
            }
            for (uint32_t bits = first; bits; bits &= bits - 1) {       // once more from where a sequence begins
                const int from = __ffs(bits) - 1;
                h = row(P.S0, from);
    #pragma unroll
                for (int i = 0; i < kRun; ++i)
                    if (i >= from) {
                        const P4 xv = x_at(i);
                        e[i] = fma4(a.at(i), h, mul4(dw.at(i), xv));
                        h = fma4(a.at(i), h, mul4(w.at(i), xv));
                    }
            }
            // 3. the gradients
            P4 c = ld4(out + 3 * M::kRuns);
    #pragma unroll
            for (int i = kRun - 1; i >= 0; --i) {
                G[i] = add4(u_at(i), c);
                c = mul4(a.at(i), G[i]);
            }
            for (uint32_t bits = last; bits;) {                         // once more from where a sequence ends
                const int from = 31 - __clz(bits);
                bits ^= 1u << from;
                c = row(P.dST, from);
    #pragma unroll
                for (int i = kRun - 1; i >= 0; --i)
                    if (i <= from) {
                        G[i] = add4(u_at(i), c);
                        c = mul4(a.at(i), G[i]);
                    }
            }
            const int live = L.on ? P.T - tw : 0;
            float* dx = P.dx + (L.z * P.T + tw) * P.d + L.c;
            float* dg = P.dg + (L.z * P.T + tw) * (kShared ? 1 : P.d) + (kShared ? 0 : L.c);
    #pragma unroll
            for (int i = 0; i < kRun; ++i) {
                const P4 dgv = mul4(e[i], G[i]);
                if (i < live) {
                    st4(dx + i * P.d, mul4(w.at(i), G[i]));
                    if (!kShared) st4(dg + i * P.d, dgv);
                }
                if (kShared) {      // over the head's channels; a part of a wide head leaves a partial sum
                    float sum = i < live ? (dgv.lo.x + dgv.lo.y) + (dgv.hi.x + dgv.hi.y) : 0.f;
                    for (int far = S.heads > 1 ? S.dv / 2 : 16; far > 0; far >>= 1)
                        sum += __shfl_xor_sync(0xffffffffu, sum, far);
                    if (i < live && (S.heads > 1 ? lane % S.dv == 0 : lane == 0)) {
                        if (S.per_head == 1) dg[i] = sum;
                        else parts[((long)(strip % S.per_head) * P.Z + L.z) * P.T + tw + i] = sum;
                    }
                }
            }
            for (uint32_t bits = P.dS0 ? first : 0u; bits; bits &= bits - 1) {
                const int from = __ffs(bits) - 1;
                P4 d0 = all4(0.f);
    #pragma unroll
                for (int i = 0; i < kRun; ++i)
                    if (i == from) d0 = mul4(a.at(i), G[i]);
                if (L.on) st4(P.dS0 + row_of(from), d0);
            }
            warp_arrive(spent + st);
        }
    }
    if (blocks > 1) cluster_sync();
}

__global__ void __launch_bounds__(256) scan_parts_kernel(const float* __restrict__ parts, float* __restrict__ dg,
                                                         long n, int count) {
    for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long)gridDim.x * 256) {
        float sum = parts[i];
        for (int p = 1; p < count; ++p) sum += parts[p * n + i];
        dg[i] = sum;
    }
}

// One token: a thread per four channels of a row.
template <typename Tin>
__global__ void __launch_bounds__(256) scan_step_kernel(const Tin* __restrict__ x, const float* __restrict__ g,
                                                        float* S, Tin* __restrict__ o, int N, int H, int d, int gw,
                                                        int rule, PagedRows P, bool paged, int pieces) {
    const int n = blockIdx.x / pieces;
    const int j = ((blockIdx.x % pieces) * 256 + threadIdx.x) * 4;      // channel of the row's H * d
    const long row = (long)n * H * d;
    const float* from = S + row;
    float* to = S + row;
    if (paged) {
        const RowPages p = paged_row(P, N, n);
        if (!p.active) return;
        to = reinterpret_cast<float*>(reinterpret_cast<char*>(S) + p.write * P.page_bytes);
        from = p.read < 0 ? nullptr : reinterpret_cast<float*>(reinterpret_cast<char*>(S) + p.read * P.page_bytes);
    }
    if (j >= H * d) return;
    P4 a, w, dw;
    if (gw == 1) token_gates<true, false>(rule, nullptr, g[(long)n * H + j / d], &a, &w, &dw);
    else token_gates<false, false>(rule, g + row + j, 0.f, &a, &w, &dw);
    const P4 h = fma4(a, from ? ld4(from + j) : all4(0.f), mul4(w, ld4(x + row + j)));
    st4(to + j, h);
    st4(o + row + j, h);
}

}  // namespace

static size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
static long scan_steps(int T) { return ((long)T + kTok - 1) / kTok; }

size_t scan_states_bytes(long Z, int T, int d) { return (size_t)scan_steps(T) * Strips(Z, d).count * kCh * sizeof(float); }
// the partial sums of a shared decay's gradient where a head is wider than a strip
size_t scan_scratch_bytes(long Z, int T, int d, int gw, bool backward) {
    const Strips S(Z, d);
    return backward && gw == 1 && S.per_head > 1 ? up256((size_t)S.per_head * Z * T * sizeof(float)) : 0;
}

namespace {

// How many clusters of each size a device holds at once, asked once per device and kernel.
struct Room {
    std::atomic<int> clusters[5];      // of 1, 2, 4, 8, 16 blocks
    std::atomic<int> sms;
};

template <typename Kernel>
cudaError_t config(Kernel kernel, int blocks, int smem, long strips, cudaStream_t stream, cudaLaunchConfig_t* cfg,
                   cudaLaunchAttribute* attr) {
    *cfg = cudaLaunchConfig_t{};
    cfg->gridDim = dim3((unsigned)(strips * blocks));
    cfg->blockDim = dim3(kThreads);
    cfg->dynamicSmemBytes = (size_t)smem;
    cfg->stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg->attrs = attr;
    cfg->numAttrs = blocks > 1 ? 1 : 0;
    return cudaSuccess;
}

template <typename Kernel>
cudaError_t find_room(Kernel kernel, int (*smem)(int), Room* room) {
    int dev = 0, sms = 0;
    cudaError_t e;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem(kCluster))) != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return e;
    for (int i = 0; i < 5; ++i) {
        int n = 0;
        if (i == 0) {
            if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kThreads, smem(1))) != cudaSuccess) return e;
            n *= sms;
        } else {
            cudaLaunchConfig_t cfg;
            cudaLaunchAttribute attr[1];
            config(kernel, 1 << i, smem(1 << i), 64, nullptr, &cfg, attr);
            if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
                cudaGetLastError();       // a size that this device does not run
                n = 0;
            }
        }
        room->clusters[i].store(n, std::memory_order_relaxed);
    }
    room->sms.store(sms, std::memory_order_release);
    return cudaSuccess;
}

// Blocks per cluster: with rounds = strips / clusters held at once, a strip's turns are
// ceil(steps / blocks), and a turn takes as long as the blocks that share an SM, or, for fewer
// than two, as its own latency (about 1.6 of a block's share at full rate).
int pick_blocks(const Room& room, long strips, long steps) {
    int best = 1;
    double least = 0;
    for (int i = 0; i < 5; ++i) {
        const int n = room.clusters[i].load(std::memory_order_relaxed), blocks = 1 << i;
        if (n == 0 || (i > 0 && steps <= blocks / 2)) continue;
        const long held = strips < n ? strips : n, sms = room.sms.load(std::memory_order_relaxed);
        const double share = (double)((held * blocks + sms - 1) / sms);
        const double cost = (double)((strips + n - 1) / n) * (double)((steps + blocks - 1) / blocks) * (share < 1.6 ? 1.6 : share);
        if (i == 0 || cost < least) best = blocks, least = cost;
    }
    return best;
}

template <typename Kernel, typename... Args>
cudaError_t launch_clusters(Kernel kernel, int (*smem)(int), Room* rooms, const ScanArgs& a, cudaStream_t stream,
                            Args... args) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64) return cudaErrorInvalidDevice;
    Room& room = rooms[dev];
    if (room.sms.load(std::memory_order_acquire) == 0 && (e = find_room(kernel, smem, &room)) != cudaSuccess) return e;
    const long strips = Strips(a.Z, a.d).count, steps = scan_steps(a.T);
    const int blocks = pick_blocks(room, strips, steps);
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[1];
    config(kernel, blocks, smem(blocks), strips, stream, &cfg, attr);
    return cudaLaunchKernelEx(&cfg, kernel, a, args..., blocks, (int)steps);
}

template <typename Tin, bool kShared>
cudaError_t launch_fwd(const ScanArgs& a, cudaStream_t stream) {
    static Room rooms[64];
    return launch_clusters(scan_fwd_kernel<Tin, kShared>, FwdSmem<Tin, kShared>::bytes, rooms, a, stream);
}

template <typename Tin, bool kShared>
cudaError_t launch_bwd(const ScanArgs& a, cudaStream_t stream) {
    static Room rooms[64];
    const int per_head = Strips(a.Z, a.d).per_head;
    float* parts = static_cast<float*>(a.scratch);
    const cudaError_t e = launch_clusters(scan_bwd_kernel<Tin, kShared>, BwdSmem<Tin, kShared>::bytes, rooms, a, stream,
                                          (const float*)a.E, parts);
    if (e != cudaSuccess || !kShared || per_head == 1) return e;
    const long n = a.Z * a.T, blocks = (n + 255) / 256;
    scan_parts_kernel<<<(unsigned)(blocks < 4096 ? blocks : 4096), 256, 0, stream>>>(parts, a.dg, n, per_head);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_scan_fwd(const ScanArgs& a, bool bf16, cudaStream_t stream) {
    if (bf16) return a.gw == 1 ? launch_fwd<__nv_bfloat16, true>(a, stream) : launch_fwd<__nv_bfloat16, false>(a, stream);
    return a.gw == 1 ? launch_fwd<float, true>(a, stream) : launch_fwd<float, false>(a, stream);
}

cudaError_t launch_scan_bwd(const ScanArgs& a, bool bf16, cudaStream_t stream) {
    if (bf16) return a.gw == 1 ? launch_bwd<__nv_bfloat16, true>(a, stream) : launch_bwd<__nv_bfloat16, false>(a, stream);
    return a.gw == 1 ? launch_bwd<float, true>(a, stream) : launch_bwd<float, false>(a, stream);
}

cudaError_t launch_scan_step(const void* x, const float* g, float* S, void* o, int N, int H, int d, int gw, bool bf16,
                             int rule, const PagedRows* paged, cudaStream_t stream) {
    const int pieces = (int)(((long)H * d / 4 + 255) / 256);
    const unsigned grid = (unsigned)((long)pieces * N);
    const PagedRows p = paged ? *paged : PagedRows();
    if (bf16)
        scan_step_kernel<<<grid, 256, 0, stream>>>((const __nv_bfloat16*)x, g, S, (__nv_bfloat16*)o, N, H, d, gw, rule,
                                                   p, paged != nullptr, pieces);
    else
        scan_step_kernel<<<grid, 256, 0, stream>>>((const float*)x, g, S, (float*)o, N, H, d, gw, rule, p,
                                                   paged != nullptr, pieces);
    return cudaGetLastError();
}

}  // namespace efla
