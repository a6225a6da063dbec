// efla_scan.cu -- the per-channel gated linear recurrence: forward, backward, one token.
//
// The recurrence is affine in the state: over any run of tokens h_out = A h_in + B, and runs
// compose.  A strip is 128, 64 or 32 channels, a tile 32, 64 or 128 tokens of it (4096 values).
// A cluster of blocks takes one strip along time: in each turn its blocks hold consecutive tiles,
// and
//   1. the eight compute warps reduce runs of four tokens (a lane: four channels of one run) to
//      (A, B);
//   2. the chain threads (two channels of eight runs each) fold these, write the results into the
//      shared memory of every block of the cluster, and fold what all blocks sent onto the state
//      the turn began with: the state entering their own runs, and the one that the next turn
//      begins with, which is thus known to every block without another exchange;
//   3. the compute warps continue their runs from there and write the outputs.
// Bound by memory where there are strips enough (444 heads of 128, T 2048, bf16: 150 us, 6.2 TB/s, 95%
// of the measured copy rate), by a turn's latency, about 2 us from its loads to the next state,
// where there are few (64 heads: 32 us, 4.2 TB/s; 16 heads, T 32768: 125 us, 4.3 TB/s, in a graph of calls, 127 to 129 call
// by call): strips as narrow as 32 channels and clusters along time are there to have more turns in flight.  A turn of 64
// heads' 3370 cycles: products 1400, fold 200, exchange 410, entering 240, outputs 600, waits 500; with six blocks in a cluster a turn
// takes about 4900, half of them the exchange, which waits for the slowest block.
// Inputs are staged some turns ahead and read from memory once; tokens behind the end and
// channels beside a head are staged as zeros, which change nothing (e^0 = 1, x = 0).  Everything
// is folded in token order, so the results are the same bits on every run.
#include <string.h>

#include <type_traits>

#include "efla_kernels.h"
#include "efla_pages.cuh"
#include "efla_scan.cuh"
#include "efla_tma.cuh"
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

constexpr int kValues = 4096, kWarps = 8, kRun = 4, kLanes4 = 128;      // values of a tile; channels x runs of a warp
constexpr int kComputeThreads = kWarps * 32, kChainThreads = 64, kThreads = kComputeThreads + kChainThreads;
constexpr int kCluster = 8;        // most blocks of a cluster
constexpr int kMarks = 4;          // tiles whose marks are kept
constexpr uint64_t kWaitNs = 2000000000ull;

// How streams, channels and tokens make strips and tiles: a function of the shape alone, since
// the states kept for the backward pass lie by it.
struct Geo {
    int width;         // channels of a strip: 128, 64, 32
    int groups;        // runs of a warp side by side: 128 / width
    int tokens;        // of a tile: 32 groups
    int heads;         // whole heads packed side by side in a strip (their width divides the strip's)
    int per_head;      // strips of a head that is wider
    int strips, steps;
    int box;           // channels of one staged box: a head, or a strip's part of it
    int planned;       // blocks that the plan counts on in a forward
};

// What a lane holds: channels c .. c + 3 of stream z, run `run` of each tile.
struct Lane {
    long z;
    int c, run;
    bool on;
    int smem, row;     // element offset of the run's first token in a staged tile; elements between tokens
};
__device__ __forceinline__ Lane lane_of(const Geo& G, long Z, int d, int strip, int warp, int lane) {
    const int lanes = G.width / 4, dv = d / 4, q = lane % lanes;      // q: four channels of the strip
    Lane L;
    L.run = warp * G.groups + lane / lanes;
    L.row = G.box;
    if (G.heads > 1) {
        const int p = q / dv;
        L.z = (long)strip * G.heads + p;
        L.c = (q % dv) * 4;
        L.smem = p * G.tokens * d + L.c;
    } else {
        L.z = strip / G.per_head;
        L.c = (strip % G.per_head) * G.width + q * 4;
        L.smem = q * 4 < G.box ? q * 4 : 0;
    }
    L.on = L.z < Z && L.c < d;
    L.smem += L.run * kRun * L.row;
    return L;
}

// Staging by one warp: bytes that will arrive, then each tensor's copies.  A strip of whole heads is
// contiguous per head (one bulk copy each, about a tenth faster than TMA boxes); what lies behind
// the end or beside the last head is zeroed.  A part of a wide head is a TMA box, which fills
// with zeros itself.
struct Stager {
    int heads, z0, c0;        // heads that there are, the first of them, and the first channel
    const Geo& G;
    long T;
    __device__ __forceinline__ Stager(const Geo& G_, long Z, int T_, int strip) : G(G_), T(T_) {
        z0 = G.per_head > 1 ? strip / G.per_head : strip * G.heads;
        c0 = G.per_head > 1 ? (strip % G.per_head) * G.width : 0;
        heads = (int)min((long)G.heads, Z - z0);
    }
    __device__ __forceinline__ int rows(int t0) const { return (int)min((long)G.tokens, T - t0); }
    __device__ __forceinline__ int values(int t0) const {
        return G.per_head > 1 ? kValues : heads * rows(t0) * G.box;
    }
    template <typename E>
    __device__ __forceinline__ void zero_rest(E* dst, int t0) const {
        if (G.per_head > 1 || (T - t0 >= G.tokens && heads == G.heads)) return;
        const int lane = threadIdx.x & 31, head = G.tokens * G.box, there = rows(t0) * G.box;
        for (int p = 0; p < G.heads; ++p)
            for (int i = (p < heads ? there : 0) + lane * 4; i < head; i += 128) st4(dst + p * head + i, all4(0.f));
        fence_proxy_async_smem();      // (a later tile's copy may write there)
    }
    template <typename E>
    __device__ __forceinline__ void stage(E* dst, const E* src, const CUtensorMap* map, int t0, uint64_t* bar) const {
        const int lane = threadIdx.x & 31;
        if (G.per_head > 1) {
            if (lane == 0) tma_load_3d(dst, map, bar, c0, t0, z0);
        } else if (lane < heads) {
            bulk_load(dst + lane * G.tokens * G.box, src + ((z0 + lane) * T + t0) * G.box, rows(t0) * G.box * (int)sizeof(E), bar);
        }
    }
};

// The packed sequence that holds token t, the largest n with cu[n] <= t, by one warp: 32 offsets at a time.
__device__ __forceinline__ int seq_of(const int* cu, int nseq, int t) {
    int lo = 0;
    for (long span = nseq; span > 1;) {
        const long step = (span + 31) / 32, at = lo + (threadIdx.x & 31) * step;
        const int below = __popc(__ballot_sync(0xffffffffu, at < lo + span && cu[at] <= t)) - 1;
        span = min(step, span - below * step);
        lo += (int)(below * step);
    }
    return lo;
}

// Which of a tile's tokens begin or end a sequence (bit l of word j: token 32 j + l), which sequence that is,
// and whether any does.  The warp that stages a tile finds them, and asks for the rows of state that the
// tile will read there: looked up by the compute warps themselves they cost a packed batch a third more time.
struct Marks {
    uint32_t first[4], last[4];
    int seq[kLanes4];
};
struct MarkRing {
    Marks m[kMarks];
    uint32_t any[kMarks];
    int2 extent[32];       // of a lane's sequence, where there are up to 32 of them
};
// The part of a row of states that a strip reads, towards this SM.
struct StateRow {
    const float* base;      // of sequence 0, or null
    long stride;            // floats between sequences
    int floats;
    __device__ __forceinline__ void prefetch(int n) const {
        if (!base) return;
        for (int i = 0; i < floats; i += 32)
            asm volatile("prefetch.global.L1 [%0];" ::"l"(base + n * stride + i) : "memory");
    }
};
// One warp: the sequences from the one that holds t0 on, a lane each.  (A call, so that what few
// tiles need costs the kernels no registers.)
__device__ __noinline__ bool find_marks(const int* cu, int nseq, int2 own, int t0, int t1, StateRow begins, StateRow ends,
                                        Marks* m) {
    const int lane = threadIdx.x & 31;
    const bool few = nseq <= 32;
    uint32_t* words = m->first;                // and m->last behind it
    if (lane < 8) words[lane] = 0;
    __syncwarp();
    bool any = false;
    for (int n0 = few ? 0 : seq_of(cu, nseq, t0);; n0 += 32) {
        const int n = n0 + lane;
        const int from = few ? own.x : n >= nseq ? t1 : cu[n], to = few ? own.y : n >= nseq ? t1 : cu[n + 1];
        if (from < to && from >= t0 && from < t1) {
            atomicOr(words + ((from - t0) >> 5), 1u << ((from - t0) & 31));
            m->seq[from - t0] = n;
            begins.prefetch(n);
            any = true;
        }
        if (from < to && to > t0 && to <= t1) {
            atomicOr(words + 4 + ((to - 1 - t0) >> 5), 1u << ((to - 1 - t0) & 31));
            m->seq[to - 1 - t0] = n;           // (the same one, if the token is its first too)
            ends.prefetch(n);
            any = true;
        }
        if (few || __any_sync(0xffffffffu, from >= t1)) break;
    }
    return __any_sync(0xffffffffu, any);
}
// Held by the staging warp for itself: looked up for every tile, the offsets cost it, and with it the next turn, two
// loads one behind the other (packed requests 78.4 us instead of 75).
__device__ __forceinline__ void hold_extents(const int* cu, int nseq, int T, MarkRing* ring) {
    const int n = threadIdx.x & 31;
    ring->extent[n] = n < nseq ? (cu ? make_int2(cu[n], cu[n + 1]) : make_int2(0, T)) : make_int2(0, 0);
}
__device__ __forceinline__ void make_marks(const ScanArgs& P, const int* cu, const Stager& S, int chunk, const float* begins,
                                           const float* ends, MarkRing* ring, int slot) {
    const int t0 = chunk * S.G.tokens, t1 = t0 + min(S.G.tokens, P.T - t0), nseq = cu ? P.nseq : 1;
    const int2 own = ring->extent[threadIdx.x & 31];
    bool any = nseq > 32 || __any_sync(0xffffffffu, own.x < own.y && ((own.x >= t0 && own.x < t1) ||
                                                                          (own.y > t0 && own.y <= t1)));
    if (any) {
        const long at = (long)S.z0 * P.d + S.c0, row = P.Z * P.d;
        const int floats = (int)min((long)(S.G.per_head > 1 ? min(S.G.width, P.d - S.c0) : S.heads * P.d), row - at);
        any = find_marks(cu, nseq, own, t0, t1, StateRow{begins ? begins + at : nullptr, row, floats},
                         StateRow{ends ? ends + at : nullptr, row, floats}, ring->m + slot);
    }
    if ((threadIdx.x & 31) == 0) ring->any[slot] = any;
}
__device__ __forceinline__ uint32_t run_bits(const uint32_t* words, int run) {
    return words[run >> 3] >> (run & 7) * kRun & ((1u << kRun) - 1u);
}

// Whether a warp's runs of a tile have any mark.
__device__ __forceinline__ bool warp_marked(const MarkRing* ring, int slot, int warp, const Geo& G) {
    if (!ring->any[slot]) return false;
    const int bits = G.groups * kRun, at = warp * bits;       // 4, 8 or 16 tokens
    const Marks& m = ring->m[slot];
    return (m.first[at >> 5] | m.last[at >> 5]) >> (at & 31) & ((1u << bits) - 1u);
}

// Sequences without tokens pass their states through.
__device__ __forceinline__ void pass_empty(const ScanArgs& P, const int* cu, const float* in, float* out) {
    if (!cu || !out) return;
    for (int n = blockIdx.x; n < P.nseq; n += gridDim.x)
        if (cu[n] == cu[n + 1])
            for (long i = threadIdx.x; i < P.Z * P.d; i += kThreads)
                out[n * P.Z * P.d + i] = in ? in[n * P.Z * P.d + i] : 0.f;
}

// A of a run with a sequence's begin in it: what came before does not matter, not even a NaN.
// (No product of decays is -0.)  A cut is one for all channels.
constexpr float kCut = -0.0f;
__device__ __forceinline__ bool is_cut(float A) { return __float_as_uint(A) == 0x80000000u; }
__device__ __forceinline__ float2 run_on(float2 A, float2 h, float2 B) { return is_cut(A.x) ? B : fma2(A, h, B); }
__device__ __forceinline__ float2 ld2(const float* p) { return *reinterpret_cast<const float2*>(p); }

// Eight runs folded to one (A, B); the state entering each of them takes the place of its B.
struct Fold {
    float2 A, B;
};
__device__ __forceinline__ bool is_finite(float x) { return fabsf(x) <= 3.402823466e38f; }
template <bool kReverse>
__device__ __forceinline__ Fold fold_runs(const float* runA, const float* runB, int width) {
    Fold f{both(1.f), both(0.f)};
    bool cut = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int w = kReverse ? 7 - i : i;
        const float2 a = ld2(runA + w * width);
        cut |= is_cut(a.x);
        f.B = run_on(a, f.B, ld2(runB + w * width));
        f.A = mul2(f.A, a);
    }
    if (cut) f.A = both(kCut);
    return f;
}
__device__ __forceinline__ Fold fold_two(const Fold& f, const Fold& then) {
    const bool cut = is_cut(f.A.x) || is_cut(then.A.x);
    return Fold{cut ? both(kCut) : mul2(f.A, then.A), run_on(then.A, f.B, then.B)};
}
template <bool kReverse>
__device__ __forceinline__ void enter_runs(const float* runA, float* runB, int width, float2 h) {
    float2 A[8], B[8];
#pragma unroll
    for (int w = 0; w < 8; ++w) A[w] = ld2(runA + w * width), B[w] = ld2(runB + w * width);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int w = kReverse ? 7 - i : i;
        *reinterpret_cast<float2*>(runB + w * width) = h;
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
    __syncwarp();
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

// A chain thread's part of one turn: it sends its eight runs' (A, B) to every block and folds
// everybody's, in the order of time, onto `carry`, the state the turn began with, which becomes
// the one the next turn begins with.  Returns the state entering its own runs.
// sent: [2][blocks * groups][width / 2] x {A, B of two channels}; `entry`: its place in that order.
__device__ __forceinline__ float2 chain_turn(const Fold& f, int blocks, const Geo& G, int entry, int pair, int n,
                                             float4* sent, uint64_t* got, float2* carry, bool* dead, uint32_t* err) {
    float2 h = *carry;
    const int entries = blocks * G.groups;
    if (entries == 1) {
        *carry = run_on(f.A, h, f.B);
        return h;
    }
    const int buf = n & 1, row = G.width / 2;
    float4* all = sent + buf * blocks * kChainThreads;
    if (blocks == 1) {
        all[entry * row + pair] = make_float4(f.A.x, f.A.y, f.B.x, f.B.y);
        bar_sync(1, kChainThreads);
    } else {
        const uint32_t to = smem_u32(all + entry * row + pair), bar = smem_u32(got + buf);
        for (int q = 0; q < blocks; ++q) send(in_block(to, q), in_block(bar, q), f.A, f.B);
        if (threadIdx.x == kComputeThreads) mbar_arrive_expect_tx(got + buf, blocks * kChainThreads * 16);
        wait_or_give_up(got + buf, n >> 1 & 1, dead, err);
    }
    float2 mine = h;
#pragma unroll 4
    for (int q = 0; q < entries; ++q) {
        const float4 v = all[q * row + pair];
        if (q == entry) mine = h;
        h = run_on(make_float2(v.x, v.y), h, make_float2(v.z, v.w));
    }
    *carry = h;
    return mine;
}

// The same for a forward's strip of 32 channels in a cluster: of its four parts a warp has two and sends them as one, each
// half of it to every other block (the long document in a graph of calls 131.7 -> 125.0 us, packed requests 76.6 -> 73.2.
// Within one block, and in the backward, whose registers it takes, it costs more than it gives: layer prefill 32.2 -> 34.5).
// The decays of two parts, 64 tokens, may multiply to more than fp32 holds where those of each do not (growth), and so may
// what they leave of their inputs.  The state behind such a pair is then not finite, whatever entered it.  All warps of the
// cluster read all pairs of the strip, so all see it, and the parts follow (as they do where inputs are not finite).  To look
// for it costs a turn 0.05 us (without it 122.7 and 71.7); a document that grows so in every turn takes 175 us.
struct Parts {
    float2 mine, h;            // the state entering the warp's own pair, and the last one
    bool dead;
};
// Folds the turn's pairs onto h, those that fp32 does not hold part by part.  The parts go to the second half of `sent`,
// counted by a barrier of their own: every block has read one turn's parts before it sends the next turn's pairs, and no
// block sends parts again before it has got these.  A channel's state comes from its own pairs and parts alone.  (A call,
// so that what few streams need costs the kernels few registers.)
__device__ __noinline__ Parts fold_parts(Fold f, float2 h, int blocks, int place, const float4* pairs, float4* sent,
                                         uint64_t* got, bool dead, uint32_t* err) {
    const int lane = threadIdx.x & 31, second = lane >> 4;
    int* turns = reinterpret_cast<int*>(got + 1) + (place & 1);      // this warp's earlier ones
    const int phase = *turns & 1;
    float4* parts = sent + blocks * kChainThreads + (lane & 15);
    const uint32_t to = smem_u32(parts + (2 * place + second) * 16), bar = smem_u32(got);
    for (int q = 0; q < blocks; ++q) send(in_block(to, q), in_block(bar, q), f.A, f.B);
    if (threadIdx.x == kComputeThreads) mbar_arrive_expect_tx(got, blocks * kChainThreads * 16);
    __syncwarp();
    if (lane == 0) ++*turns;
    wait_or_give_up(got, phase, &dead, err);
    float2 now = h, mine = now;
#pragma unroll 1
    for (int q = 0; q < 2 * blocks; ++q) {
        const float4 v = pairs[q * 16], p = parts[q * 32], r = parts[q * 32 + 16];
        if (q == place) mine = now;
        const float2 one = run_on(make_float2(v.x, v.y), now, make_float2(v.z, v.w));
        now = run_on(make_float2(p.x, p.y), now, make_float2(p.z, p.w));
        now = run_on(make_float2(r.x, r.y), now, make_float2(r.z, r.w));
        if (is_finite(v.x) && is_finite(v.z)) now.x = one.x;
        if (is_finite(v.y) && is_finite(v.w)) now.y = one.y;
    }
    return Parts{mine, now, dead};
}
__device__ __forceinline__ float2 chain_turn_pairs(const Fold& f, int blocks, int rank, int n, float4* sent,
                                                   uint64_t* got, float2* carry, bool* dead, uint32_t* err) {
    const int lane = threadIdx.x & 31, place = rank * 2 + (threadIdx.x >> 5 & 1), buf = n & 1;
    const bool second = lane >= 16;
    const Fold other{make_float2(__shfl_xor_sync(0xffffffffu, f.A.x, 16), __shfl_xor_sync(0xffffffffu, f.A.y, 16)),
                     make_float2(__shfl_xor_sync(0xffffffffu, f.B.x, 16), __shfl_xor_sync(0xffffffffu, f.B.y, 16))};
    const Fold whole = second ? fold_two(other, f) : fold_two(f, other);
    float4* all = sent + buf * blocks * (kChainThreads / 2) + (lane & 15);
    const uint32_t to = smem_u32(all + place * 16), bar = smem_u32(got + buf);
    for (int q = second; q < blocks; q += 2) send(in_block(to, q), in_block(bar, q), whole.A, whole.B);
    if (threadIdx.x == kComputeThreads) mbar_arrive_expect_tx(got + buf, blocks * 2 * 16 * 16);
    wait_or_give_up(got + buf, n >> 1 & 1, dead, err);
    float2 h = *carry, mine = h, zero = both(0.f);      // zero: until a state is not finite, NaN from there on
#pragma unroll 4
    for (int q = 0; q < 2 * blocks; ++q) {
        const float4 v = all[q * 16];
        if (q == place) mine = h;
        h = run_on(make_float2(v.x, v.y), h, make_float2(v.z, v.w));
        zero = fma2(h, both(0.f), zero);
    }
    if (__any_sync(0xffffffffu, zero.x + zero.y != 0.f)) {
        const Parts parts = fold_parts(f, *carry, blocks, place, all, sent, got + 2, *dead, err);
        mine = parts.mine;
        h = parts.h;
        *dead = parts.dead;
    }
    *carry = h;
    return second ? run_on(other.A, mine, other.B) : mine;
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

// The sums of four tokens over `span` lanes, stored to to[0 .. live).  In the first two steps a lane
// passes on the tokens that it does not keep, so one value is left for the others: six shuffles
// instead of twenty.
__device__ __forceinline__ void sum_tokens(const float* sum, float* to, int span, int lane, int live) {
    if (span >= 4) {
        const bool b0 = lane & 1, b1 = lane & 2;
        float t0 = (b0 ? sum[2] : sum[0]) + __shfl_xor_sync(0xffffffffu, b0 ? sum[0] : sum[2], 1);
        float t1 = (b0 ? sum[3] : sum[1]) + __shfl_xor_sync(0xffffffffu, b0 ? sum[1] : sum[3], 1);
        float u = (b1 ? t1 : t0) + __shfl_xor_sync(0xffffffffu, b1 ? t0 : t1, 2);
#pragma unroll
        for (int far = 4; far <= 16; far *= 2)
            if (far < span) u += __shfl_xor_sync(0xffffffffu, u, far);
        const int i = 2 * b0 + b1;
        if (lane % span < 4 && i < live) to[i] = u;
        return;
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
        float u = sum[i];
        if (span == 2) u += __shfl_xor_sync(0xffffffffu, u, 1);
        if (lane % span == 0 && i < live) to[i] = u;
    }
}

// The staged tensors.
struct Maps {
    CUtensorMap x, g, dO;
};
// The offsets of a packed batch of few sequences, as an argument.
struct Offsets {
    int cu[kScanInline + 1];
};

template <typename Tin, bool kShared>
struct FwdSmem {
    static constexpr int kX = kValues * sizeof(Tin), kG = kShared ? 0 : kValues * 4;
    static constexpr int kStage = kX + kG, kStages = 2;
    static constexpr int kRuns = kWarps * kLanes4;              // floats of one value of all runs
    static constexpr int bytes(int blocks) {
        return kStages * kStage + 2 * kRuns * 4 + 2 * blocks * kChainThreads * 16 + 64 + (int)sizeof(MarkRing);
    }
};

template <typename Tin, bool kShared>
__global__ void __launch_bounds__(kThreads, 3) scan_fwd_kernel(ScanArgs P, const __grid_constant__ Maps maps, Geo G,
                                                               int blocks, const __grid_constant__ Offsets offsets) {
    using M = FwdSmem<Tin, kShared>;
    extern __shared__ __align__(128) char smem[];
    float* runs = reinterpret_cast<float*>(smem + M::kStages * M::kStage);     // [A, B (then: entering)][run][width]
    float4* sent = reinterpret_cast<float4*>(runs + 2 * M::kRuns);
    uint64_t* full = reinterpret_cast<uint64_t*>(sent + 2 * blocks * kChainThreads);
    uint64_t* ready = full + M::kStages;      // the tile's (A, B) of all runs are there
    uint64_t* entered = ready + 1;            // the states entering them are
    uint64_t* got = entered + 1;              // [2] all blocks' (A, B) are; the parts of pairs
    MarkRing* ring = reinterpret_cast<MarkRing*>(full + 8);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blocks > 1 ? (int)cluster_rank() : 0;
    const int strip = blockIdx.x / blocks, turns = (G.steps + blocks - 1) / blocks;
    const int* cu = P.by_value ? offsets.cu : P.cu;
    if (threadIdx.x == 0) {
        for (int i = 0; i < M::kStages; ++i) mbar_init(full + i, 1);
        mbar_init(ready, kWarps);
        mbar_init(entered, kChainThreads / 32);
        mbar_init(got, 1);
        mbar_init(got + 1, 1);
        mbar_init(got + 2, 1);
        got[3] = 0;               // how often parts have followed, by warp
        fence_mbar_init();
    }
    __syncthreads();
    after_previous(P.next);
    if (P.clear_err && blockIdx.x == 0 && threadIdx.x == 0) *P.err = kDevOk;
    const Stager stager(G, P.Z, P.T, strip);
    auto prefetch = [&](int n) {      // by the last warp
        const int chunk = n * blocks + rank;
        if (chunk >= G.steps) return;
        const int st = n % M::kStages;
        const int t0 = chunk * G.tokens;
        Tin* dx = reinterpret_cast<Tin*>(smem + st * M::kStage);
        float* dg = reinterpret_cast<float*>(smem + st * M::kStage + M::kX);
        make_marks(P, cu, stager, chunk, P.S0, nullptr, ring, n % kMarks);
        stager.zero_rest(dx, t0);
        if (!kShared) stager.zero_rest(dg, t0);
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(full + st, stager.values(t0) * (int)(sizeof(Tin) + (kShared ? 0 : 4)));
        __syncwarp();
        stager.stage(dx, static_cast<const Tin*>(P.x), &maps.x, t0, full + st);
        if (!kShared) stager.stage(dg, P.g, &maps.g, t0, full + st);
    };
    if (warp == kThreads / 32 - 1) {
        hold_extents(cu, cu ? P.nseq : 1, P.T, ring);
        for (int i = 0; i < M::kStages; ++i) prefetch(i);
    }
    pass_empty(P, cu, P.S0, P.S_T);
    if (blocks > 1) cluster_sync();       // every block's barriers are set up
    bool dead = false;

    if (warp >= kWarps) {                 // the chain
        const int k = threadIdx.x - kComputeThreads, pair = k % (G.width / 2), part = k / (G.width / 2);
        float* runA = runs + part * 8 * G.width + pair * 2;
        float* runB = runA + M::kRuns;
        const bool pairs = G.groups == 4 && blocks > 1;
        float2 carry = both(0.f);
        for (int n = 0; n < turns; ++n) {
            const int chunk = n * blocks + rank;
            const bool tile = chunk < G.steps;
            Fold f{both(1.f), both(0.f)};
            if (tile) {
                wait_or_give_up(ready, n & 1, &dead, P.err);
                f = fold_runs<false>(runA, runB, G.width);
            }
            const float2 h = pairs ? chain_turn_pairs(f, blocks, rank, n, sent, got, &carry, &dead, P.err)
                                   : chain_turn(f, blocks, G, rank * G.groups + part, pair, n, sent, got, &carry, &dead,
                                                P.err);
            if (tile) {
                enter_runs<false>(runA, runB, G.width, h);
                warp_arrive(entered);
                if (P.E && part == 0)
                    *reinterpret_cast<float2*>(P.E + ((size_t)chunk * G.strips + strip) * G.width + pair * 2) = h;
                if (warp == kThreads / 32 - 1) prefetch(n + M::kStages);      // the stage was read before `ready`
            }
        }
    } else {
        const Lane L = lane_of(G, P.Z, P.d, strip, warp, lane);
        float* run = runs + warp * kLanes4 + lane * 4;
        const Tin* x0 = reinterpret_cast<const Tin*>(smem) + L.smem;
        const float* g0 = reinterpret_cast<const float*>(smem + M::kX) + L.smem;
        float gn[kRun];                    // a shared decay's values for the next turn
        auto load_shared = [&](int n) {
            const int t = (n * blocks + rank) * G.tokens + L.run * kRun;
#pragma unroll
            for (int i = 0; i < kRun; ++i) gn[i] = L.on && t + i < P.T ? P.g[L.z * P.T + t + i] : 0.f;
        };
        if (kShared) load_shared(0);
        for (int n = 0; n < turns; ++n) {
            const int chunk = n * blocks + rank;
            if (chunk >= G.steps) break;
            const int tw = chunk * G.tokens + L.run * kRun, st = n % M::kStages;
            const int live = L.on ? P.T - tw : 0;
            float gs[kRun];
            if (kShared) {
#pragma unroll
                for (int i = 0; i < kRun; ++i) gs[i] = gn[i];
                load_shared(n + 1);
            }
            wait_or_give_up(full + st, n / M::kStages & 1, &dead, P.err);
            const Tin* xs = x0 + st * (M::kStage / (int)sizeof(Tin));
            const float* gt = g0 + st * (M::kStage / 4);
            // most runs have no begin or end of a sequence in them; their code knows it, and the rule
            auto tile = [&](auto plain_, auto rule_) {
                constexpr bool plain = decltype(plain_)::value;
                const int rule = decltype(rule_)::value < 0 ? P.rule : decltype(rule_)::value;
                const uint32_t first = plain ? 0u : run_bits(ring->m[n % kMarks].first, L.run);
                const int* seqs = ring->m[n % kMarks].seq + L.run * kRun;
                // 1. the run's tokens as h = a h' + b, and the run's (A, B)
                Gate<kShared> a;
                P4 b[kRun], ra = all4(1.f), rb = all4(0.f);
#pragma unroll
                for (int i = 0; i < kRun; ++i) {
                    P4 a1, w, dw;
                    token_gates<kShared, false>(rule, gt + i * L.row, gs[i], &a1, &w, &dw);
                    b[i] = mul4(w, ld4(xs + i * L.row));
                    if (!plain && (first >> i & 1u)) {       // a sequence begins: its own state enters, no other
                        if (P.S0 && L.on)
                            b[i] = fma4(a1, ld4(P.S0 + ((long)seqs[i] * P.Z + L.z) * P.d + L.c), b[i]);
                        a1 = all4(0.f);
                    }
                    a.set(i, a1);
                }
#pragma unroll
                for (int i = 0; i < kRun; ++i) {
                    if (!plain && (first >> i & 1u)) rb = all4(0.f);
                    ra = mul4(ra, a.at(i));
                    rb = fma4(a.at(i), rb, b[i]);
                }
                if (!plain && first) ra = all4(kCut);
                st4(run, ra);
                st4(run + M::kRuns, rb);
                warp_arrive(ready);
                // 3. the outputs
                wait_or_give_up(entered, n & 1, &dead, P.err);
                P4 h = ld4(run + M::kRuns);
                Tin* out = static_cast<Tin*>(P.o) + (L.z * P.T + tw) * P.d + L.c;
                const uint32_t last = plain || !P.S_T ? 0u : run_bits(ring->m[n % kMarks].last, L.run);
#pragma unroll
                for (int i = 0; i < kRun; ++i) {
                    if (!plain && (first >> i & 1u)) h = all4(0.f);      // its state is in b
                    h = fma4(a.at(i), h, b[i]);
                    if (P.o && i < live) st4(out + i * P.d, h);
                    if (!plain && (last >> i & 1u) && L.on)
                        st4(P.S_T + ((long)seqs[i] * P.Z + L.z) * P.d + L.c, h);
                }
            };
            if (warp_marked(ring, n % kMarks, warp, G)) tile(std::false_type(), std::integral_constant<int, -1>());
            else if (P.rule == kRuleExact) tile(std::true_type(), std::integral_constant<int, kRuleExact>());
            else tile(std::true_type(), std::integral_constant<int, kRuleEuler>());
        }
    }
    if (blocks > 1) cluster_sync();       // no block leaves while another may still send to it
}

// The reverse pass.  c = e^{g_t} G_t flows from token t into t - 1 (dS_T into a sequence's last
// token), G_t = dO_t + c: affine again, c_out = A c_in + R over a run, and the tiles are taken
// from the last to the first.  A tile's own states are put together again from the state that
// the forward kept for it, so no other state is ever stored.  296 heads of 128, T 2048, bf16: 209 us,
// 5.9 TB/s (90% of the measured copy rate); 64 heads: 60 us, 4.5 TB/s.  Three kinds of gate of four
// tokens stay in registers from the products to the gradients: 96 of them a thread, two blocks on an SM.  Stages of fp32
// with a decay per channel are twice as large and leave room for one block: 296 heads 310 us, 5.0 TB/s; 64 heads 84 us.
template <typename Tin, bool kShared>
struct BwdSmem {
    static constexpr int kX = kValues * sizeof(Tin), kG = kShared ? 0 : kValues * 4;
    static constexpr int kStage = 2 * kX + kG, kStages = 2;
    static constexpr int kRuns = kWarps * kLanes4;
    static constexpr int bytes(int blocks) {
        return kStages * kStage + 4 * kRuns * 4 + 2 * blocks * kChainThreads * 16 + kChainThreads * 16 + 64 +
               (int)sizeof(MarkRing);
    }
};

template <typename Tin, bool kShared>
__global__ void __launch_bounds__(kThreads, 2) scan_bwd_kernel(ScanArgs P, const __grid_constant__ Maps maps, Geo G,
                                                               int blocks, const __grid_constant__ Offsets offsets) {
    using M = BwdSmem<Tin, kShared>;
    extern __shared__ __align__(128) char smem[];
    // [A, B (then: the state entering), reverse A, R (then: the flow entering)][run][width]
    float* runs = reinterpret_cast<float*>(smem + M::kStages * M::kStage);
    float4* sent = reinterpret_cast<float4*>(runs + 4 * M::kRuns);
    float4* folds = sent + 2 * blocks * kChainThreads;      // the parts' forward (A, B)
    uint64_t* full = reinterpret_cast<uint64_t*>(folds + kChainThreads);
    uint64_t* spent = full + M::kStages;      // a stage has been read to its end
    uint64_t* ready = spent + M::kStages;
    uint64_t* entered = ready + 1;
    uint64_t* got = entered + 1;
    MarkRing* ring = reinterpret_cast<MarkRing*>(full + 8);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blocks > 1 ? (int)cluster_rank() : 0;
    const int strip = blockIdx.x / blocks, turns = (G.steps + blocks - 1) / blocks;
    const int* cu = P.by_value ? offsets.cu : P.cu;
    if (threadIdx.x == 0) {
        for (int i = 0; i < M::kStages; ++i) mbar_init(full + i, 1), mbar_init(spent + i, kWarps);
        mbar_init(ready, kWarps);
        mbar_init(entered, kChainThreads / 32);
        mbar_init(got, 1);
        mbar_init(got + 1, 1);
        fence_mbar_init();
    }
    __syncthreads();
    after_previous(P.next);
    if (P.clear_err && blockIdx.x == 0 && threadIdx.x == 0) *P.err = kDevOk;
    const Stager stager(G, P.Z, P.T, strip);
    auto prefetch = [&](int n) {
        const int chunk = G.steps - 1 - (n * blocks + rank);
        if (chunk < 0) return;
        const int st = n % M::kStages;
        const int t0 = chunk * G.tokens;
        Tin* sx = reinterpret_cast<Tin*>(smem + st * M::kStage);
        float* sg = reinterpret_cast<float*>(smem + st * M::kStage + 2 * M::kX);
        make_marks(P, cu, stager, chunk, P.S0, P.dST, ring, n % kMarks);
        stager.zero_rest(sx, t0);
        stager.zero_rest(sx + kValues, t0);
        if (!kShared) stager.zero_rest(sg, t0);
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(full + st, stager.values(t0) * (int)(2 * sizeof(Tin) + (kShared ? 0 : 4)));
        __syncwarp();
        stager.stage(sx, static_cast<const Tin*>(P.x), &maps.x, t0, full + st);
        stager.stage(sx + kValues, static_cast<const Tin*>(P.dO), &maps.dO, t0, full + st);
        if (!kShared) stager.stage(sg, P.g, &maps.g, t0, full + st);
    };
    if (warp == kThreads / 32 - 1) {
        hold_extents(cu, cu ? P.nseq : 1, P.T, ring);
        for (int i = 0; i < M::kStages; ++i) prefetch(i);
    }
    pass_empty(P, cu, P.dST, P.dS0);
    if (blocks > 1) cluster_sync();
    bool dead = false;

    if (warp >= kWarps) {             // the chain
        const int k = threadIdx.x - kComputeThreads, pair = k % (G.width / 2), part = k / (G.width / 2);
        float* runA = runs + part * 8 * G.width + pair * 2;
        float* runB = runA + M::kRuns;
        float* revA = runB + M::kRuns;
        float* revB = revA + M::kRuns;
        float2 carry = both(0.f);
        for (int n = 0; n < turns; ++n) {
            const int chunk = G.steps - 1 - (n * blocks + rank);
            const bool tile = chunk >= 0;
            float2 h = both(0.f);
            Fold f{both(1.f), both(0.f)};
            if (tile) {
                if (chunk > 0) h = ld2(P.E + ((size_t)chunk * G.strips + strip) * G.width + pair * 2);
                wait_or_give_up(ready, n & 1, &dead, P.err);
                f = fold_runs<true>(revA, revB, G.width);
            }
            const float2 c = chain_turn(f, blocks, G, rank * G.groups + G.groups - 1 - part, pair, n, sent, got, &carry,
                                        &dead, P.err);
            if (tile) {
                if (G.groups > 1) {       // the state entering this part, by the parts before it
                    const Fold own = fold_runs<false>(runA, runB, G.width);
                    folds[k] = make_float4(own.A.x, own.A.y, own.B.x, own.B.y);
                    bar_sync(1, kChainThreads);
                    for (int p = 0; p < part; ++p) {
                        const float4 v = folds[p * (G.width / 2) + pair];
                        h = run_on(make_float2(v.x, v.y), h, make_float2(v.z, v.w));
                    }
                }
                enter_runs<true>(revA, revB, G.width, c);
                enter_runs<false>(runA, runB, G.width, h);
                warp_arrive(entered);
                if (warp == kThreads / 32 - 1 && chunk - M::kStages * blocks >= 0) {
                    wait_or_give_up(spent + n % M::kStages, n / M::kStages & 1, &dead, P.err);
                    prefetch(n + M::kStages);
                }
            }
        }
    } else {
        const Lane L = lane_of(G, P.Z, P.d, strip, warp, lane);
        float* run = runs + warp * kLanes4 + lane * 4;
        const Tin* x0 = reinterpret_cast<const Tin*>(smem) + L.smem;
        const float* g0 = reinterpret_cast<const float*>(smem + 2 * M::kX) + L.smem;
        float* parts = static_cast<float*>(P.scratch);
        const int span = G.heads > 1 ? P.d / 4 : G.width / 4;      // lanes of a head
        float gn[kRun];                    // a shared decay's values for the next turn
        auto load_shared = [&](int n) {
            const int t = (G.steps - 1 - (n * blocks + rank)) * G.tokens + L.run * kRun;
#pragma unroll
            for (int i = 0; i < kRun; ++i) gn[i] = L.on && t >= 0 && t + i < P.T ? P.g[L.z * P.T + t + i] : 0.f;
        };
        if (kShared) load_shared(0);
        for (int n = 0; n < turns; ++n) {
            const int chunk = G.steps - 1 - (n * blocks + rank);
            if (chunk < 0) break;
            const int tw = chunk * G.tokens + L.run * kRun, st = n % M::kStages;
            const int live = L.on ? P.T - tw : 0;
            float gs[kRun];
            if (kShared) {
#pragma unroll
                for (int i = 0; i < kRun; ++i) gs[i] = gn[i];
                load_shared(n + 1);
            }
            wait_or_give_up(full + st, n / M::kStages & 1, &dead, P.err);
            const Tin* xs = x0 + st * (M::kStage / (int)sizeof(Tin));
            const Tin* us = xs + kValues;
            const float* gt = g0 + st * (M::kStage / 4);
            auto tile = [&](auto plain_, auto rule_) {
                constexpr bool plain = decltype(plain_)::value;
                const int rule = decltype(rule_)::value < 0 ? P.rule : decltype(rule_)::value;
                const uint32_t first = plain ? 0u : run_bits(ring->m[n % kMarks].first, L.run);
                const uint32_t last = plain ? 0u : run_bits(ring->m[n % kMarks].last, L.run);
                // (volatile: read where it is needed, and not held in registers that the products want)
                auto row_of = [&](int i) {
                    const int seq = *const_cast<volatile int*>(&ring->m[n % kMarks].seq[L.run * kRun + i]);
                    return ((long)seq * P.Z + L.z) * P.d + L.c;
                };
                auto row = [&](const float* from, int i) { return from && L.on ? ld4(from + row_of(i)) : all4(0.f); };
                // 1. the gates, and the run's (A, B) forward and in reverse
                Gate<kShared> a, w, dw;
                P4 ra = all4(1.f), rb = all4(0.f);
#pragma unroll
                for (int i = 0; i < kRun; ++i) {
                    P4 a1, w1, dw1;
                    token_gates<kShared, true>(rule, gt + i * L.row, gs[i], &a1, &w1, &dw1);
                    a.set(i, a1);
                    w.set(i, w1);
                    dw.set(i, dw1);
                    if (!plain && (first >> i & 1u)) rb = row(P.S0, i);
                    ra = mul4(ra, a1);
                    rb = fma4(a1, rb, mul4(w1, ld4(xs + i * L.row)));
                }
                if (!plain && first) ra = all4(kCut);
                st4(run, ra);
                st4(run + M::kRuns, rb);
                ra = all4(1.f);
                rb = all4(0.f);
#pragma unroll
                for (int i = kRun - 1; i >= 0; --i) {
                    if (!plain && (last >> i & 1u)) rb = row(P.dST, i);
                    ra = mul4(ra, a.at(i));
                    rb = mul4(a.at(i), add4(ld4(us + i * L.row), rb));
                }
                if (!plain && last) ra = all4(kCut);
                st4(run + 2 * M::kRuns, ra);
                st4(run + 3 * M::kRuns, rb);
                warp_arrive(ready);
                wait_or_give_up(entered, n & 1, &dead, P.err);
                // 2. the states before the run's tokens: e = a h' + w' x
                P4 e[kRun];
                P4 h = ld4(run + M::kRuns);
#pragma unroll
                for (int i = 0; i < kRun; ++i) {
                    if (!plain && (first >> i & 1u)) h = row(P.S0, i);
                    const P4 xv = ld4(xs + i * L.row);
                    e[i] = fma4(a.at(i), h, mul4(dw.at(i), xv));
                    h = fma4(a.at(i), h, mul4(w.at(i), xv));
                }
                // 3. the gradients
                P4 c = ld4(run + 3 * M::kRuns);
                float sum[kRun];
                float* dx = P.dx + (L.z * P.T + tw) * P.d + L.c;
                float* dg = P.dg + (L.z * P.T + tw) * (kShared ? 1 : P.d) + (kShared ? 0 : L.c);
#pragma unroll
                for (int i = kRun - 1; i >= 0; --i) {
                    if (!plain && (last >> i & 1u)) c = row(P.dST, i);
                    const P4 Gt = add4(ld4(us + i * L.row), c);
                    const P4 dgv = mul4(e[i], Gt);
                    c = mul4(a.at(i), Gt);
                    if (i < live) {
                        st4(dx + i * P.d, mul4(w.at(i), Gt));
                        if (!kShared) st4(dg + i * P.d, dgv);
                    }
                    if (kShared) sum[i] = L.on ? (dgv.lo.x + dgv.lo.y) + (dgv.hi.x + dgv.hi.y) : 0.f;
                    if (!plain && P.dS0 && (first >> i & 1u) && L.on) st4(P.dS0 + row_of(i), c);
                }
                if (kShared) {      // over the head's channels; a part of a wide head leaves a partial sum
                    float* to = G.per_head == 1 ? dg : parts + ((long)(strip % G.per_head) * P.Z + L.z) * P.T + tw;
                    sum_tokens(sum, to, span, lane, L.z < P.Z ? P.T - tw : 0);
                }
            };
            if (warp_marked(ring, n % kMarks, warp, G)) tile(std::false_type(), std::integral_constant<int, -1>());
            else if (P.rule == kRuleExact) tile(std::true_type(), std::integral_constant<int, kRuleExact>());
            else tile(std::true_type(), std::integral_constant<int, kRuleEuler>());
            warp_arrive(spent + st);
        }
    }
    if (blocks > 1) cluster_sync();
}

__global__ void __launch_bounds__(256) scan_parts_kernel(const float* parts, float* dg,
                                                         long n, int count) {
    after_previous();
    for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long)gridDim.x * 256) {
        float sum = parts[i];
        for (int p = 1; p < count; ++p) sum += parts[p * n + i];
        dg[i] = sum;
    }
}

// One token: a thread per four channels of a row, all loads at once.  Launch and latency are what it takes: 256 rows of
// 16 heads of 128 in pages, 8.4 MB, 4.2 us one behind the other; 4 rows of 4 heads of 64 1.8 us.
template <typename Tin>
__global__ void __launch_bounds__(256) scan_step_kernel(const Tin* x, const float* g,
                                                        float* S, Tin* o, int N, int H, int d, int gw,
                                                        int rule, PagedRows P, bool paged, int pieces) {
    after_previous();
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

// ---------------------------------------------------------------- host
// The time of a scan, in microseconds as measured on a B200 (tiles of 4096 bf16 values with a decay
// per channel): a turn takes 1.3, 1.8 and 2.3 with one to three blocks on an SM, and the exchange
// about 0.2 + 0.13 per block of the cluster; `held` clusters run at once, the others after them.
// The rule does not know the type.  Of fp32 with a decay per channel two forward blocks fit on an SM, and one
// backward block: 64 heads of 128, T 2048, take 37 and 84 us, their bytes 30.7 and 51.1 (bf16: 32 and 60, 20.5 and 40.9).
double scan_cost(long strips, long steps, int groups, int blocks, long held, long sms) {
    const long rounds = (strips + held - 1) / held, turns = (steps + blocks - 1) / blocks;
    const long share = ((strips < held ? strips : held) * blocks + sms - 1) / sms;
    const double exchange = blocks > 1 ? 0.2 + 0.13 * blocks : groups > 1 ? 0.1 : 0.0;
    return (double)(rounds * turns) * (0.75 + 0.53 * (double)share + exchange);
}

constexpr long kPlaces = 444;      // of forward blocks, three on each of 148 SMs (all types but fp32 with a decay per channel)
bool lies_evenly(long grid, long places) { return 3 * grid <= places || 4 * grid >= 3 * places; }

// The strips' width: the one with the least time at its best number of blocks, on 148 SMs with
// three blocks each.  (64 heads of 128, T 2048: 37.5 us at width 128 with four blocks, 34 at 32 with
// one; 16 heads, T 32768: 263 us at 128 with eight, 125 at 32 with six; 444 heads: 150 at 128, 160 at 32.)
Geo scan_geo(long Z, int T, int d) {
    static thread_local struct {
        long Z;
        int T, d;
        Geo geo;
    } before{-1, 0, 0, {}};          // (a call asks for its sizes several times)
    if (before.Z == Z && before.T == T && before.d == d) return before.geo;
    Geo best{};
    double least = 0;
    for (int groups = 1; groups <= 4; groups *= 2) {
        Geo G;
        G.groups = groups;
        G.width = kLanes4 / groups;
        G.tokens = 32 * groups;
        G.heads = d < G.width && G.width % d == 0 ? G.width / d : 1;
        G.per_head = (d + G.width - 1) / G.width;
        G.strips = (int)(G.heads > 1 ? (Z + G.heads - 1) / G.heads : Z * G.per_head);
        G.steps = (int)(((long)T + G.tokens - 1) / G.tokens);
        G.box = d < G.width ? d : G.width;
        double cost = 0;
        for (int b = 1; b <= kCluster && (b == 1 || b <= G.steps); ++b) {
            const double c = scan_cost(G.strips, G.steps, groups, b, kPlaces / b, 148);
            if (b == 1 || c < cost) cost = c, G.planned = G.strips * b;
        }
        if (groups == 1 || cost < least) best = G, least = cost;
    }
    before = {Z, T, d, best};
    return best;
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

size_t scan_states_bytes(long Z, int T, int d) {
    const Geo G = scan_geo(Z, T, d);
    return up256((size_t)G.steps * G.strips * G.width * sizeof(float));
}
// the partial sums of a shared decay's gradient where a head is wider than a strip
size_t scan_scratch_bytes(long Z, int T, int d, int gw, bool backward) {
    const Geo G = scan_geo(Z, T, d);
    return backward && gw == 1 && G.per_head > 1 ? up256((size_t)G.per_head * Z * T * sizeof(float)) : 0;
}

namespace {

// How many clusters of each size a device holds at once, asked once per device and kernel.
struct Room {
    std::atomic<int> clusters[kCluster + 1];
    std::atomic<int> sms;
};

template <typename Kernel>
void config(Kernel, int blocks, int smem, long strips, bool early, cudaStream_t stream, cudaLaunchConfig_t* cfg,
            cudaLaunchAttribute* attr) {
    *cfg = cudaLaunchConfig_t{};
    cfg->gridDim = dim3((unsigned)(strips * blocks));
    cfg->blockDim = dim3(kThreads);
    cfg->dynamicSmemBytes = (size_t)smem;
    cfg->stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg->attrs = blocks > 1 ? attr : attr + 1;
    cfg->numAttrs = (blocks > 1) + early;
}

template <typename Kernel>
cudaError_t find_room(Kernel kernel, int (*smem)(int), Room* room) {
    int dev = 0, sms = 0;
    cudaError_t e;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem(kCluster))) != cudaSuccess) return e;
    for (int b = 1; b <= kCluster; ++b) {
        int n = 0;
        if (b == 1) {
            if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kThreads, smem(1))) != cudaSuccess) return e;
            n *= sms;
        } else {
            cudaLaunchConfig_t cfg;
            cudaLaunchAttribute attr[2];
            config(kernel, b, smem(b), 64, false, nullptr, &cfg, attr);
            if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
                cudaGetLastError();       // a size that this device does not run
                n = 0;
            }
        }
        room->clusters[b].store(n, std::memory_order_relaxed);
    }
    room->sms.store(sms, std::memory_order_release);
    return cudaSuccess;
}

int pick_blocks(const Room& room, const Geo& G) {
    int best = 1;
    double least = 0;
    for (int b = 1; b <= kCluster && (b == 1 || b <= G.steps); ++b) {
        const long held = room.clusters[b].load(std::memory_order_relaxed);
        if (held == 0) continue;
        const double c = scan_cost(G.strips, G.steps, G.groups, b, held, room.sms.load(std::memory_order_relaxed));
        if (b == 1 || c < least) best = b, least = c;
    }
    return best;
}

template <typename T>
bool map_tokens(CUtensorMap* map, const void* ptr, const ScanArgs& a, const Geo& G) {
    auto fn = tma_encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)a.d, (cuuint64_t)a.T, (cuuint64_t)a.Z};
    cuuint64_t strides[2] = {(cuuint64_t)a.d * sizeof(T), (cuuint64_t)a.T * a.d * sizeof(T)};
    cuuint32_t box[3] = {(cuuint32_t)G.box, (cuuint32_t)G.tokens, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
              const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename Tin, bool kShared, typename Kernel>
cudaError_t launch_clusters(Kernel kernel, int (*smem)(int), Room* rooms, const ScanArgs& a, const Geo& G,
                            cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64) return cudaErrorInvalidDevice;
    Room& room = rooms[dev];
    if (room.sms.load(std::memory_order_acquire) == 0 && (e = find_room(kernel, smem, &room)) != cudaSuccess) return e;
    Maps maps{};
    if (G.per_head > 1 &&
        (!map_tokens<Tin>(&maps.x, a.x, a, G) || (!kShared && !map_tokens<float>(&maps.g, a.g, a, G)) ||
         (a.dO && !map_tokens<Tin>(&maps.dO, a.dO, a, G))))
        return cudaErrorInvalidValue;
    Offsets offsets;
    if (a.by_value) memcpy(offsets.cu, a.cu, ((size_t)a.nseq + 1) * sizeof(int));
    const int blocks = pick_blocks(room, G);
    // A scan that is set up while this one runs takes the places that this one leaves free, and its blocks may lie unevenly:
    // a layer's prefill of 256 blocks for 444 places takes 39.4 us instead of 32.6 so, and behind a backward that lets it in
    // a training step 101 instead of 92.5.  With 384 blocks there is a gain (a training step with shared decays 62.6 -> 57.0),
    // with one per SM at most too (short prompt 5.0 -> 4.5).  So a scan lets the next one in if a scan of its kind
    // and a forward of its shape, which is what follows a backward, are of those sizes.
    ScanArgs args = a;
    args.next = lies_evenly((long)G.strips * blocks, room.clusters[1].load(std::memory_order_relaxed)) &&
                lies_evenly(G.planned, kPlaces);
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    config(kernel, blocks, smem(blocks), G.strips, true, stream, &cfg, attr);
    e = cudaLaunchKernelEx(&cfg, kernel, args, maps, G, blocks, offsets);
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

template <typename Tin, bool kShared>
cudaError_t launch_fwd(const ScanArgs& a, cudaStream_t stream) {
    static Room rooms[64];
    return launch_clusters<Tin, kShared>(scan_fwd_kernel<Tin, kShared>, FwdSmem<Tin, kShared>::bytes, rooms, a,
                                         scan_geo(a.Z, a.T, a.d), stream);
}

template <typename Tin, bool kShared>
cudaError_t launch_bwd(const ScanArgs& a, cudaStream_t stream) {
    static Room rooms[64];
    const Geo G = scan_geo(a.Z, a.T, a.d);
    const cudaError_t e =
        launch_clusters<Tin, kShared>(scan_bwd_kernel<Tin, kShared>, BwdSmem<Tin, kShared>::bytes, rooms, a, G, stream);
    if (e != cudaSuccess || !kShared || G.per_head == 1) return e;
    const long n = a.Z * a.T, blocks = (n + 255) / 256;
    return launch_after(scan_parts_kernel, (unsigned)(blocks < 4096 ? blocks : 4096), 256, 0, stream,
                        static_cast<const float*>(a.scratch), a.dg, n, G.per_head);
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
        return launch_after(scan_step_kernel<__nv_bfloat16>, grid, 256, 0, stream, (const __nv_bfloat16*)x, g, S,
                            (__nv_bfloat16*)o, N, H, d, gw, rule, p, paged != nullptr, pieces);
    return launch_after(scan_step_kernel<float>, grid, 256, 0, stream, (const float*)x, g, S, (float*)o, N, H, d, gw,
                            rule, p, paged != nullptr, pieces);
}

}  // namespace efla
