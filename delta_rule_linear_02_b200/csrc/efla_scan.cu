// efla_scan.cu -- the per-channel gated linear recurrence: forward, backward, one token.
//
// The recurrence is affine in the state: over any run of tokens h_out = A h_in + B, and runs
// compose.  A tile is 64 tokens x 128 channels (a "strip"); its eight compute warps take eight
// tokens each, a lane four channels.  Per tile:
//   1. every compute thread reduces its run to (A, B), which goes to shared memory;
//   2. the chain warps (a thread per channel) publish the tile's (A, B), put the state entering
//      the tile together from the preceding tiles of the strip (look back: the state that entered
//      a tile some steps before and the (A, B) since, in token order), publish the state leaving
//      the tile, and hand every run the state entering it;
//   3. every compute thread continues its run from there and writes the outputs.
// Inputs are staged by bulk copies some tiles ahead, and are read from memory once.
//
// What is published is its own signal: a word that is not there yet holds a bit pattern that no
// result has (all ones), so publishing takes one store and reading it one load, without fences
// or flags.  The state leaving a tile is always fma(A, entering, B) of the same numbers, wherever
// the look back started, so results do not depend on timing.  The grid is launched cooperatively:
// all blocks are resident and take tiles in time order (block b: tiles b, b + grid, ...), so
// every wait is for a tile that a running block has begun or finished; each wait is bounded.
#include <cooperative_groups.h>

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
constexpr int kComputeThreads = kWarps * 32, kThreads = kComputeThreads + kCh;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kBack = 16;          // most (A, B) that one look back folds

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

struct Lane {
    long z;
    int c;           // first channel
    bool on;
    int smem;        // element offset of token 0 in a staged tile
    int row;         // elements between tokens there
};
__device__ __forceinline__ Lane lane_of(const Strips& S, long Z, int d, int strip, int lane) {
    Lane L;
    if (S.heads > 1) {
        const int p = lane / S.dv;
        L.z = (long)strip * S.heads + p;
        L.c = (lane % S.dv) * 4;
        L.on = L.z < Z;
        L.smem = p * kTok * d + L.c;
        L.row = d;
    } else {
        const int part = strip % S.per_head;
        L.z = strip / S.per_head;
        L.c = (part * 32 + lane) * 4;
        L.on = L.c < d;
        L.smem = lane * 4;
        L.row = S.per_head > 1 ? kCh : d;
        if (!L.on) L.smem = 0;       // read something that is there, use nothing of it
    }
    return L;
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

// What the tiles of a strip publish, by step (chunk in the direction of the recurrence) and strip,
// and which of a chunk's tokens begin or end a sequence (bit l: token l; packed batches).
struct Chain {
    unsigned long long* agg;     // [steps][strips][128]: A, B
    float* state;                // [steps][strips][128]: entering
    ulonglong2* marks;           // [chunks]: first, last
    int strips, steps;
};
constexpr unsigned long long kNoAgg = ~0ull;
constexpr uint32_t kNoState = ~0u;
// A of a run with a sequence's begin in it: what came before does not matter, not even a NaN.
// (No product of decays is -0.)
constexpr float kCut = -0.0f;
__device__ __forceinline__ float run_on(float A, float h, float B) {
    return __float_as_uint(A) == 0x80000000u ? B : fmaf(A, h, B);
}

__device__ __forceinline__ unsigned long long load_word(const unsigned long long* p) {
    unsigned long long v;
    asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t load_word(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.relaxed.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void publish(unsigned long long* p, float A, float B) {
    // a NaN that happens to have the pattern is made the usual one
    uint32_t b = __float_as_uint(B);
    if (b == ~0u) b = 0x7fffffffu;
    const unsigned long long v = (unsigned long long)b << 32 | __float_as_uint(A);
    asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}
__device__ __forceinline__ void publish(float* p, float h) {
    uint32_t b = __float_as_uint(h);
    if (b == ~0u) b = 0x7fffffffu;
    asm volatile("st.relaxed.gpu.global.b32 [%0], %1;" ::"l"(p), "r"(b) : "memory");
}

// Before the first tile: nothing is published, the chunks' marks, states of empty sequences.
// All blocks pass the grid's barrier before any of them looks at another's words.
__device__ __forceinline__ void begin_chain(const ScanArgs& P, const Chain& C, const float* in, float* out) {
    const long words = (long)C.steps * C.strips * kCh, all = (long)gridDim.x * kThreads;
    const long me = (long)blockIdx.x * kThreads + threadIdx.x;
    if (C.steps > 1)
        for (long i = me; i < words; i += all) {
            C.agg[i] = kNoAgg;
            reinterpret_cast<uint32_t*>(C.state)[i] = kNoState;
        }
    if (P.cu) {
        const int lane = threadIdx.x & 31;
        for (long s = me / 32; s < C.steps; s += all / 32) {
            unsigned long long first = 0, last = 0;
            for (int half = 0; half < 2; ++half) {
                const int t = (int)s * kTok + half * 32 + lane;
                const int n = t < P.T ? seq_of(P, t) : 0;
                first |= (unsigned long long)__ballot_sync(0xffffffffu, t < P.T && P.cu[n] == t) << (half * 32);
                last |= (unsigned long long)__ballot_sync(0xffffffffu, t < P.T && P.cu[n + 1] == t + 1) << (half * 32);
            }
            if (lane == 0) C.marks[s] = make_ulonglong2(first, last);
        }
        if (out)
            for (int n = blockIdx.x; n < P.nseq; n += gridDim.x)
                if (P.cu[n] == P.cu[n + 1])
                    for (long i = threadIdx.x; i < P.Z * P.d; i += kThreads)
                        out[n * P.Z * P.d + i] = in ? in[n * P.Z * P.d + i] : 0.f;
    }
    if (C.steps > 1 || P.cu) cooperative_groups::this_grid().sync();
}
__device__ __forceinline__ ulonglong2 chunk_marks(const ScanArgs& P, const Chain& C, int chunk) {
    if (P.cu) return __ldcg(C.marks + chunk);
    const int left = P.T - chunk * kTok;
    return make_ulonglong2(chunk == 0 ? 1ull : 0ull, left <= kTok ? 1ull << (left - 1) : 0ull);
}

// Thread k of the chain warps, channel k of the strip: publishes the tile's (A, B), returns the
// state entering the tile and publishes the one leaving it.  `reset`: A is zero, the leaving state
// does not depend on the entering one; `fresh`: the entering state is not needed.
__device__ __forceinline__ float chain_step(const Chain& C, int step, int strip, int k, float A, float B, bool reset,
                                            bool fresh, bool* dead, uint32_t* err) {
    const size_t at = ((size_t)step * C.strips + strip) * kCh + k, up = (size_t)C.strips * kCh;
    const bool more = step + 1 < C.steps;
    if (more) {
        if (reset) publish(C.state + at + up, B);
        publish(C.agg + at, reset ? kCut : A, B);
    }
    if (fresh) return 0.f;
    // the tiles of this grid's wave before this one publish (A, B) without waiting for states; the
    // state before them comes from an earlier wave
    const int J = min(min((int)blockIdx.x / C.strips, kBack), step - 1);
    const unsigned long long* agg = C.agg + at - J * up;
    const uint32_t* root = reinterpret_cast<const uint32_t*>(C.state) + (at - J * up);
    unsigned long long ab[kBack];
    uint32_t h0 = load_word(root);
#pragma unroll
    for (int i = 0; i < kBack; ++i) ab[i] = i < J ? load_word(agg + i * up) : 0ull;
    uint64_t begin = 0;
    for (;;) {
        bool missing = h0 == kNoState;
#pragma unroll
        for (int i = 0; i < kBack; ++i) missing |= ab[i] == kNoAgg;
        if (!missing || *dead) break;
        const uint64_t now = globaltimer_ns();
        if (begin == 0) begin = now;
        if (now - begin > kWaitNs) {
            atomicOr(err, kDevTimeout);
            *dead = true;
            break;
        }
        if (h0 == kNoState) h0 = load_word(root);
#pragma unroll
        for (int i = 0; i < kBack; ++i)
            if (ab[i] == kNoAgg) ab[i] = load_word(agg + i * up);
    }
    float h = __uint_as_float(h0);
#pragma unroll
    for (int i = 0; i < kBack; ++i) {
        if (i >= J) break;
        h = run_on(__uint_as_float((uint32_t)ab[i]), h, __uint_as_float((uint32_t)(ab[i] >> 32)));
    }
    if (more && !reset) publish(C.state + at + up, fmaf(A, h, B));
    return h;
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

// 256 compute threads and 128 chain threads share the registers of 384 x 168.
constexpr int kComputeRegs = 200, kChainRegs = 96;
static_assert(kComputeRegs * kComputeThreads + kChainRegs * kCh <= 168 * kThreads, "more registers than the block has");
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

template <typename Tin, bool kShared>
struct FwdSmem {
    static constexpr int kX = kTok * kCh * sizeof(Tin), kG = kShared ? 0 : kTok * kCh * 4;
    static constexpr int kStage = kX + kG, kStages = 3;
    static constexpr int kRuns = kWarps * kCh;                  // floats of one value of all runs
    static constexpr int kBytes = kStages * kStage + (4 + 2) * kRuns * 4 + 128;
};

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
__global__ void __launch_bounds__(kThreads, 1) scan_fwd_kernel(ScanArgs P, Chain C, int tiles) {
    using M = FwdSmem<Tin, kShared>;
    extern __shared__ __align__(128) char smem[];
    float* runs = reinterpret_cast<float*>(smem + M::kStages * M::kStage);     // [2][A, B][warp][128]
    float* entering = runs + 4 * M::kRuns;                                     // [2][warp][128]
    uint64_t* full = reinterpret_cast<uint64_t*>(entering + 2 * M::kRuns);
    uint64_t* ready = full + M::kStages;      // a tile's (A, B) of all runs are there
    uint64_t* entered = ready + 2;            // the states entering them are
    const Strips S(P.Z, P.d);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Tin* x = static_cast<const Tin*>(P.x);
    Tin* o = static_cast<Tin*>(P.o);
    if (threadIdx.x == 0) {
        for (int i = 0; i < M::kStages; ++i) mbar_init(full + i, 1);
        for (int i = 0; i < 2; ++i) mbar_init(ready + i, kWarps), mbar_init(entered + i, kCh / 32);
        fence_mbar_init();
    }
    __syncthreads();
    const int count = (tiles - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
    auto prefetch = [&](int n) {      // by the last warp
        if (n >= count) return;
        const int tile = blockIdx.x + n * gridDim.x, st = n % M::kStages;
        const int strip = tile % S.count, t0 = tile / S.count * kTok, rows = min(kTok, P.T - t0);
        if (lane == 0)
            mbar_arrive_expect_tx(full + st, rows * strip_channels(S, P.Z, P.d, strip) * (int)(sizeof(Tin) + (kShared ? 0 : 4)));
        __syncwarp();
        char* dst = smem + st * M::kStage;
        stage(reinterpret_cast<Tin*>(dst), x, S, P.Z, P.T, P.d, strip, t0, rows, full + st);
        if (!kShared) stage(reinterpret_cast<float*>(dst + M::kX), P.g, S, P.Z, P.T, P.d, strip, t0, rows, full + st);
    };
    if (warp == kThreads / 32 - 1)
        for (int i = 0; i < M::kStages; ++i) prefetch(i);
    begin_chain(P, C, P.S0, P.S_T);
    bool dead = false;

    if (warp >= kWarps) {             // the chain
        fewer_registers<kChainRegs>();
        const int k = threadIdx.x - kComputeThreads;
        for (int n = 0; n < count; ++n) {
            const int tile = blockIdx.x + n * gridDim.x, strip = tile % S.count, step = tile / S.count;
            const ulonglong2 m = chunk_marks(P, C, step);
            wait_or_give_up(ready + (n & 1), n >> 1 & 1, &dead, P.err);
            if (warp == kThreads / 32 - 1) prefetch(n + M::kStages);
            const float* ra = runs + (n & 1) * 2 * M::kRuns + k;
            float A[kWarps], B[kWarps], tA = 1.f, tB = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                A[w] = ra[w * kCh];
                B[w] = ra[M::kRuns + w * kCh];
                tB = run_on(A[w], tB, B[w]);
                tA *= A[w];
            }
            float h = chain_step(C, step, strip, k, tA, tB, m.x != 0, m.x & 1ull, &dead, P.err);
            float* en = entering + (n & 1) * M::kRuns + k;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                en[w * kCh] = h;
                h = run_on(A[w], h, B[w]);
            }
            warp_arrive(entered + (n & 1));
        }
        return;
    }
    more_registers<kComputeRegs>();

    struct Set {
        Gate<kShared> a;
        P4 b[kRun];
    };
    auto reduce = [&](Set& s, int n) {
        const int tile = blockIdx.x + n * gridDim.x, strip = tile % S.count, step = tile / S.count;
        const int tw = step * kTok + warp * kRun, st = n % M::kStages;
        const Lane L = lane_of(S, P.Z, P.d, strip, lane);
        const uint32_t first = (uint32_t)(chunk_marks(P, C, step).x >> (warp * kRun)) & ((1u << kRun) - 1u);
        const bool plain = first == 0 && tw + kRun <= P.T;
        float gs[kRun];
        if (kShared) {
#pragma unroll
            for (int i = 0; i < kRun; ++i) gs[i] = L.on && tw + i < P.T ? P.g[L.z * P.T + tw + i] : 0.f;
        }
        wait_or_give_up(full + st, n / M::kStages & 1, &dead, P.err);
        const Tin* xs = reinterpret_cast<const Tin*>(smem + st * M::kStage) + L.smem + warp * kRun * L.row;
        const float* gt = reinterpret_cast<const float*>(smem + st * M::kStage + M::kX) + L.smem + warp * kRun * L.row;
        P4 ra = all4(1.f), rb = all4(0.f);
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            P4 a, w, dw;
            token_gates<kShared, false>(P.rule, gt + i * L.row, gs[i], &a, &w, &dw);
            P4 b = mul4(w, ld4(xs + i * L.row));
            if (!plain) {
                if (tw + i >= P.T) {             // behind the end: a token that changes nothing
                    a = all4(1.f);
                    b = all4(0.f);
                }
                if (first >> i & 1u) {           // a sequence begins: its own state enters, no other
                    const int q = seq_of(P, tw + i);
                    if (P.S0 && L.on) b = fma4(a, ld4(P.S0 + ((long)q * P.Z + L.z) * P.d + L.c), b);
                    a = rb = all4(0.f);
                }
            }
            ra = mul4(ra, a);
            rb = fma4(a, rb, b);
            s.a.set(i, a);
            s.b[i] = b;
        }
        float* out = runs + (n & 1) * 2 * M::kRuns + warp * kCh + lane * 4;
        if (first) ra = all4(kCut);
        st4(out, ra);
        st4(out + M::kRuns, rb);
        warp_arrive(ready + (n & 1));
    };
    auto finish = [&](const Set& s, int n) {
        const int tile = blockIdx.x + n * gridDim.x, strip = tile % S.count, step = tile / S.count;
        const int tw = step * kTok + warp * kRun;
        const Lane L = lane_of(S, P.Z, P.d, strip, lane);
        const ulonglong2 m = chunk_marks(P, C, step);
        const uint32_t first = (uint32_t)(m.x >> (warp * kRun)) & ((1u << kRun) - 1u);
        const uint32_t last = (uint32_t)(m.y >> (warp * kRun)) & ((1u << kRun) - 1u);
        wait_or_give_up(entered + (n & 1), n >> 1 & 1, &dead, P.err);
        P4 h = ld4(entering + (n & 1) * M::kRuns + warp * kCh + lane * 4);
        Tin* out = o ? o + (L.z * P.T + tw) * P.d + L.c : nullptr;
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            if (first >> i & 1u) h = all4(0.f);          // its state is in b
            h = fma4(s.a.at(i), h, s.b[i]);
            if (o && L.on && tw + i < P.T) st4(out + i * P.d, h);
            if (P.S_T && (last >> i & 1u) && L.on) st4(P.S_T + ((long)seq_of(P, tw + i) * P.Z + L.z) * P.d + L.c, h);
        }
    };
    Set s0, s1;      // a tile's run waits in one set while the next one is reduced into the other
    for (int n = 0; n < count; n += 2) {
        reduce(s0, n);
        if (n > 0) finish(s1, n - 1);
        if (n + 1 < count) reduce(s1, n + 1);
        finish(s0, n);
    }
    if (count % 2 == 0) finish(s1, count - 1);
}

// The reverse pass.  c = e^{g_t} G_t flows from token t into t - 1 (dS_T into a sequence's last
// token), G_t = dO_t + c: affine again, c_out = A c_in + R over a run, and the tiles are taken
// from the last to the first.  A tile's own states are put together again from the state that
// the forward kept for it, so no state but one of 64 tokens is ever stored.
template <typename Tin, bool kShared>
struct BwdSmem {
    static constexpr int kX = kTok * kCh * sizeof(Tin), kG = kShared ? 0 : kTok * kCh * 4;
    static constexpr int kStage = 2 * kX + kG, kStages = 2;
    static constexpr int kRuns = kWarps * kCh;
    static constexpr int kBytes = kStages * kStage + 6 * kRuns * 4 + 128;
};

template <typename Tin, bool kShared>
__global__ void __launch_bounds__(kThreads, 1) scan_bwd_kernel(ScanArgs P, Chain C, const float* states, float* parts,
                                                               int tiles) {
    using M = BwdSmem<Tin, kShared>;
    extern __shared__ __align__(128) char smem[];
    float* runs = reinterpret_cast<float*>(smem + M::kStages * M::kStage);     // [A, B, reverse A, R][warp][128]
    float* entering = runs + 4 * M::kRuns;                                     // [state, flow][warp][128]
    uint64_t* full = reinterpret_cast<uint64_t*>(entering + 2 * M::kRuns);
    uint64_t* spent = full + M::kStages;      // a stage has been read to its end
    uint64_t* ready = spent + M::kStages;
    uint64_t* entered = ready + 1;
    const Strips S(P.Z, P.d);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Tin* x = static_cast<const Tin*>(P.x);
    const Tin* dO = static_cast<const Tin*>(P.dO);
    if (threadIdx.x == 0) {
        for (int i = 0; i < M::kStages; ++i) mbar_init(full + i, 1), mbar_init(spent + i, kWarps);
        mbar_init(ready, kWarps);
        mbar_init(entered, kCh / 32);
        fence_mbar_init();
    }
    __syncthreads();
    const int count = (tiles - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
    auto prefetch = [&](int n) {
        if (n >= count) return;
        const int tile = blockIdx.x + n * gridDim.x, st = n % M::kStages;
        const int strip = tile % S.count, t0 = (C.steps - 1 - tile / S.count) * kTok, rows = min(kTok, P.T - t0);
        if (lane == 0)
            mbar_arrive_expect_tx(full + st,
                                  rows * strip_channels(S, P.Z, P.d, strip) * (int)(2 * sizeof(Tin) + (kShared ? 0 : 4)));
        __syncwarp();
        char* dst = smem + st * M::kStage;
        stage(reinterpret_cast<Tin*>(dst), x, S, P.Z, P.T, P.d, strip, t0, rows, full + st);
        stage(reinterpret_cast<Tin*>(dst + M::kX), dO, S, P.Z, P.T, P.d, strip, t0, rows, full + st);
        if (!kShared) stage(reinterpret_cast<float*>(dst + 2 * M::kX), P.g, S, P.Z, P.T, P.d, strip, t0, rows, full + st);
    };
    if (warp == kThreads / 32 - 1)
        for (int i = 0; i < M::kStages; ++i) prefetch(i);
    begin_chain(P, C, P.dST, P.dS0);
    bool dead = false;

    if (warp >= kWarps) {             // the chain
        fewer_registers<kChainRegs>();
        const int k = threadIdx.x - kComputeThreads;
        for (int n = 0; n < count; ++n) {
            const int tile = blockIdx.x + n * gridDim.x, strip = tile % S.count, step = tile / S.count;
            const int chunk = C.steps - 1 - step;
            const ulonglong2 m = chunk_marks(P, C, chunk);
            float h = m.x & 1ull ? 0.f : states[((size_t)chunk * S.count + strip) * kCh + k];
            wait_or_give_up(ready, n & 1, &dead, P.err);
            float A[kWarps], B[kWarps], tA = 1.f, tB = 0.f;
#pragma unroll
            for (int w = kWarps - 1; w >= 0; --w) {
                A[w] = runs[2 * M::kRuns + w * kCh + k];
                B[w] = runs[3 * M::kRuns + w * kCh + k];
                tB = run_on(A[w], tB, B[w]);
                tA *= A[w];
            }
            const bool at_end = P.T - chunk * kTok <= kTok || (m.y >> (kTok - 1) & 1ull);     // nothing flows in
            float c = chain_step(C, step, strip, k, tA, tB, m.y != 0, at_end, &dead, P.err);
#pragma unroll
            for (int w = kWarps - 1; w >= 0; --w) {
                entering[M::kRuns + w * kCh + k] = c;
                c = run_on(A[w], c, B[w]);
            }
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                entering[w * kCh + k] = h;
                h = run_on(runs[w * kCh + k], h, runs[M::kRuns + w * kCh + k]);
            }
            warp_arrive(entered);
            if (warp == kThreads / 32 - 1 && n + M::kStages < count) {
                wait_or_give_up(spent + n % M::kStages, n / M::kStages & 1, &dead, P.err);
                prefetch(n + M::kStages);
            }
        }
        return;
    }
    more_registers<kComputeRegs>();

    for (int n = 0; n < count; ++n) {
        const int tile = blockIdx.x + n * gridDim.x, strip = tile % S.count, step = tile / S.count;
        const int chunk = C.steps - 1 - step, tw = chunk * kTok + warp * kRun, st = n % M::kStages;
        const Lane L = lane_of(S, P.Z, P.d, strip, lane);
        const ulonglong2 m = chunk_marks(P, C, chunk);
        const uint32_t first = (uint32_t)(m.x >> (warp * kRun)) & ((1u << kRun) - 1u);
        const uint32_t last = (uint32_t)(m.y >> (warp * kRun)) & ((1u << kRun) - 1u);
        const bool plain = (first | last) == 0 && tw + kRun <= P.T;
        float gs[kRun];
        if (kShared) {
#pragma unroll
            for (int i = 0; i < kRun; ++i) gs[i] = L.on && tw + i < P.T ? P.g[L.z * P.T + tw + i] : 0.f;
        }
        wait_or_give_up(full + st, n / M::kStages & 1, &dead, P.err);
        const int off = L.smem + warp * kRun * L.row;
        const Tin* xs = reinterpret_cast<const Tin*>(smem + st * M::kStage) + off;
        const Tin* us = reinterpret_cast<const Tin*>(smem + st * M::kStage + M::kX) + off;
        const float* gt = reinterpret_cast<const float*>(smem + st * M::kStage + 2 * M::kX) + off;
        auto state0 = [&](const float* from, int t) {      // a sequence's row of S0 or dS_T
            return from && L.on ? ld4(from + ((long)seq_of(P, t) * P.Z + L.z) * P.d + L.c) : all4(0.f);
        };
        // 1. the gates, and the run's (A, B) forward and in reverse
        Gate<kShared> a, w, dw;
        P4 ra = all4(1.f), rb = all4(0.f);
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            P4 a1, w1, dw1;
            token_gates<kShared, true>(P.rule, gt + i * L.row, gs[i], &a1, &w1, &dw1);
            if (!plain) {
                if (tw + i >= P.T) {
                    a1 = all4(1.f);
                    w1 = dw1 = all4(0.f);
                }
                if (first >> i & 1u) {
                    ra = all4(0.f);
                    rb = state0(P.S0, tw + i);
                }
            }
            ra = mul4(ra, a1);
            P4 b = mul4(w1, ld4(xs + i * L.row));
            if (!plain && tw + i >= P.T) b = all4(0.f);     // the stage holds anything there
            rb = fma4(a1, rb, b);
            a.set(i, a1);
            w.set(i, w1);
            dw.set(i, dw1);
        }
        float* out = runs + warp * kCh + lane * 4;
        if (first) ra = all4(kCut);
        st4(out, ra);
        st4(out + M::kRuns, rb);
        ra = all4(1.f);
        rb = all4(0.f);
#pragma unroll
        for (int i = kRun - 1; i >= 0; --i) {
            P4 u = ld4(us + i * L.row);
            if (!plain) {
                if (tw + i >= P.T) u = all4(0.f);
                if (last >> i & 1u) {
                    ra = all4(0.f);
                    rb = state0(P.dST, tw + i);
                }
            }
            ra = mul4(ra, a.at(i));
            rb = mul4(a.at(i), add4(u, rb));
        }
        if (last) ra = all4(kCut);
        st4(out + 2 * M::kRuns, ra);
        st4(out + 3 * M::kRuns, rb);
        warp_arrive(ready);
        wait_or_give_up(entered, n & 1, &dead, P.err);
        // 2. the states before the run's tokens: e = a h' + w' x
        P4 e[kRun];
        P4 h = ld4(entering + warp * kCh + lane * 4);
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            if (!plain && (first >> i & 1u)) h = state0(P.S0, tw + i);
            const P4 xv = ld4(xs + i * L.row);
            e[i] = fma4(a.at(i), h, mul4(dw.at(i), xv));
            h = fma4(a.at(i), h, mul4(w.at(i), xv));
        }
        // 3. the gradients
        P4 c = ld4(entering + M::kRuns + warp * kCh + lane * 4);
        float* dx = P.dx + (L.z * P.T + tw) * P.d + L.c;
        float* dg = P.dg + (L.z * P.T + tw) * (kShared ? 1 : P.d) + (kShared ? 0 : L.c);
#pragma unroll
        for (int i = kRun - 1; i >= 0; --i) {
            const bool live = L.on && tw + i < P.T;
            if (!plain && (last >> i & 1u)) c = state0(P.dST, tw + i);
            const P4 G = add4(ld4(us + i * L.row), c);
            const P4 dgv = mul4(e[i], G);
            c = mul4(a.at(i), G);
            if (!plain && tw + i >= P.T) c = all4(0.f);      // behind the end; the last token's own comes next
            if (live) {
                st4(dx + i * P.d, mul4(w.at(i), G));
                if (!kShared) st4(dg + i * P.d, dgv);
            }
            if (kShared) {      // over the head's channels; a part of a wide head leaves a partial sum
                float sum = live ? (dgv.lo.x + dgv.lo.y) + (dgv.hi.x + dgv.hi.y) : 0.f;
                for (int far = S.heads > 1 ? S.dv / 2 : 16; far > 0; far >>= 1)
                    sum += __shfl_xor_sync(0xffffffffu, sum, far);
                if (live && (S.heads > 1 ? lane % S.dv == 0 : lane == 0)) {
                    if (S.per_head == 1) dg[i] = sum;
                    else parts[((long)(strip % S.per_head) * P.Z + L.z) * P.T + tw + i] = sum;
                }
            }
            if (!plain && P.dS0 && (first >> i & 1u) && L.on)
                st4(P.dS0 + ((long)seq_of(P, tw + i) * P.Z + L.z) * P.d + L.c, c);
        }
        warp_arrive(spent + st);
    }
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
// (A, B) of every tile and the chunks' marks; backward: also the flows between tiles, and the
// partial sums of a shared decay's gradient where a head is wider than a strip
size_t scan_scratch_bytes(long Z, int T, int d, int gw, bool backward) {
    const Strips S(Z, d);
    const size_t tiles = (size_t)scan_steps(T) * S.count;
    size_t n = tiles * kCh * sizeof(unsigned long long) + up256(scan_steps(T) * sizeof(ulonglong2));
    if (backward) {
        n += tiles * kCh * sizeof(float);
        if (gw == 1 && S.per_head > 1) n += up256((size_t)S.per_head * Z * T * sizeof(float));
    }
    return n;
}

namespace {

// Launches with every block resident at once, at most one per tile.
template <typename Kernel, typename... Args>
cudaError_t launch_tiles(Kernel kernel, int smem, std::atomic<int>* resident, bool waits, long tiles,
                         cudaStream_t stream, Args... args) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int most = dev < 64 ? resident[dev].load(std::memory_order_relaxed) : 0;
    if (most == 0) {
        int sms = 0, per = 0;
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
        if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
        // the register split of compute and chain warps fits what the block is launched with
        cudaFuncAttributes fa;
        if ((e = cudaFuncGetAttributes(&fa, kernel)) != cudaSuccess) return e;
        if (fa.numRegs * kThreads < kComputeRegs * kComputeThreads + kChainRegs * kCh) return cudaErrorInvalidConfiguration;
        if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, kThreads, smem)) != cudaSuccess) return e;
        most = sms * per;
        if (dev < 64) resident[dev].store(most, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles < most ? tiles : most));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = waits ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

Chain scan_chain(const ScanArgs& a, float* states, long* tiles) {
    Chain C;
    C.strips = Strips(a.Z, a.d).count;
    C.steps = (int)scan_steps(a.T);
    *tiles = (long)C.steps * C.strips;
    C.agg = static_cast<unsigned long long*>(a.scratch);
    C.marks = reinterpret_cast<ulonglong2*>(C.agg + (size_t)*tiles * kCh);
    C.state = states ? states
                     : reinterpret_cast<float*>(reinterpret_cast<char*>(C.marks) + up256(C.steps * sizeof(ulonglong2)));
    return C;
}

template <typename Tin, bool kShared>
cudaError_t launch_fwd(const ScanArgs& a, cudaStream_t stream) {
    static std::atomic<int> resident[64];
    long tiles;
    const Chain C = scan_chain(a, a.E, &tiles);
    if (tiles >= (1l << 31)) return cudaErrorInvalidValue;
    return launch_tiles(scan_fwd_kernel<Tin, kShared>, FwdSmem<Tin, kShared>::kBytes, resident, C.steps > 1 || a.cu, tiles,
                        stream, a, C, (int)tiles);
}

template <typename Tin, bool kShared>
cudaError_t launch_bwd(const ScanArgs& a, cudaStream_t stream) {
    static std::atomic<int> resident[64];
    long tiles;
    const Chain C = scan_chain(a, nullptr, &tiles);
    if (tiles >= (1l << 31)) return cudaErrorInvalidValue;
    const int per_head = Strips(a.Z, a.d).per_head;
    float* parts = C.state + (size_t)tiles * kCh;
    cudaError_t e = launch_tiles(scan_bwd_kernel<Tin, kShared>, BwdSmem<Tin, kShared>::kBytes, resident,
                                 C.steps > 1 || a.cu, tiles, stream, a, C, (const float*)a.E, parts, (int)tiles);
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
