// efla_scan.cu -- the per-channel gated linear recurrence: forward, backward, one token.
#include "efla_kernels.h"
#include "efla_pages.cuh"
#include "efla_scan.cuh"
#include "sm100.cuh"

namespace efla {
using namespace sm100;
namespace {

struct V4 {
    float v[4];
};
template <typename T>
__device__ __forceinline__ V4 ld4(const T* p) {
    const float4 f = load4(p);
    return V4{{f.x, f.y, f.z, f.w}};
}
template <typename T>
__device__ __forceinline__ void st4(T* p, const V4& v) {
    store4(p, make_float4(v.v[0], v.v[1], v.v[2], v.v[3]));
}
__device__ __forceinline__ V4 zero4() { return V4{{0.f, 0.f, 0.f, 0.f}}; }

// ---------------------------------------------------------------- tiles
// The recurrence is affine in the state: over any run of tokens h_out = A h_in + B, and runs
// compose.  A tile is 32 tokens x 128 channels (a "strip"): its eight warps take four tokens
// each, a lane four channels, so a thread's run lives in registers and is read from memory once.
//   1. every thread reduces its run to (A, B); the warps exchange them in shared memory;
//   2. the tile's (A, B) is published, the state entering the tile is put together from the
//      preceding tiles of the strip (look back: the nearest published state, then the published
//      (A, B) after it, in token order), and the state leaving the tile is published;
//   3. every thread continues its run from the state entering it and writes the outputs.
// A tile's leaving state is always fma(A, entering, B) of the same numbers, wherever the look
// back started, so results do not depend on timing.  The grid is launched cooperatively: all
// blocks are resident and take tiles in time order (block b: tiles b, b + grid, ...), so every
// wait is for a tile that a running block has already begun or finished, and each is bounded.
constexpr int kTok = kScanChunk, kWarps = 8, kRun = kTok / kWarps, kCh = 128;
constexpr int kThreads = kWarps * 32;
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
        L.smem = S.per_head > 1 ? lane * 4 : L.c;
        L.row = S.per_head > 1 ? kCh : d;
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
    } else if (lane < rows) {
        const long z = strip / S.per_head;
        const int c0 = (strip % S.per_head) * kCh;
        bulk_load(dst + lane * kCh, src + (z * Ttot + t0 + lane) * d + c0, min(kCh, d - c0) * (int)sizeof(T), bar);
    }
}
__device__ __forceinline__ int strip_channels(const Strips& S, long Z, int d, int strip) {
    if (S.heads > 1) return (int)min((long)S.heads, Z - (long)strip * S.heads) * d;
    return S.per_head == 1 ? d : min(kCh, d - (strip % S.per_head) * kCh);
}

// Which of the tile's tokens begin or end a sequence (bit l: token t0 + l), and, per lane, the
// sequence that token t0 + lane belongs to.
struct Marks {
    uint32_t first, last;
    int n;
};
__device__ __forceinline__ Marks tile_marks(const int* cu, int nseq, int T, int t0) {
    Marks m{t0 == 0 ? 1u : 0u, 0u, 0};
    const int t = t0 + (threadIdx.x & 31);
    if (!cu) {
        if (T - t0 <= kTok) m.last = 1u << (T - 1 - t0);
        return m;
    }
    int lo = 0, hi = nseq;               // the largest n with cu[n] <= t: the sequence that holds t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    m.n = lo;
    m.first = __ballot_sync(0xffffffffu, t < T && cu[lo] == t);
    m.last = __ballot_sync(0xffffffffu, t < T && cu[lo + 1] == t + 1);
    return m;
}

__device__ __forceinline__ int load_acquire(const int* p) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void store_release(int* p, int v) {
    asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// What the tiles of a strip publish, by step (chunk in the direction of the recurrence) and strip:
// flag 1: the tile's (A, B); 2: also the state leaving it, stored as the state entering the next.
enum : int { kAgg = 1, kState = 2 };
struct Chain {
    int* flag;          // [steps][strips]
    float2* agg;        // [steps][strips][128]
    float* state;       // [steps][strips][128]: entering
    int strips, steps;
};

// Threads 0 .. 127 of the block, thread k for channel k of the strip: publishes the tile's (A, B),
// returns the state entering the tile and publishes the one leaving it.  `reset`: A is zero, the
// leaving state does not depend on the entering one; `fresh`: the entering state is not needed.
__device__ __forceinline__ float chain_step(const Chain& C, int step, int strip, float A, float B, bool reset,
                                            bool fresh, bool* dead, int* window, uint32_t* err) {
    const int k = threadIdx.x;
    const size_t at = (size_t)step * C.strips + strip;
    const bool more = step + 1 < C.steps;
    if (reset) {
        if (more) {
            C.state[(at + C.strips) * kCh + k] = B;
            __threadfence();
            bar_sync(1, kCh);
            if (k == 0) store_release(C.flag + at, kState);
        }
        if (fresh) return 0.f;
    } else if (more) {
        C.agg[at * kCh + k] = make_float2(A, B);
        __threadfence();
        bar_sync(1, kCh);
        if (k == 0) store_release(C.flag + at, kAgg);
    }
    if (k < 32) {       // the nearest preceding tile with a state, all tiles after it with (A, B)
        const int p = step - 1 - k;
        const int* flag = C.flag + (size_t)p * C.strips + strip;
        int found = -1;
        uint64_t begin = 0;
        for (;;) {
            const int f = p >= 0 ? load_acquire(flag) : 0;
            const uint32_t state = __ballot_sync(0xffffffffu, f == kState);
            const uint32_t any = __ballot_sync(0xffffffffu, f != 0);
            const int j = __ffs(state) - 1;
            if (j >= 0 && (any & ((1u << j) - 1u)) == (1u << j) - 1u) {
                found = j;
                break;
            }
            if (*dead) break;
            const uint64_t now = globaltimer_ns();
            if (begin == 0) begin = now;
            if (__any_sync(0xffffffffu, now - begin > kWaitNs)) {
                if (k == 0) atomicOr(err, kDevTimeout);
                *dead = true;
                break;
            }
        }
        if (k == 0) *window = found;
    }
    bar_sync(1, kCh);
    const int j = *window;
    float h = 0.f;
    if (j >= 0) {
        h = __ldcg(C.state + (at - (size_t)j * C.strips) * kCh + k);
        const float2* agg = C.agg + (at - (size_t)j * C.strips) * kCh + k;
        for (int i = 0; i < j; i += 8) {
            float2 ab[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (i + u < j) ab[u] = __ldcg(agg + (size_t)(i + u) * C.strips * kCh);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (i + u < j) h = fmaf(ab[u].x, h, ab[u].y);
        }
    }
    if (more && !reset) {
        C.state[(at + C.strips) * kCh + k] = fmaf(A, h, B);
        __threadfence();
        bar_sync(1, kCh);
        if (k == 0) store_release(C.flag + at, kState);
    }
    return h;
}

// Sequences without tokens pass their states through.
__device__ __forceinline__ void pass_empty(const ScanArgs& A, const float* in, float* out) {
    if (!A.cu || !out) return;
    for (int n = blockIdx.x; n < A.nseq; n += gridDim.x)
        if (A.cu[n] == A.cu[n + 1])
            for (long i = threadIdx.x; i < A.Z * A.d; i += blockDim.x)
                out[n * A.Z * A.d + i] = in ? in[n * A.Z * A.d + i] : 0.f;
}

template <typename Tin, bool kShared>
struct FwdSmem {
    static constexpr int kX = kTok * kCh * sizeof(Tin), kG = kShared ? 0 : kTok * kCh * 4;
    static constexpr int kStage = kX + kG;
    static constexpr int kStages = 2;
    static constexpr int kRuns = kWarps * kCh * 4;              // one of A, B of all warps
    static constexpr int kBytes = kStages * kStage + 4 * kRuns + kCh * 4 + 128;
};

template <typename Tin, bool kShared>
__global__ void __launch_bounds__(kThreads, 3) scan_fwd_kernel(ScanArgs P, Chain C, int tiles) {
    using M = FwdSmem<Tin, kShared>;
    extern __shared__ __align__(128) char smem[];
    float* runs = reinterpret_cast<float*>(smem + M::kStages * M::kStage);     // [2][A, B][warp][128]
    float* entering = runs + 4 * kWarps * kCh;
    uint64_t* full = reinterpret_cast<uint64_t*>(entering + kCh);
    int* window = reinterpret_cast<int*>(full + M::kStages);
    const Strips S(P.Z, P.d);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Tin* x = static_cast<const Tin*>(P.x);
    Tin* o = static_cast<Tin*>(P.o);
    if (threadIdx.x == 0) {
        for (int i = 0; i < M::kStages; ++i) mbar_init(full + i, 1);
        fence_mbar_init();
    }
    __syncthreads();
    pass_empty(P, P.S0, P.S_T);
    bool dead = false;

    auto prefetch = [&](int tile, int st) {     // by warp 7
        if (tile >= tiles) return;
        const int strip = tile % S.count, t0 = tile / S.count * kTok, rows = min(kTok, P.T - t0);
        if (lane == 0)
            mbar_arrive_expect_tx(full + st, rows * strip_channels(S, P.Z, P.d, strip) * (int)(sizeof(Tin) + (kShared ? 0 : 4)));
        __syncwarp();
        char* dst = smem + st * M::kStage;
        stage(reinterpret_cast<Tin*>(dst), x, S, P.Z, P.T, P.d, strip, t0, rows, full + st);
        if (!kShared) stage(reinterpret_cast<float*>(dst + M::kX), P.g, S, P.Z, P.T, P.d, strip, t0, rows, full + st);
    };
    if (warp == kWarps - 1)
        for (int i = 0; i < M::kStages; ++i) prefetch(blockIdx.x + i * gridDim.x, i);

    int it = 0;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, ++it) {
        const int strip = tile % S.count, step = tile / S.count, t0 = step * kTok;
        const int st = it % M::kStages;
        const Lane L = lane_of(S, P.Z, P.d, strip, lane);
        const Marks m = tile_marks(P.cu, P.nseq, P.T, t0);
        const int tw = t0 + warp * kRun;        // the run's first token
        float gs[kRun];
        if (kShared) {
#pragma unroll
            for (int i = 0; i < kRun; ++i) gs[i] = L.on && tw + i < P.T ? P.g[L.z * P.T + tw + i] : 0.f;
        }
        if (!mbar_wait(full + st, (it / M::kStages) & 1, dead ? 0 : kWaitNs)) {
            if (!dead && lane == 0) atomicOr(P.err, kDevTimeout);
            dead = true;
        }
        // 1. the run's tokens as h = a h' + b, and the run's (A, B)
        V4 a[kRun], b[kRun], ra = V4{{1.f, 1.f, 1.f, 1.f}}, rb = zero4();
        const Tin* xs = reinterpret_cast<const Tin*>(smem + st * M::kStage) + L.smem + warp * kRun * L.row;
        const float* gt = reinterpret_cast<const float*>(smem + st * M::kStage + M::kX) + L.smem + warp * kRun * L.row;
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            a[i] = V4{{1.f, 1.f, 1.f, 1.f}};
            b[i] = zero4();
            if (L.on && tw + i < P.T) {
                const V4 xv = ld4(xs + i * L.row);
                V4 w;
                if (kShared) {
                    scan_gates(P.rule, gs[i], &a[i].v[0], &w.v[0]);
                    for (int e = 1; e < 4; ++e) a[i].v[e] = a[i].v[0], w.v[e] = w.v[0];
                } else {
                    const V4 gv = ld4(gt + i * L.row);
#pragma unroll
                    for (int e = 0; e < 4; ++e) scan_gates(P.rule, gv.v[e], &a[i].v[e], &w.v[e]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) b[i].v[e] = w.v[e] * xv.v[e];
            }
            if (m.first >> (warp * kRun + i) & 1u) {      // a sequence begins: its own state enters, no other
                const int n = __shfl_sync(0xffffffffu, m.n, warp * kRun + i);
                if (P.S0 && L.on) {
                    const V4 s0 = ld4(P.S0 + ((long)n * P.Z + L.z) * P.d + L.c);
#pragma unroll
                    for (int e = 0; e < 4; ++e) b[i].v[e] = fmaf(a[i].v[e], s0.v[e], b[i].v[e]);
                }
                a[i] = zero4();
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                ra.v[e] *= a[i].v[e];
                rb.v[e] = fmaf(a[i].v[e], rb.v[e], b[i].v[e]);
            }
        }
        float* runA = runs + (it & 1) * 2 * kWarps * kCh;
        float* runB = runA + kWarps * kCh;
        st4(runA + warp * kCh + lane * 4, ra);
        st4(runB + warp * kCh + lane * 4, rb);
        __syncthreads();
        if (warp == kWarps - 1) prefetch(tile + M::kStages * gridDim.x, st);
        // 2. the state entering the tile
        if (threadIdx.x < kCh) {
            const int k = threadIdx.x;
            float A = 1.f, B = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                B = fmaf(runA[w * kCh + k], B, runB[w * kCh + k]);
                A *= runA[w * kCh + k];
            }
            entering[k] = chain_step(C, step, strip, A, B, m.first != 0, m.first & 1u, &dead, window, P.err);
        }
        __syncthreads();
        // 3. the outputs
        V4 h = ld4(entering + lane * 4);
        for (int w = 0; w < warp; ++w) {
            const V4 pa = ld4(runA + w * kCh + lane * 4), pb = ld4(runB + w * kCh + lane * 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) h.v[e] = fmaf(pa.v[e], h.v[e], pb.v[e]);
        }
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) h.v[e] = fmaf(a[i].v[e], h.v[e], b[i].v[e]);
            if (o && L.on && tw + i < P.T) st4(o + (L.z * P.T + tw + i) * P.d + L.c, h);
            if (P.S_T && (m.last >> (warp * kRun + i) & 1u)) {
                const int n = __shfl_sync(0xffffffffu, m.n, warp * kRun + i);
                if (L.on) st4(P.S_T + ((long)n * P.Z + L.z) * P.d + L.c, h);
            }
        }
    }
}

// The reverse pass.  c_t = e^{g_t} G_t flows from token t into t - 1 (dS_T into a sequence's last
// token), G_t = dO_t + c_{t+1}: affine again, c_out = A c_in + R over a run, and the tiles are
// taken from the last to the first.  A tile's own states are put together again from the state
// that the forward kept for it, so no state but one of 32 tokens is ever stored.
template <typename Tin, bool kShared>
struct BwdSmem {
    static constexpr int kX = kTok * kCh * sizeof(Tin), kG = kShared ? 0 : kTok * kCh * 4;
    static constexpr int kStage = 2 * kX + kG;
    static constexpr int kStages = 2;
    static constexpr int kRuns = kWarps * kCh * 4;
    static constexpr int kBytes = kStages * kStage + 8 * kRuns + kCh * 4 + 128;
};

template <typename Tin, bool kShared>
__global__ void __launch_bounds__(kThreads, 2) scan_bwd_kernel(ScanArgs P, Chain C, const float* states, float* parts,
                                                               int tiles) {
    using M = BwdSmem<Tin, kShared>;
    extern __shared__ __align__(128) char smem[];
    float* runs = reinterpret_cast<float*>(smem + M::kStages * M::kStage);     // [2][A, B, Ar, R][warp][128]
    float* entering = runs + 8 * kWarps * kCh;
    uint64_t* full = reinterpret_cast<uint64_t*>(entering + kCh);
    int* window = reinterpret_cast<int*>(full + M::kStages);
    const Strips S(P.Z, P.d);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Tin* x = static_cast<const Tin*>(P.x);
    const Tin* dO = static_cast<const Tin*>(P.dO);
    if (threadIdx.x == 0) {
        for (int i = 0; i < M::kStages; ++i) mbar_init(full + i, 1);
        fence_mbar_init();
    }
    __syncthreads();
    pass_empty(P, P.dST, P.dS0);
    bool dead = false;

    auto prefetch = [&](int tile, int st) {
        if (tile >= tiles) return;
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
    if (warp == kWarps - 1)
        for (int i = 0; i < M::kStages; ++i) prefetch(blockIdx.x + i * gridDim.x, i);

    int it = 0;
    for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, ++it) {
        const int strip = tile % S.count, step = tile / S.count, chunk = C.steps - 1 - step, t0 = chunk * kTok;
        const int st = it % M::kStages;
        const Lane L = lane_of(S, P.Z, P.d, strip, lane);
        const Marks m = tile_marks(P.cu, P.nseq, P.T, t0);
        const int tw = t0 + warp * kRun;
        float gs[kRun];
        if (kShared) {
#pragma unroll
            for (int i = 0; i < kRun; ++i) gs[i] = L.on && tw + i < P.T ? P.g[L.z * P.T + tw + i] : 0.f;
        }
        V4 h = m.first & 1u ? zero4() : ld4(states + ((size_t)chunk * S.count + strip) * kCh + lane * 4);
        if (!mbar_wait(full + st, (it / M::kStages) & 1, dead ? 0 : kWaitNs)) {
            if (!dead && lane == 0) atomicOr(P.err, kDevTimeout);
            dead = true;
        }
        // 1. the run's tokens: a, w, b = w x, e = w' x, u = dO; the forward's and the reverse's (A, B)
        V4 a[kRun], w[kShared ? 1 : kRun], b[kRun], e[kRun], u[kRun];
        float ws[kRun];
        V4 ra = V4{{1.f, 1.f, 1.f, 1.f}}, rb = zero4();
        const Tin* xs = reinterpret_cast<const Tin*>(smem + st * M::kStage) + L.smem + warp * kRun * L.row;
        const Tin* us = reinterpret_cast<const Tin*>(smem + st * M::kStage + M::kX) + L.smem + warp * kRun * L.row;
        const float* gt = reinterpret_cast<const float*>(smem + st * M::kStage + 2 * M::kX) + L.smem + warp * kRun * L.row;
        V4 s0 = zero4();          // the state of the last sequence that begins in the run
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            a[i] = V4{{1.f, 1.f, 1.f, 1.f}};
            b[i] = e[i] = u[i] = zero4();
            ws[i] = 0.f;
            if (!kShared) w[i] = zero4();
            if (L.on && tw + i < P.T) {
                const V4 xv = ld4(xs + i * L.row);
                u[i] = ld4(us + i * L.row);
                if (kShared) {
                    float dw;
                    scan_gates(P.rule, gs[i], &a[i].v[0], &ws[i], &dw);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        a[i].v[j] = a[i].v[0];
                        b[i].v[j] = ws[i] * xv.v[j];
                        e[i].v[j] = dw * xv.v[j];
                    }
                } else {
                    const V4 gv = ld4(gt + i * L.row);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float dw;
                        scan_gates(P.rule, gv.v[j], &a[i].v[j], &w[i].v[j], &dw);
                        b[i].v[j] = w[i].v[j] * xv.v[j];
                        e[i].v[j] = dw * xv.v[j];
                    }
                }
            }
            const bool first = m.first >> (warp * kRun + i) & 1u;
            if (first) {
                const int n = __shfl_sync(0xffffffffu, m.n, warp * kRun + i);
                s0 = P.S0 && L.on ? ld4(P.S0 + ((long)n * P.Z + L.z) * P.d + L.c) : zero4();
                ra = zero4();
                rb = s0;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                ra.v[j] *= a[i].v[j];
                rb.v[j] = fmaf(a[i].v[j], rb.v[j], b[i].v[j]);
            }
        }
        float* runA = runs + (it & 1) * 4 * kWarps * kCh;
        float* runB = runA + kWarps * kCh;
        float* revA = runB + kWarps * kCh;
        float* revB = revA + kWarps * kCh;
        st4(runA + warp * kCh + lane * 4, ra);
        st4(runB + warp * kCh + lane * 4, rb);
        ra = V4{{1.f, 1.f, 1.f, 1.f}};
        rb = zero4();
#pragma unroll
        for (int i = kRun - 1; i >= 0; --i) {
            if (m.last >> (warp * kRun + i) & 1u) {
                const int n = __shfl_sync(0xffffffffu, m.n, warp * kRun + i);
                ra = zero4();
                rb = P.dST && L.on ? ld4(P.dST + ((long)n * P.Z + L.z) * P.d + L.c) : zero4();
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                ra.v[j] *= a[i].v[j];
                rb.v[j] = a[i].v[j] * (u[i].v[j] + rb.v[j]);
            }
        }
        st4(revA + warp * kCh + lane * 4, ra);
        st4(revB + warp * kCh + lane * 4, rb);
        __syncthreads();
        if (warp == kWarps - 1) prefetch(tile + M::kStages * gridDim.x, st);
        // 2. what flows into the tile from behind
        if (threadIdx.x < kCh) {
            const int k = threadIdx.x;
            float A = 1.f, B = 0.f;
#pragma unroll
            for (int q = kWarps - 1; q >= 0; --q) {
                B = fmaf(revA[q * kCh + k], B, revB[q * kCh + k]);
                A *= revA[q * kCh + k];
            }
            const bool at_end = t0 + kTok >= P.T || (m.last >> (kTok - 1) & 1u);   // nothing flows in
            entering[k] = chain_step(C, step, strip, A, B, m.last != 0, at_end, &dead, window, P.err);
        }
        // 3. the states before the run's tokens: e becomes a h' + w' x
        for (int q = 0; q < warp; ++q) {
            const V4 pa = ld4(runA + q * kCh + lane * 4), pb = ld4(runB + q * kCh + lane * 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) h.v[j] = fmaf(pa.v[j], h.v[j], pb.v[j]);
        }
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            if (m.first >> (warp * kRun + i) & 1u) {
                const int n = __shfl_sync(0xffffffffu, m.n, warp * kRun + i);
                h = P.S0 && L.on ? ld4(P.S0 + ((long)n * P.Z + L.z) * P.d + L.c) : zero4();
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float ah = a[i].v[j] * h.v[j];
                e[i].v[j] += ah;
                h.v[j] = ah + b[i].v[j];
            }
        }
        __syncthreads();
        // 4. the gradients
        V4 c = ld4(entering + lane * 4);
        for (int q = kWarps - 1; q > warp; --q) {
            const V4 pa = ld4(revA + q * kCh + lane * 4), pb = ld4(revB + q * kCh + lane * 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) c.v[j] = fmaf(pa.v[j], c.v[j], pb.v[j]);
        }
#pragma unroll
        for (int i = kRun - 1; i >= 0; --i) {
            const int t = tw + i;
            if (m.last >> (warp * kRun + i) & 1u) {
                const int n = __shfl_sync(0xffffffffu, m.n, warp * kRun + i);
                c = P.dST && L.on ? ld4(P.dST + ((long)n * P.Z + L.z) * P.d + L.c) : zero4();
            }
            V4 dx, dg;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float G = u[i].v[j] + c.v[j];
                dx.v[j] = (kShared ? ws[i] : w[kShared ? 0 : i].v[j]) * G;
                dg.v[j] = G * e[i].v[j];
                c.v[j] = a[i].v[j] * G;
            }
            const bool live = L.on && t < P.T;
            if (live) {
                st4(P.dx + (L.z * P.T + t) * P.d + L.c, dx);
                if (!kShared) st4(P.dg + (L.z * P.T + t) * P.d + L.c, dg);
            }
            if (kShared) {      // over the head's channels; a part of a wide head leaves a partial sum
                float sum = live ? (dg.v[0] + dg.v[1]) + (dg.v[2] + dg.v[3]) : 0.f;
                for (int off = S.heads > 1 ? S.dv / 2 : 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                if (live && (S.heads > 1 ? lane % S.dv == 0 : lane == 0)) {
                    if (S.per_head == 1) P.dg[L.z * P.T + t] = sum;
                    else parts[((long)(strip % S.per_head) * P.Z + L.z) * P.T + t] = sum;
                }
            }
            if (P.dS0 && (m.first >> (warp * kRun + i) & 1u)) {
                const int n = __shfl_sync(0xffffffffu, m.n, warp * kRun + i);
                if (L.on) st4(P.dS0 + ((long)n * P.Z + L.z) * P.d + L.c, c);
            }
        }
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
    const V4 xv = ld4(x + row + j);
    V4 gv;
    if (gw == 1) gv.v[0] = gv.v[1] = gv.v[2] = gv.v[3] = g[(long)n * H + j / d];
    else gv = ld4(g + row + j);
    V4 h = from ? ld4(from + j) : zero4();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, w;
        scan_gates(rule, gv.v[i], &a, &w);
        h.v[i] = fmaf(a, h.v[i], w * xv.v[i]);
    }
    st4(to + j, h);
    st4(o + row + j, h);
}

}  // namespace

static size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
static long scan_steps(int T) { return ((long)T + kTok - 1) / kTok; }

size_t scan_states_bytes(long Z, int T, int d) {
    return up256((size_t)scan_steps(T) * Strips(Z, d).count * kCh * sizeof(float));
}
// flags and (A, B) of every tile; backward: also the flows between tiles, and the partial sums of
// a shared decay's gradient where a head is wider than a strip
size_t scan_scratch_bytes(long Z, int T, int d, int gw, bool backward) {
    const Strips S(Z, d);
    const size_t tiles = (size_t)scan_steps(T) * S.count;
    size_t n = up256(tiles * sizeof(int)) + tiles * kCh * sizeof(float2);
    if (backward) {
        n += up256(tiles * kCh * sizeof(float));
        if (gw == 1 && S.per_head > 1) n += up256((size_t)S.per_head * Z * T * sizeof(float));
    }
    return n;
}

namespace {

// Launches with every block resident at once (at most one per tile), after clearing the flags.
template <typename Kernel, typename... Args>
cudaError_t launch_tiles(Kernel kernel, int smem, std::atomic<int>* resident, const Chain& C, long tiles,
                         cudaStream_t stream, Args... args) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int most = dev < 64 ? resident[dev].load(std::memory_order_relaxed) : 0;
    if (most == 0) {
        int sms = 0, per = 0;
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
        if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
        if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, kThreads, smem)) != cudaSuccess) return e;
        most = sms * per;
        if (dev < 64) resident[dev].store(most, std::memory_order_relaxed);
    }
    if (C.steps > 1 &&
        (e = cudaMemsetAsync(C.flag, 0, (size_t)C.steps * C.strips * sizeof(int), stream)) != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles < most ? tiles : most));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = C.steps > 1 ? 1 : 0;      // blocks wait for one another only across steps
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

Chain scan_chain(const ScanArgs& a, float* states, long* tiles) {
    const Strips S(a.Z, a.d);
    Chain C;
    C.strips = S.count;
    C.steps = (int)scan_steps(a.T);
    *tiles = (long)C.steps * C.strips;
    C.flag = static_cast<int*>(a.scratch);
    C.agg = reinterpret_cast<float2*>(static_cast<char*>(a.scratch) + up256((size_t)*tiles * sizeof(int)));
    C.state = states ? states : reinterpret_cast<float*>(C.agg + (size_t)*tiles * kCh);
    return C;
}

template <typename Tin, bool kShared>
cudaError_t launch_fwd(const ScanArgs& a, cudaStream_t stream) {
    static std::atomic<int> resident[64];
    long tiles;
    const Chain C = scan_chain(a, a.E, &tiles);
    if (tiles >= (1l << 31)) return cudaErrorInvalidValue;
    return launch_tiles(scan_fwd_kernel<Tin, kShared>, FwdSmem<Tin, kShared>::kBytes, resident, C, tiles, stream, a, C,
                        (int)tiles);
}

template <typename Tin, bool kShared>
cudaError_t launch_bwd(const ScanArgs& a, cudaStream_t stream) {
    static std::atomic<int> resident[64];
    long tiles;
    const Chain C = scan_chain(a, nullptr, &tiles);
    if (tiles >= (1l << 31)) return cudaErrorInvalidValue;
    const int per_head = Strips(a.Z, a.d).per_head;
    float* parts = reinterpret_cast<float*>(reinterpret_cast<char*>(C.state) + up256((size_t)tiles * kCh * sizeof(float)));
    cudaError_t e = launch_tiles(scan_bwd_kernel<Tin, kShared>, BwdSmem<Tin, kShared>::kBytes, resident, C, tiles, stream,
                                 a, C, (const float*)a.E, parts, (int)tiles);
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
