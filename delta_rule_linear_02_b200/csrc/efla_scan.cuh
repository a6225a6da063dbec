// efla_scan.cuh -- the per-channel gated linear recurrence: gates and launchers (internal).
//
//     h_t = a_t h_{t-1} + w_t x_t,   o_t = h_t,   a_t = e^{g_t},
//
// the vector-state sibling of the gated flow: dh/dtau = g h + x over the token's unit interval
// has the exact flow w = phi(g) = (e^g - 1) / g (phi(0) = 1); the Euler rule writes w = 1.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "efla_common.cuh"

namespace efla {

// Pairs of fp32 in one instruction (the FMA pipe takes two per lane and issue).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
          "l"(reinterpret_cast<unsigned long long&>(c)));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long&>(d))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float fast_rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// a = e^g, w = phi(g) and, for the backward pass, w' = phi'(g) in fp32, two at a time.
// For |g| < 1 all come from v(g) = (phi(g) - 1) / g = sum_n g^n / (n + 2)!, as its Chebyshev
// series on [-1, 1] cut after degree 6 (4.7e-8 off at most): w = 1 + g v, a = 1 + g w, and from phi' = (a - w) / g,
// w' = w - v.  Nothing cancels near 0, and a long memory's a is as good as its rounding.
// Elsewhere a is 2^(g log2 e), w = (a - 1) / g and w' = (a - w) / g by their definitions
// (|a - 1| >= 0.63, |a - w| >= 0.26).  Relative errors in u = 2^-24, by their roundings and as measured over 4 million
// values of g in each range: for |g| < 1 a 5 u (4.9), w 6 u (2.6), w' 24 u (10.5).  Elsewhere a (2.8 + 1.25 |g|) u, from
// the power's 2^-22.5 and its rounded argument (|g| < 2: 3.5, 8: 8.2, 80: 62.7); for g <= -1 that belongs to a memory of a
// token or two, and w stays below 6 u (3.4), w' below 24 u (12).  For g >= 1 w and w' have a's error and 3 u.
// g = -inf gives a = w = w' = 0: the token forgets everything and writes nothing.
__device__ __forceinline__ void scan_gates1(int rule, float g, float* a, float* w) {
    float v = 2.5358645e-05f;
    v = fmaf(v, g, 2.0329201e-04f);
    v = fmaf(v, g, 1.3885395e-03f);
    v = fmaf(v, g, 8.3308842e-03f);
    v = fmaf(v, g, 4.1666737e-02f);
    v = fmaf(v, g, 1.6666697e-01f);
    v = fmaf(v, g, 0.5f);
    const float w0 = fmaf(g, v, 1.0f), a0 = fmaf(g, w0, 1.0f);
    const float a1 = fast_exp2(g * 1.44269504f), w1 = (a1 - 1.0f) * fast_rcp(g);
    const bool near = fabsf(g) < 1.0f;
    *a = near ? a0 : a1;
    *w = rule == kRuleEuler ? 1.0f : near ? w0 : w1;
}
// The forward takes them one by one (its register budget leaves no room for the paired
// coefficients: 444 heads of 128, T 2048 run in 152 us, with pairs in 159), the backward in pairs
// (296 heads: 210 us, one by one 215).
template <bool kSlope>
__device__ __forceinline__ void scan_gates2(int rule, float2 g, float2* a, float2* w, float2* dw) {
    if constexpr (!kSlope) {
        scan_gates1(rule, g.x, &a->x, &w->x);
        scan_gates1(rule, g.y, &a->y, &w->y);
        return;
    }
    float2 v = both(2.5358645e-05f);
    v = fma2(v, g, both(2.0329201e-04f));
    v = fma2(v, g, both(1.3885395e-03f));
    v = fma2(v, g, both(8.3308842e-03f));
    v = fma2(v, g, both(4.1666737e-02f));
    v = fma2(v, g, both(1.6666697e-01f));
    v = fma2(v, g, both(0.5f));
    const float2 w0 = fma2(g, v, both(1.0f)), a0 = fma2(g, w0, both(1.0f));
    const float2 t = mul2(g, both(1.44269504f)), r = make_float2(fast_rcp(g.x), fast_rcp(g.y));
    const float2 a1 = make_float2(fast_exp2(t.x), fast_exp2(t.y));
    const float2 w1 = mul2(add2(a1, both(-1.0f)), r);
    const bool sx = fabsf(g.x) < 1.0f, sy = fabsf(g.y) < 1.0f;
    *a = make_float2(sx ? a0.x : a1.x, sy ? a0.y : a1.y);
    *w = make_float2(sx ? w0.x : w1.x, sy ? w0.y : w1.y);
    const float2 d0 = fma2(v, both(-1.0f), w0), d1 = mul2(fma2(w1, both(-1.0f), a1), r);
    *dw = make_float2(sx ? d0.x : d1.x, sy ? d0.y : d1.y);
    if (rule == kRuleEuler) *w = both(1.0f), *dw = both(0.0f);
}

// The kernels of this family may be set up while the one before them in their stream still runs: launched by
// launch_after, a kernel touches no global memory before after_previous(), which returns when the previous kernel has
// ended and its writes are seen.  (No pointer of these kernels is __restrict__: loads marked as never changing might be
// moved before it.)  With `next` it lets the next one be set up in turn while it runs: up to a us less for each call of a
// run of them (a server's tick 27.8 -> 26.4 us, nine rows' delta step 6.7 -> 6.3, the short prompt 5.0 -> 4.5 on the device).
__device__ __forceinline__ void after_previous(bool next = true) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (next) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <typename... Params, typename... Args>
cudaError_t launch_after(void (*kernel)(Params...), unsigned grid, unsigned threads, size_t smem, cudaStream_t stream,
                         Args... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
    if (e != cudaSuccess) cudaGetLastError();      // it is answered, not left for a later call
    return e;
}

// Streams [Z][T][d] (dense: Z = B*H, one sequence each; packed: Z = H, sequences cu[n] ..
// cu[n+1] of every stream); states [(n * Z + z) * d], n = 0 for dense batches.
// Offsets of up to kScanInline sequences travel as a kernel argument: no copy before the launch (packed
// requests: about 6 us less), and a graph holds them itself.
constexpr int kScanInline = 255;
struct ScanArgs {
    const void* x = nullptr;
    const float* g = nullptr;       // [Z][T][gw], gw = d or 1
    const int* cu = nullptr;        // null: dense
    bool by_value = false;          // cu is a host array, handed over with the launch; else a device one
    int nseq = 1;                   // packed sequences (1 for dense)
    long Z = 0;
    int T = 0, d = 0, gw = 0, rule = 0;
    const float* S0 = nullptr;
    void* o = nullptr;              // forward; null: states only
    float* S_T = nullptr;
    float* E = nullptr;             // the state entering each tile, as efla_scan.cu lays them out (kept by the forward)
    // backward
    const void* dO = nullptr;
    const float* dST = nullptr;
    float* dx = nullptr;
    float* dg = nullptr;
    float* dS0 = nullptr;
    void* scratch = nullptr;
    uint32_t* err = nullptr;
    bool next = false;              // the next kernel may be set up while this one runs (the launcher's choice)
    bool clear_err = true;          // the first kernel of a call forgets the last call's errors
};
size_t scan_states_bytes(long Z, int T, int d);
size_t scan_scratch_bytes(long Z, int T, int d, int gw, bool backward);
cudaError_t launch_scan_fwd(const ScanArgs& a, bool bf16, cudaStream_t stream);
cudaError_t launch_scan_bwd(const ScanArgs& a, bool bf16, cudaStream_t stream);

// one token: row n's state at S + n * H * d, or, paged, in the page of slot slots[n]
struct PagedRows {
    const int* table = nullptr;     // slot -> page
    const int* slots = nullptr;     // [N]: the row's slot, -1: no row
    const int* source = nullptr;    // [N] or null: the slot the entering state is read from (-1: zero)
    int n_pages = 0, n_slots = 0;
    size_t page_bytes = 0;
    uint32_t* err = nullptr;
};
cudaError_t launch_scan_step(const void* x, const float* g, float* S, void* o, int N, int H, int d, int gw, bool bf16,
                             int rule, const PagedRows* paged, cudaStream_t stream);
cudaError_t launch_decode_paged(const void* q, const void* k, const void* v, const void* beta, const float* g,
                                float* pool, void* o, int N, int H, int D, bool bf16, int rule,
                                const PagedRows& paged, cudaStream_t stream);

}  // namespace efla
