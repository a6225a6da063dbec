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

// a = e^g, w = phi(g) and, for the backward pass, w' = phi'(g) in fp32.
// For |g| < 1/2 all three come from v(g) = (phi(g) - 1) / g = sum_n g^n / (n + 2)!, cut after
// g^6 / 8! (the rest is below g^7 / 9! < 2.2e-8): w = 1 + g v and, from phi' = (e^g - phi) / g
// with e^g = 1 + g phi, w' = w - v, which has no cancellation near 0.  Elsewhere w = (a - 1) / g
// and w' = (a - w) / g by their definitions (|a - 1| >= 0.39 and |a - w| >= 0.18: few digits
// cancel, and none for long decays).
// g = -inf gives a = w = w' = 0: the token forgets everything and writes nothing.
__device__ __forceinline__ float scan_v(float g) {
    float v = 1.0f / 40320.0f;
    v = fmaf(v, g, 1.0f / 5040.0f);
    v = fmaf(v, g, 1.0f / 720.0f);
    v = fmaf(v, g, 1.0f / 120.0f);
    v = fmaf(v, g, 1.0f / 24.0f);
    v = fmaf(v, g, 1.0f / 6.0f);
    return fmaf(v, g, 0.5f);
}
__device__ __forceinline__ void scan_gates(int rule, float g, float* a, float* w) {
    *a = expf(g);
    if (rule == kRuleEuler) {
        *w = 1.0f;
        return;
    }
    const float near0 = fmaf(g, scan_v(g), 1.0f);
    const float far = __fdividef(*a - 1.0f, g);
    *w = fabsf(g) < 0.5f ? near0 : far;
}
__device__ __forceinline__ void scan_gates(int rule, float g, float* a, float* w, float* dw) {
    *a = expf(g);
    if (rule == kRuleEuler) {
        *w = 1.0f;
        *dw = 0.0f;
        return;
    }
    const bool small = fabsf(g) < 0.5f;
    const float v = scan_v(g), near0 = fmaf(g, v, 1.0f);
    const float far = __fdividef(*a - 1.0f, g);
    *w = small ? near0 : far;
    *dw = small ? near0 - v : __fdividef(*a - far, g);
}

// Streams [Z][T][d] (dense: Z = B*H, one sequence each; packed: Z = H, sequences cu[n] ..
// cu[n+1] of every stream); states [(n * Z + z) * d], n = 0 for dense batches.
constexpr int kScanChunk = 32;      // tokens between two saved states
struct ScanArgs {
    const void* x = nullptr;
    const float* g = nullptr;       // [Z][T][gw], gw = d or 1
    const int* cu = nullptr;        // device, or null (dense)
    int nseq = 1;                   // packed sequences (1 for dense)
    long Z = 0;
    int T = 0, d = 0, gw = 0, rule = 0;
    const float* S0 = nullptr;
    void* o = nullptr;              // forward; null: states only
    float* S_T = nullptr;
    float* E = nullptr;             // [ceil(T / 32)][Z][d]: the state before token 32 c (written by the forward)
    // backward
    const void* dO = nullptr;
    const float* dST = nullptr;
    float* dx = nullptr;
    float* dg = nullptr;
    float* dS0 = nullptr;
    void* scratch = nullptr;
    uint32_t* err = nullptr;
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
