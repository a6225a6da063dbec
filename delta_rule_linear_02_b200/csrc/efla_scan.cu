// efla_scan.cu -- the per-channel gated linear recurrence: forward, backward, one token.
#include "efla_kernels.h"
#include "efla_pages.cuh"
#include "efla_scan.cuh"

namespace efla {
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

// One warp per (sequence, stream), token by token; lane l carries channels 4 l .. 4 l + 3.
template <typename Tin, bool kShared>
__global__ void __launch_bounds__(32) scan_fwd_kernel(ScanArgs A) {
    const int n = blockIdx.x / A.Z;
    const long z = blockIdx.x % A.Z;
    const int y0 = A.cu ? A.cu[n] : 0, y1 = A.cu ? A.cu[n + 1] : A.T;
    const Tin* x = static_cast<const Tin*>(A.x);
    Tin* o = static_cast<Tin*>(A.o);
    for (int c = threadIdx.x * 4; c < A.d; c += 128) {
        const long s = ((long)n * A.Z + z) * A.d + c;
        V4 h = A.S0 ? ld4(A.S0 + s) : zero4();
        for (int t = y0; t < y1; ++t) {
            const long row = z * A.T + t, at = row * A.d + c;
            if (A.E && t % kScanChunk == 0) st4(A.E + ((long)(t / kScanChunk) * A.Z + z) * A.d + c, h);
            const V4 xv = ld4(x + at);
            V4 gv;
            if (kShared) gv.v[0] = gv.v[1] = gv.v[2] = gv.v[3] = A.g[row];
            else gv = ld4(A.g + at);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float a, w;
                scan_gates(A.rule, gv.v[i], &a, &w);
                h.v[i] = fmaf(a, h.v[i], w * xv.v[i]);
            }
            if (o) st4(o + at, h);
        }
        if (A.S_T) st4(A.S_T + s, h);
    }
}

// The reverse pass: per chunk of 32 tokens the states are recomputed from the saved one.
template <typename Tin, bool kShared>
__global__ void __launch_bounds__(32) scan_bwd_kernel(ScanArgs A) {
    const int n = blockIdx.x / A.Z;
    const long z = blockIdx.x % A.Z;
    const int y0 = A.cu ? A.cu[n] : 0, y1 = A.cu ? A.cu[n + 1] : A.T;
    const Tin* x = static_cast<const Tin*>(A.x);
    const Tin* dO = static_cast<const Tin*>(A.dO);
    for (int c0 = 0; c0 < A.d; c0 += 128) {
        const int c = c0 + threadIdx.x * 4;
        const bool on = c < A.d;
        const long s = ((long)n * A.Z + z) * A.d + c;
        V4 flow = on && A.dST ? ld4(A.dST + s) : zero4();
        for (int end = y1; end > y0;) {
            const int chunk = (end - 1) / kScanChunk;
            const int begin = max(y0, chunk * kScanChunk);
            V4 prev[kScanChunk];
            V4 h = zero4();
            if (on) {
                if (begin == y0) h = A.S0 ? ld4(A.S0 + s) : zero4();
                else h = ld4(A.E + ((long)chunk * A.Z + z) * A.d + c);
            }
            for (int t = begin; t < end; ++t) {
                prev[t - begin] = h;
                if (!on) continue;
                const long row = z * A.T + t;
                const V4 xv = ld4(x + row * A.d + c);
                const V4 gv = kShared ? V4{{A.g[row], A.g[row], A.g[row], A.g[row]}} : ld4(A.g + row * A.d + c);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float a, w;
                    scan_gates(A.rule, gv.v[i], &a, &w);
                    h.v[i] = fmaf(a, h.v[i], w * xv.v[i]);
                }
            }
            for (int t = end - 1; t >= begin; --t) {
                const long row = z * A.T + t, at = row * A.d + c;
                float sum = 0.f;
                if (on) {
                    const V4 xv = ld4(x + at), dv = ld4(dO + at);
                    const V4 gv = kShared ? V4{{A.g[row], A.g[row], A.g[row], A.g[row]}} : ld4(A.g + at);
                    V4 dxv, dgv;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float a, w, dw;
                        scan_gates(A.rule, gv.v[i], &a, &w, &dw);
                        const float G = dv.v[i] + flow.v[i];
                        dxv.v[i] = w * G;
                        dgv.v[i] = G * fmaf(a, prev[t - begin].v[i], dw * xv.v[i]);
                        flow.v[i] = a * G;
                        sum += dgv.v[i];
                    }
                    st4(A.dx + at, dxv);
                    if (!kShared) st4(A.dg + at, dgv);
                }
                if (kShared) {
                    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                    if (threadIdx.x == 0) A.dg[row] = c0 == 0 ? sum : A.dg[row] + sum;
                }
            }
            end = begin;
        }
        if (on && A.dS0) st4(A.dS0 + s, flow);
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

size_t scan_states_bytes(long Z, int T, int d) {
    return (size_t)((T + kScanChunk - 1) / kScanChunk) * Z * d * sizeof(float);
}
size_t scan_scratch_bytes(long, int, int, int, bool) { return 0; }

cudaError_t launch_scan_fwd(const ScanArgs& a, bool bf16, cudaStream_t stream) {
    const unsigned grid = (unsigned)(a.nseq * a.Z);
    if (bf16) {
        if (a.gw == 1) scan_fwd_kernel<__nv_bfloat16, true><<<grid, 32, 0, stream>>>(a);
        else scan_fwd_kernel<__nv_bfloat16, false><<<grid, 32, 0, stream>>>(a);
    } else {
        if (a.gw == 1) scan_fwd_kernel<float, true><<<grid, 32, 0, stream>>>(a);
        else scan_fwd_kernel<float, false><<<grid, 32, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

cudaError_t launch_scan_bwd(const ScanArgs& a, bool bf16, cudaStream_t stream) {
    const unsigned grid = (unsigned)(a.nseq * a.Z);
    if (bf16) {
        if (a.gw == 1) scan_bwd_kernel<__nv_bfloat16, true><<<grid, 32, 0, stream>>>(a);
        else scan_bwd_kernel<__nv_bfloat16, false><<<grid, 32, 0, stream>>>(a);
    } else {
        if (a.gw == 1) scan_bwd_kernel<float, true><<<grid, 32, 0, stream>>>(a);
        else scan_bwd_kernel<float, false><<<grid, 32, 0, stream>>>(a);
    }
    return cudaGetLastError();
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
