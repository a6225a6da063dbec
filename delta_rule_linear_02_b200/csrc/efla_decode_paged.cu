// efla_decode_paged.cu -- one recurrent (decode) token for the rows of a batch whose states lie in
// the pages of a state cache: the update of the dense step (the exact flow, gated or not),
//     r = k^T S, p = q^T S, c = q.k,  w = d alpha r - abar v,  S <- d S - k w^T,  o = d p - c w,
// d = e^g (1 without g), with S read from one page and written to the same or another one.
// Column j of the new state needs column j of the old one alone: a block owns 32 columns of one
// head and passes them through registers once.
#include "efla_kernels.h"
#include "efla_pages.cuh"
#include "efla_scan.cuh"

namespace efla {
namespace {
constexpr int kCols = 32;
constexpr int kThreads = 256;

template <typename Tin, int D>
__global__ void __launch_bounds__(kThreads) decode_paged_kernel(const Tin* __restrict__ q, const Tin* __restrict__ k,
                                                                const Tin* __restrict__ v,
                                                                const Tin* __restrict__ beta,
                                                                const float* __restrict__ g, char* pool,
                                                                Tin* __restrict__ o, int N, int H, int rule,
                                                                PagedRows P) {
    constexpr int RPT = D / 32;
    constexpr int SLICES = D / kCols;
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

template <typename Tin, int D>
cudaError_t launch_t(const void* q, const void* k, const void* v, const void* beta, const float* g, float* pool,
                     void* o, int N, int H, int rule, const PagedRows& paged, cudaStream_t stream) {
    const long blocks = (long)N * H * (D / kCols);
    decode_paged_kernel<Tin, D><<<(unsigned)blocks, kThreads, 0, stream>>>(
        (const Tin*)q, (const Tin*)k, (const Tin*)v, (const Tin*)beta, g, reinterpret_cast<char*>(pool), (Tin*)o, N, H,
        rule, paged);
    return cudaGetLastError();
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
