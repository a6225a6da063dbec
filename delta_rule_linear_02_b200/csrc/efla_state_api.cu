// efla_state_api.cu -- the C ABI of the per-channel gated recurrence, the state cache's pages and
// the decode steps on them (include/efla.h): argument checks, then launches.
#include <stdint.h>

#include "../../include/efla.h"
#include "efla_kernels.h"
#include "efla_pages.cuh"
#include "efla_scan.cuh"

namespace {

constexpr size_t kHeader = 256;   // device error word + reserved

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

struct Buf {
    const void* p;
    size_t n;
};
bool overlaps(const Buf& a, const Buf& b) {
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + b.n && b0 < a0 + a.n;
}
// Every output apart from every input and from the other outputs.
bool disjoint(const Buf* outs, int no, const Buf* ins, int ni) {
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j)
            if (overlaps(outs[i], ins[j])) return false;
        for (int j = i + 1; j < no; ++j)
            if (overlaps(outs[i], outs[j])) return false;
    }
    return true;
}

size_t elem_size(int dtype) { return dtype == EFLA_DTYPE_BF16 ? 2 : 4; }
int from_cuda(cudaError_t e) { return e == cudaSuccess ? EFLA_OK : EFLA_ERR_CUDA; }

int check_scan_shape(int B, int H, int T, int d, int g_width, int dtype) {
    if (B < 0 || H < 0 || T < 0 || d <= 0) return EFLA_ERR_INVALID_ARG;
    if (dtype != EFLA_DTYPE_F32 && dtype != EFLA_DTYPE_BF16) return EFLA_ERR_UNSUPPORTED;
    if (g_width != 1 && g_width != d) return EFLA_ERR_INVALID_ARG;
    if (d > 4096 || (d * elem_size(dtype)) % 16 != 0 || T > (1 << 30)) return EFLA_ERR_UNSUPPORTED;
    if ((long long)B * H * ((d + 31) / 32) >= (1ll << 31)) return EFLA_ERR_UNSUPPORTED;      // strips of 32 channels
    return EFLA_OK;
}

// Offsets of a packed batch: 0, non-decreasing, T in the end.
bool good_offsets(const int* cu, int N, int T) {
    if (N < 1 || cu[0] != 0 || cu[N] != T) return false;
    for (int n = 0; n < N; ++n)
        if (cu[n + 1] < cu[n]) return false;
    return true;
}

// Where a call's kernels find the offsets: in its launches' arguments, or copied to `to`.  A captured copy would
// read the host array again on every replay, so it is refused from memory that is not pinned.
int place_offsets(const int* cu, int B, bool copy, char* to, cudaStream_t s, efla::ScanArgs* a) {
    a->by_value = B <= efla::kScanInline;
    a->cu = a->by_value ? cu : reinterpret_cast<const int*>(to);
    if (a->by_value || !copy) return EFLA_OK;
    cudaStreamCaptureStatus capture;
    if (cudaStreamIsCapturing(s, &capture) != cudaSuccess) return EFLA_ERR_CUDA;
    if (capture != cudaStreamCaptureStatusNone) {
        cudaPointerAttributes at;
        if (cudaPointerGetAttributes(&at, cu) != cudaSuccess) return EFLA_ERR_CUDA;
        if (at.type != cudaMemoryTypeHost) return EFLA_ERR_INVALID_ARG;
    }
    return cudaMemcpyAsync(to, cu, ((size_t)B + 1) * sizeof(int), cudaMemcpyHostToDevice, s) == cudaSuccess ? EFLA_OK
                                                                                                           : EFLA_ERR_CUDA;
}

size_t cu_bytes(int B, bool packed) { return packed ? (((size_t)B + 1) * sizeof(int) + 255) & ~(size_t)255 : 0; }

}  // namespace

extern "C" {

size_t efla_scan_workspace_bytes(int B, int H, int T, int d, int g_width, int dtype, int packed) {
    if (check_scan_shape(B, H, T, d, g_width, dtype) != EFLA_OK) return 0;
    const long Z = packed ? H : (long)B * H;
    return kHeader + cu_bytes(B, packed) + efla::scan_states_bytes(Z, T, d) +
           efla::scan_scratch_bytes(Z, T, d, g_width, false);
}

size_t efla_scan_backward_workspace_bytes(int B, int H, int T, int d, int g_width, int dtype, int packed, int saved) {
    if (check_scan_shape(B, H, T, d, g_width, dtype) != EFLA_OK) return 0;
    const long Z = packed ? H : (long)B * H;
    const size_t back = kHeader + efla::scan_scratch_bytes(Z, T, d, g_width, true);
    return saved ? back : back + efla_scan_workspace_bytes(B, H, T, d, g_width, dtype, packed);
}

int efla_scan_fwd(const void* x, const float* g, const int* cu_seqlens, const float* S0, void* o, float* S_T, int B,
                  int H, int T, int d, int g_width, int dtype, int rule, void* workspace, size_t workspace_bytes,
                  efla_stream_t stream) {
    const int st = check_scan_shape(B, H, T, d, g_width, dtype);
    if (st != EFLA_OK) return st;
    if (rule != EFLA_RULE_EXACT && rule != EFLA_RULE_EULER) return EFLA_ERR_INVALID_ARG;
    if (B == 0 || H == 0) return EFLA_OK;
    const bool packed = cu_seqlens != nullptr;
    if (packed && !good_offsets(cu_seqlens, B, T)) return EFLA_ERR_INVALID_ARG;
    const long Z = packed ? H : (long)B * H;
    const size_t ns = (size_t)B * H * d * sizeof(float), n = (size_t)Z * T * d;
    if ((S0 && !aligned16(S0)) || (S_T && !aligned16(S_T))) return EFLA_ERR_INVALID_ARG;
    const size_t need = efla_scan_workspace_bytes(B, H, T, d, g_width, dtype, packed);
    if (!workspace || !aligned16(workspace) || workspace_bytes < need) return EFLA_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    const Buf ins[3] = {{x, n * elem_size(dtype)}, {g, (size_t)Z * T * g_width * sizeof(float)}, {S0, ns}};
    const Buf outs[3] = {{o, n * elem_size(dtype)}, {workspace, workspace_bytes}, {S_T, ns}};
    if (!disjoint(outs, 2, ins, 3) || overlaps(outs[0], outs[2]) || overlaps(outs[1], outs[2]) ||
        overlaps(outs[2], ins[0]) || overlaps(outs[2], ins[1]) || (S_T != S0 && overlaps(outs[2], ins[2])))
        return EFLA_ERR_INVALID_ARG;
    if (T == 0) {   // no token: the states pass through, and nothing can go wrong on the device
        if (cudaMemsetAsync(workspace, 0, sizeof(uint32_t), s) != cudaSuccess) return EFLA_ERR_CUDA;
        if (!S_T || S_T == S0) return EFLA_OK;
        return from_cuda(S0 ? cudaMemcpyAsync(S_T, S0, ns, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(S_T, 0, ns, s));
    }
    if (!x || !g || !o || !aligned16(x) || !aligned16(g) || !aligned16(o)) return EFLA_ERR_INVALID_ARG;
    char* ws = static_cast<char*>(workspace);
    efla::ScanArgs a;
    const int placed = packed ? place_offsets(cu_seqlens, B, true, ws + kHeader, s, &a) : EFLA_OK;
    if (placed != EFLA_OK) return placed;
    a.x = x;
    a.g = g;
    a.nseq = packed ? B : 1;
    a.Z = Z;
    a.T = T;
    a.d = d;
    a.gw = g_width;
    a.rule = rule;
    a.S0 = S0;
    a.o = o;
    a.S_T = S_T;
    a.E = reinterpret_cast<float*>(ws + kHeader + cu_bytes(B, packed));
    a.scratch = ws + kHeader + cu_bytes(B, packed) + efla::scan_states_bytes(Z, T, d);
    a.err = reinterpret_cast<uint32_t*>(ws);
    return from_cuda(efla::launch_scan_fwd(a, dtype == EFLA_DTYPE_BF16, s));
}

int efla_scan_backward(const void* x, const float* g, const int* cu_seqlens, const float* S0, const void* dO,
                       const float* dS_T, float* dx, float* dg, float* dS0, int B, int H, int T, int d, int g_width,
                       int dtype, int rule, const void* saved, size_t saved_bytes, void* workspace,
                       size_t workspace_bytes, efla_stream_t stream) {
    const int st = check_scan_shape(B, H, T, d, g_width, dtype);
    if (st != EFLA_OK) return st;
    if (rule != EFLA_RULE_EXACT && rule != EFLA_RULE_EULER) return EFLA_ERR_INVALID_ARG;
    if (B == 0 || H == 0) return EFLA_OK;
    const bool packed = cu_seqlens != nullptr;
    if (packed && !good_offsets(cu_seqlens, B, T)) return EFLA_ERR_INVALID_ARG;
    const long Z = packed ? H : (long)B * H;
    const size_t ns = (size_t)B * H * d * sizeof(float), n = (size_t)Z * T * d;
    const size_t ng = (size_t)Z * T * g_width * sizeof(float);
    if ((S0 && !aligned16(S0)) || (dS_T && !aligned16(dS_T)) || (dS0 && !aligned16(dS0))) return EFLA_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    const size_t fwd = efla_scan_workspace_bytes(B, H, T, d, g_width, dtype, packed);
    const size_t need = efla_scan_backward_workspace_bytes(B, H, T, d, g_width, dtype, packed, saved != nullptr);
    if (!workspace || !aligned16(workspace) || workspace_bytes < need) return EFLA_ERR_INVALID_ARG;
    if (saved && (!aligned16(saved) || saved_bytes < fwd)) return EFLA_ERR_INVALID_ARG;
    const Buf ins[6] = {{x, n * elem_size(dtype)}, {g, ng}, {S0, ns}, {dO, n * elem_size(dtype)}, {dS_T, ns},
                        {saved, saved ? saved_bytes : 0}};
    const Buf outs[4] = {{dx, n * sizeof(float)}, {dg, ng}, {dS0, ns}, {workspace, workspace_bytes}};
    if (!disjoint(outs, 4, ins, 6)) return EFLA_ERR_INVALID_ARG;
    if (T == 0) {
        if (cudaMemsetAsync(workspace, 0, sizeof(uint32_t), s) != cudaSuccess) return EFLA_ERR_CUDA;
        if (!dS0) return EFLA_OK;
        return from_cuda(dS_T ? cudaMemcpyAsync(dS0, dS_T, ns, cudaMemcpyDeviceToDevice, s)
                              : cudaMemsetAsync(dS0, 0, ns, s));
    }
    if (!x || !g || !dO || !dx || !dg || !aligned16(x) || !aligned16(g) || !aligned16(dO) || !aligned16(dx) ||
        !aligned16(dg))
        return EFLA_ERR_INVALID_ARG;
    char* ws = static_cast<char*>(workspace);
    const bool bf16 = dtype == EFLA_DTYPE_BF16;
    // without saved states the workspace holds a forward's in front of the backward's
    char* states = saved ? static_cast<char*>(const_cast<void*>(saved)) : ws;
    efla::ScanArgs a;
    const int placed = packed ? place_offsets(cu_seqlens, B, !saved, states + kHeader, s, &a) : EFLA_OK;
    if (placed != EFLA_OK) return placed;
    a.x = x;
    a.g = g;
    a.nseq = packed ? B : 1;
    a.Z = Z;
    a.T = T;
    a.d = d;
    a.gw = g_width;
    a.rule = rule;
    a.S0 = S0;
    a.E = reinterpret_cast<float*>(states + kHeader + cu_bytes(B, packed));
    a.err = reinterpret_cast<uint32_t*>(ws);
    if (!saved) {   // the states alone: a forward without outputs
        a.scratch = ws + kHeader + cu_bytes(B, packed) + efla::scan_states_bytes(Z, T, d);
        const cudaError_t e = efla::launch_scan_fwd(a, bf16, s);
        if (e != cudaSuccess) return EFLA_ERR_CUDA;
        a.clear_err = false;
    }
    a.scratch = ws + (saved ? 0 : fwd) + kHeader;
    a.dO = dO;
    a.dST = dS_T;
    a.dx = dx;
    a.dg = dg;
    a.dS0 = dS0;
    return from_cuda(efla::launch_scan_bwd(a, bf16, s));
}

// ---------------------------------------------------------------- one token
static int check_step_shape(int N, int H, int d, int g_width, int dtype, int rule) {
    if (rule != EFLA_RULE_EXACT && rule != EFLA_RULE_EULER) return EFLA_ERR_INVALID_ARG;
    const int st = check_scan_shape(N, H, 1, d, g_width, dtype);
    if (st != EFLA_OK) return st;
    if ((long long)H * d >= (1ll << 30) || (long long)N * (((long long)H * d + 1023) / 1024) >= (1ll << 31))
        return EFLA_ERR_UNSUPPORTED;
    return EFLA_OK;
}

int efla_scan_step(const void* x, const float* g, float* S, void* o, int N, int H, int d, int g_width, int dtype,
                   int rule, efla_stream_t stream) {
    const int st = check_step_shape(N, H, d, g_width, dtype, rule);
    if (st != EFLA_OK) return st;
    if (N == 0 || H == 0) return EFLA_OK;
    if (!x || !g || !S || !o || !aligned16(x) || !aligned16(g) || !aligned16(S) || !aligned16(o))
        return EFLA_ERR_INVALID_ARG;
    const size_t n = (size_t)N * H * d;
    const Buf ins[2] = {{x, n * elem_size(dtype)}, {g, (size_t)N * H * g_width * sizeof(float)}};
    const Buf outs[2] = {{S, n * sizeof(float)}, {o, n * elem_size(dtype)}};
    if (!disjoint(outs, 2, ins, 2)) return EFLA_ERR_INVALID_ARG;
    return from_cuda(efla::launch_scan_step(x, g, S, o, N, H, d, g_width, dtype == EFLA_DTYPE_BF16, rule, nullptr,
                                            (cudaStream_t)stream));
}

// The cache's block and pool: sizes and alignment; *pool_span: bytes from `pool` to its last page's data.
static int check_pages(const void* pages, int n_pages, int n_slots, const void* pool, size_t page_bytes,
                       size_t data_bytes, size_t* pool_span) {
    if (n_pages < 1 || n_slots < 1 || n_pages > (1 << 28) || n_slots > (1 << 28)) return EFLA_ERR_INVALID_ARG;
    if (!pages || !aligned16(pages)) return EFLA_ERR_INVALID_ARG;
    *pool_span = 0;
    if (!pool) return EFLA_OK;
    if (!aligned16(pool) || page_bytes % 16 || data_bytes % 16 || data_bytes == 0 || page_bytes < data_bytes)
        return EFLA_ERR_INVALID_ARG;
    if (page_bytes > ((size_t)1 << 46) / (size_t)n_pages) return EFLA_ERR_UNSUPPORTED;
    *pool_span = (size_t)(n_pages - 1) * page_bytes + data_bytes;
    return EFLA_OK;
}

static int paged_rows(const void* pages, int n_pages, int n_slots, const void* pool, size_t page_bytes,
                      size_t data_bytes, const int* slots, const int* source, size_t* pool_span, efla::PagedRows* rows) {
    const int st = check_pages(pages, n_pages, n_slots, pool, page_bytes, data_bytes, pool_span);
    if (st != EFLA_OK) return st;
    if (!pool || !slots || !aligned4(slots) || (source && !aligned4(source))) return EFLA_ERR_INVALID_ARG;
    const efla::PagesBlock b = efla::pages_block(const_cast<void*>(pages), n_pages, n_slots);
    rows->table = b.table;
    rows->err = b.err;
    rows->slots = slots;
    rows->source = source;
    rows->n_pages = n_pages;
    rows->n_slots = n_slots;
    rows->page_bytes = page_bytes;
    return EFLA_OK;
}

int efla_scan_step_paged(const void* x, const float* g, void* pages, int n_pages, int n_slots, float* pool,
                         size_t page_bytes, const int* slots, const int* source, void* o, int N, int H, int d,
                         int g_width, int dtype, int rule, efla_stream_t stream) {
    int st = check_step_shape(N, H, d, g_width, dtype, rule);
    if (st != EFLA_OK) return st;
    if (N == 0 || H == 0) return EFLA_OK;
    efla::PagedRows rows;
    size_t span = 0;
    st = paged_rows(pages, n_pages, n_slots, pool, page_bytes, (size_t)H * d * sizeof(float), slots, source, &span, &rows);
    if (st != EFLA_OK) return st;
    if (!x || !g || !o || !aligned16(x) || !aligned16(g) || !aligned16(o)) return EFLA_ERR_INVALID_ARG;
    const size_t n = (size_t)N * H * d, nl = (size_t)N * sizeof(int);
    const Buf ins[4] = {{x, n * elem_size(dtype)}, {g, (size_t)N * H * g_width * sizeof(float)}, {slots, nl}, {source, nl}};
    const Buf outs[3] = {{pool, span}, {o, n * elem_size(dtype)}, {pages, efla_pages_bytes(n_pages, n_slots)}};
    if (!disjoint(outs, 3, ins, 4)) return EFLA_ERR_INVALID_ARG;
    return from_cuda(efla::launch_scan_step(x, g, pool, o, N, H, d, g_width, dtype == EFLA_DTYPE_BF16, rule, &rows,
                                            (cudaStream_t)stream));
}

int efla_recurrent_step_paged(const void* q, const void* k, const void* v, const void* beta, const float* g,
                              void* pages, int n_pages, int n_slots, float* pool, size_t page_bytes, const int* slots,
                              const int* source, void* o, int N, int H, int d_k, int d_v, int dtype, int rule,
                              efla_stream_t stream) {
    if (N < 0 || H < 0 || d_k <= 0 || d_v <= 0) return EFLA_ERR_INVALID_ARG;
    if (rule != EFLA_RULE_EXACT && rule != EFLA_RULE_EULER) return EFLA_ERR_INVALID_ARG;
    if (dtype != EFLA_DTYPE_F32 && dtype != EFLA_DTYPE_BF16) return EFLA_ERR_UNSUPPORTED;
    if (d_k != d_v || (d_k != 64 && d_k != 128)) return EFLA_ERR_UNSUPPORTED;
    if ((long long)N * H * (d_k / 32) >= (1ll << 31)) return EFLA_ERR_UNSUPPORTED;
    if (N == 0 || H == 0) return EFLA_OK;
    efla::PagedRows rows;
    size_t span = 0;
    const int st = paged_rows(pages, n_pages, n_slots, pool, page_bytes, (size_t)H * d_k * d_v * sizeof(float), slots,
                              source, &span, &rows);
    if (st != EFLA_OK) return st;
    if (!q || !k || !v || !beta || !o || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(beta) ||
        !aligned16(o) || (g && !aligned16(g)))
        return EFLA_ERR_INVALID_ARG;
    const size_t es = elem_size(dtype), NH = (size_t)N * H, nl = (size_t)N * sizeof(int);
    const Buf ins[7] = {{q, NH * d_k * es}, {k, NH * d_k * es}, {v, NH * d_v * es}, {beta, NH * es},
                        {g, NH * sizeof(float)}, {slots, nl}, {source, nl}};
    const Buf outs[3] = {{pool, span}, {o, NH * d_v * es}, {pages, efla_pages_bytes(n_pages, n_slots)}};
    if (!disjoint(outs, 3, ins, 7)) return EFLA_ERR_INVALID_ARG;
    return from_cuda(efla::launch_decode_paged(q, k, v, beta, g, pool, o, N, H, d_k, dtype == EFLA_DTYPE_BF16, rule,
                                               rows, (cudaStream_t)stream));
}

// ---------------------------------------------------------------- pages
size_t efla_pages_bytes(int n_pages, int n_slots) {
    if (n_pages < 1 || n_slots < 1 || n_pages > (1 << 28) || n_slots > (1 << 28)) return 0;
    return efla::pages_words(n_pages, n_slots) * sizeof(int);
}

int efla_pages_init(void* pages, size_t pages_bytes, int n_pages, int n_slots, efla_stream_t stream) {
    size_t span;
    const int st = check_pages(pages, n_pages, n_slots, nullptr, 0, 0, &span);
    if (st != EFLA_OK) return st;
    if (pages_bytes < efla_pages_bytes(n_pages, n_slots)) return EFLA_ERR_INVALID_ARG;
    return from_cuda(efla::launch_pages_init(efla::pages_block(pages, n_pages, n_slots), (cudaStream_t)stream));
}

int efla_pages_free(void* pages, int n_pages, int n_slots, const int* slots, int n, efla_stream_t stream) {
    size_t span;
    const int st = check_pages(pages, n_pages, n_slots, nullptr, 0, 0, &span);
    if (st != EFLA_OK) return st;
    if (n < 0 || n > (1 << 28)) return EFLA_ERR_INVALID_ARG;
    if (n == 0) return EFLA_OK;
    if (!slots || !aligned4(slots) ||
        overlaps(Buf{slots, (size_t)n * sizeof(int)}, Buf{pages, efla_pages_bytes(n_pages, n_slots)}))
        return EFLA_ERR_INVALID_ARG;
    return from_cuda(efla::launch_pages_free(efla::pages_block(pages, n_pages, n_slots), slots, n, (cudaStream_t)stream));
}

static int check_lists(const void* pages, int n_pages, int n_slots, const void* pool, size_t span, const int* source,
                       const int* dest, int n) {
    const size_t nl = (size_t)n * sizeof(int), nb = efla_pages_bytes(n_pages, n_slots);
    if (!source || !dest || !aligned4(source) || !aligned4(dest)) return EFLA_ERR_INVALID_ARG;
    const Buf ins[2] = {{source, nl}, {dest, nl}};
    const Buf outs[2] = {{pages, nb}, {pool, span}};
    return disjoint(outs, 2, ins, 2) ? EFLA_OK : EFLA_ERR_INVALID_ARG;
}

int efla_pages_fork(void* pages, int n_pages, int n_slots, void* pool, size_t page_bytes, size_t data_bytes,
                    const int* source, const int* dest, int n, efla_stream_t stream) {
    size_t span;
    int st = check_pages(pages, n_pages, n_slots, pool, page_bytes, data_bytes, &span);
    if (st != EFLA_OK) return st;
    if (n < 0 || n > (1 << 28)) return EFLA_ERR_INVALID_ARG;
    if (n == 0) return EFLA_OK;
    if ((st = check_lists(pages, n_pages, n_slots, pool, span, source, dest, n)) != EFLA_OK) return st;
    return from_cuda(efla::launch_pages_fork(efla::pages_block(pages, n_pages, n_slots), pool, page_bytes, data_bytes,
                                             source, dest, n, (cudaStream_t)stream));
}

int efla_pages_copy(void* pages, int n_pages, int n_slots, void* pool, size_t page_bytes, size_t data_bytes,
                    const int* source, const int* dest, int n, efla_stream_t stream) {
    size_t span;
    int st = check_pages(pages, n_pages, n_slots, pool, page_bytes, data_bytes, &span);
    if (st != EFLA_OK) return st;
    if (!pool || n < 0) return EFLA_ERR_INVALID_ARG;
    if (n > efla::kPagesCopyMax) return EFLA_ERR_UNSUPPORTED;
    if (n == 0) return EFLA_OK;
    if ((st = check_lists(pages, n_pages, n_slots, pool, span, source, dest, n)) != EFLA_OK) return st;
    return from_cuda(efla::launch_pages_copy(efla::pages_block(pages, n_pages, n_slots), pool, page_bytes, data_bytes,
                                             source, dest, n, (cudaStream_t)stream));
}

int efla_pages_compact(void* pages, int n_pages, int n_slots, void* pool, size_t page_bytes, size_t data_bytes,
                       efla_stream_t stream) {
    size_t span;
    const int st = check_pages(pages, n_pages, n_slots, pool, page_bytes, data_bytes, &span);
    if (st != EFLA_OK) return st;
    if (!pool || overlaps(Buf{pages, efla_pages_bytes(n_pages, n_slots)}, Buf{pool, span})) return EFLA_ERR_INVALID_ARG;
    return from_cuda(efla::launch_pages_compact(efla::pages_block(pages, n_pages, n_slots), pool, page_bytes,
                                                data_bytes, (cudaStream_t)stream));
}

static int pages_rows(void* pages, int n_pages, int n_slots, void* pool, size_t page_bytes, void* rows,
                      size_t row_bytes, const int* slots, int n, bool write, efla_stream_t stream) {
    size_t span;
    const int st = check_pages(pages, n_pages, n_slots, pool, page_bytes, row_bytes, &span);
    if (st != EFLA_OK) return st;
    if (!pool || n < 0) return EFLA_ERR_INVALID_ARG;
    if (n == 0) return EFLA_OK;
    if (!rows || !aligned16(rows) || !slots || !aligned4(slots)) return EFLA_ERR_INVALID_ARG;
    if ((long long)n * (long long)((row_bytes + 4095) / 4096) >= (1ll << 31)) return EFLA_ERR_UNSUPPORTED;
    const Buf all[4] = {{pages, efla_pages_bytes(n_pages, n_slots)}, {pool, span}, {rows, (size_t)n * row_bytes},
                        {slots, (size_t)n * sizeof(int)}};
    if (!disjoint(all, 4, nullptr, 0)) return EFLA_ERR_INVALID_ARG;
    return from_cuda(efla::launch_pages_rows(efla::pages_block(pages, n_pages, n_slots), pool, page_bytes, rows,
                                             row_bytes, slots, n, write, (cudaStream_t)stream));
}

int efla_pages_write(void* pages, int n_pages, int n_slots, void* pool, size_t page_bytes, const void* rows,
                     size_t row_bytes, const int* slots, int n, efla_stream_t stream) {
    return pages_rows(pages, n_pages, n_slots, pool, page_bytes, const_cast<void*>(rows), row_bytes, slots, n, true,
                      stream);
}

int efla_pages_read(void* pages, int n_pages, int n_slots, const void* pool, size_t page_bytes, void* rows,
                    size_t row_bytes, const int* slots, int n, efla_stream_t stream) {
    return pages_rows(pages, n_pages, n_slots, const_cast<void*>(pool), page_bytes, rows, row_bytes, slots, n, false,
                      stream);
}

int efla_pages_status(void* pages, int clear, efla_stream_t stream) {
    if (!pages || !aligned16(pages)) return EFLA_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    uint32_t word = 0;
    if (cudaMemcpyAsync(&word, pages, sizeof(word), cudaMemcpyDeviceToHost, s) != cudaSuccess) return EFLA_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return EFLA_ERR_CUDA;
    if (clear && (cudaMemsetAsync(pages, 0, sizeof(word), s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess))
        return EFLA_ERR_CUDA;
    if (word & efla::kDevTimeout) return EFLA_ERR_TIMEOUT;
    if (word & efla::kPagesBadSlot) return EFLA_ERR_SLOT;
    return word & efla::kPagesFull ? EFLA_ERR_FULL : EFLA_OK;
}

}  // extern "C"
