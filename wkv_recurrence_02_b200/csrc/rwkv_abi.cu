// rwkv_abi.cu -- the extern "C" boundary of libwkv.so (declared in include/rwkv_wkv.h).
//
// Host-side argument validation (before any CUDA call), kernel selection, the
// thread-local stream and the device status word.  Every step of the recurrences
// runs in the CUDA kernels of the other files; there is no CPU fallback.
#include "rwkv_wkv.h"
#include "wkv_internal.cuh"

#include <mutex>
#include <stdio.h>
#include <string.h>

namespace {

thread_local cudaStream_t tl_stream = nullptr;
thread_local int tl_wkv6_algo = RWKV_WKV6_AUTO;
thread_local int tl_wkv6_segments = 0;
thread_local char tl_err[256] = "";

// The library's only device memory: one status word per device, allocated statically.
__device__ int g_device_status = 0;

constexpr int kMaxDevices = 64;
std::mutex g_status_mu;
int *g_status_ptr[kMaxDevices] = {nullptr};

int fail(int code, const char *fmt, const char *detail = "")
{
    snprintf(tl_err, sizeof(tl_err), fmt, detail);
    return code;
}

int cuda_fail(cudaError_t e, const char *where)
{
    snprintf(tl_err, sizeof(tl_err), "%s: %s", where, cudaGetErrorString(e));
    return RWKV_ERR_CUDA;
}

// Device address of the status word on the current device (looked up once per device).
int status_word(int **out)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return fail(RWKV_ERR_CUDA, "device index out of range%s");
    std::lock_guard<std::mutex> lock(g_status_mu);
    if (!g_status_ptr[dev]) {
        void *p = nullptr;
        e = cudaGetSymbolAddress(&p, g_device_status);
        if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(status)");
        g_status_ptr[dev] = static_cast<int *>(p);
    }
    *out = g_status_ptr[dev];
    return RWKV_OK;
}

// ---- validation helpers -----------------------------------------------------------

bool mul_ok(int64_t a, int64_t b, int64_t *out)
{
    if (a < 0 || b < 0) return false;
    if (a != 0 && b > INT64_MAX / 4 / a) return false;  // keep byte counts representable
    *out = a * b;
    return true;
}

struct Span {
    const void *p;
    int64_t bytes;
};

bool overlap(Span a, Span b)
{
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    uintptr_t a0 = (uintptr_t)a.p, a1 = a0 + (uintptr_t)a.bytes;
    uintptr_t b0 = (uintptr_t)b.p, b1 = b0 + (uintptr_t)b.bytes;
    return a0 < b1 && b0 < a1;
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// ---- WKV-4 -------------------------------------------------------------------------

int wkv4_entry(int64_t B, int64_t T, int64_t C, const float *w, const float *u,
               const void *k, const void *v, const float *s0, void *y, float *sT,
               bool bf16, bool with_state)
{
    tl_err[0] = 0;
    if (B < 0 || T < 0 || C < 0) return fail(RWKV_ERR_SHAPE, "negative size%s");
    int64_t BT, n, ns;
    if (!mul_ok(B, T, &BT) || !mul_ok(BT, C, &n) || !mul_ok(B * 3, C, &ns))
        return fail(RWKV_ERR_SHAPE, "size product overflows%s");
    const int64_t esz = bf16 ? 2 : 4;
    const bool want_state = with_state && sT != nullptr;
    if (n == 0 && !(want_state && ns > 0)) return RWKV_OK;
    if (n > 0 && (!k || !v || !y)) return fail(RWKV_ERR_NULL, "k, v and y must be non-null%s");
    if (C > 0 && B > 0 && (!w || !u)) return fail(RWKV_ERR_NULL, "w and u must be non-null%s");
    const void *ptrs[] = {w, u, k, v, y, s0, sT};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return fail(RWKV_ERR_ALIGN, "tensor pointers must be 16-byte aligned%s");
    Span sy{y, n * esz}, sk{k, n * esz}, sv{v, n * esz}, sw{w, C * 4}, su{u, C * 4};
    Span ss0{s0, with_state ? ns * 4 : 0}, ssT{sT, with_state ? ns * 4 : 0};
    if (overlap(sy, sk) || overlap(sy, sv) || overlap(sy, sw) || overlap(sy, su) ||
        overlap(sy, ss0) || overlap(sy, ssT))
        return fail(RWKV_ERR_ALIAS, "y overlaps another tensor%s");
    if (with_state && sT) {
        if (overlap(ssT, sk) || overlap(ssT, sv) || overlap(ssT, sw) || overlap(ssT, su))
            return fail(RWKV_ERR_ALIAS, "sT overlaps an input%s");
        if (s0 && s0 != sT && overlap(ssT, ss0))
            return fail(RWKV_ERR_ALIAS, "sT partially overlaps s0%s");
    }
    int *status = nullptr;
    int rc = status_word(&status);
    if (rc) return rc;
    wkv::Wkv4Args a{B, T, C, w, u, k, v, with_state ? s0 : nullptr, y,
                    with_state ? sT : nullptr, bf16, status};
    cudaError_t e = wkv::wkv4_launch(a, tl_stream);
    if (e != cudaSuccess) return cuda_fail(e, "wkv4 launch");
    return RWKV_OK;
}

// ---- WKV-6 -------------------------------------------------------------------------

int wkv6_entry(int64_t B, int64_t T, int64_t H, int64_t N, const void *r, const void *k,
               const void *v, const void *w, const float *u, const float *s0, void *y,
               float *sT, bool bf16, const void *g = nullptr, const float *ln_w = nullptr,
               const float *ln_b = nullptr, float eps = 0.f, bool gated = false, bool omega = false)
{
    tl_err[0] = 0;
    if (B < 0 || T < 0 || H < 0 || N < 0) return fail(RWKV_ERR_SHAPE, "negative size%s");
    int64_t BT, BTH, n, BH, ns;
    if (!mul_ok(B, T, &BT) || !mul_ok(BT, H, &BTH) || !mul_ok(BTH, N, &n) ||
        !mul_ok(B, H, &BH) || !mul_ok(BH, N * N, &ns))
        return fail(RWKV_ERR_SHAPE, "size product overflows%s");
    if (n == 0 && !(sT && ns > 0)) return RWKV_OK;
    if (N != 64) return fail(RWKV_ERR_UNSUPPORTED, "head size N must be 64%s");
    const int64_t esz = bf16 ? 2 : 4;
    if (n > 0 && (!r || !k || !v || !w || !y))
        return fail(RWKV_ERR_NULL, "r, k, v, w and y must be non-null%s");
    if (BH > 0 && !u) return fail(RWKV_ERR_NULL, "u must be non-null%s");
    if (gated) {
        if (n > 0 && !g) return fail(RWKV_ERR_NULL, "g must be non-null%s");
        if (H * N > 0 && (!ln_w || !ln_b)) return fail(RWKV_ERR_NULL, "ln_w and ln_b must be non-null%s");
        if (!(eps >= 0.f) || eps > 3.0e38f) return fail(RWKV_ERR_ARG, "eps must be finite and >= 0%s");
    }
    const void *ptrs[] = {r, k, v, w, u, s0, y, sT, g, ln_w, ln_b};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return fail(RWKV_ERR_ALIGN, "tensor pointers must be 16-byte aligned%s");
    Span sy{y, n * esz}, sr{r, n * esz}, sk{k, n * esz}, sv{v, n * esz}, sw{w, n * esz};
    Span su{u, H * N * 4}, ss0{s0, ns * 4}, ssT{sT, ns * 4};
    Span sg{g, n * esz}, slw{ln_w, H * N * 4}, slb{ln_b, H * N * 4};
    const Span ins[] = {sr, sk, sv, sw, su, sg, slw, slb};
    for (const Span &s : ins)
        if (overlap(sy, s)) return fail(RWKV_ERR_ALIAS, "y overlaps an input%s");
    if (overlap(sy, ss0) || overlap(sy, ssT)) return fail(RWKV_ERR_ALIAS, "y overlaps a state%s");
    if (sT) {
        for (const Span &s : ins)
            if (overlap(ssT, s)) return fail(RWKV_ERR_ALIAS, "sT overlaps an input%s");
        if (s0 && s0 != sT && overlap(ssT, ss0))
            return fail(RWKV_ERR_ALIAS, "sT partially overlaps s0%s");
    }
    int *status = nullptr;
    int rc = status_word(&status);
    if (rc) return rc;
    if (T == 0) {  // nothing to scan: sT = s0, or the zero state
        if (!sT || sT == s0) return RWKV_OK;
        cudaError_t e = s0 ? cudaMemcpyAsync(sT, s0, ns * 4, cudaMemcpyDeviceToDevice, tl_stream)
                           : cudaMemsetAsync(sT, 0, ns * 4, tl_stream);
        return e == cudaSuccess ? RWKV_OK : cuda_fail(e, "T=0 state copy");
    }
    wkv::Wkv6Args a{B, T, H, N, r, k, v, w, u, s0, y, sT, bf16, status, tl_wkv6_segments};
    a.omega = omega;
    cudaError_t e;
    if (gated) {  // fused output stage: chunked for T > 1, decode for T == 1
        a.g = g;
        a.ln_w = ln_w;
        a.ln_b = ln_b;
        a.eps = eps;
        e = T > 1 ? wkv::wkv6_chunked_launch(a, tl_stream) : wkv::wkv6_decode_launch(a, tl_stream);
        if (e != cudaSuccess) return cuda_fail(e, "wkv6 gated launch");
        return RWKV_OK;
    }
    int algo = tl_wkv6_algo;
    if (algo == RWKV_WKV6_SERIAL || !bf16)
        e = (T == 1 && algo != RWKV_WKV6_SERIAL) ? wkv::wkv6_decode_launch(a, tl_stream)
                                                 : wkv::wkv6_serial_launch(a, tl_stream);
    else if (algo == RWKV_WKV6_CHUNKED || T > 1)
        e = wkv::wkv6_chunked_launch(a, tl_stream);
    else
        e = wkv::wkv6_decode_launch(a, tl_stream);
    if (e != cudaSuccess) return cuda_fail(e, "wkv6 launch");
    return RWKV_OK;
}

// ---- WKV-6 backward -----------------------------------------------------------------

int wkv6_bwd_sizes(int64_t B, int64_t T, int64_t H, int64_t N, int64_t *n, int64_t *ns, int64_t *hn)
{
    if (B < 0 || T < 0 || H < 0 || N < 0) return fail(RWKV_ERR_SHAPE, "negative size%s");
    int64_t BT, BTH, BH;
    if (!mul_ok(B, T, &BT) || !mul_ok(BT, H, &BTH) || !mul_ok(BTH, N, n) || !mul_ok(B, H, &BH) ||
        !mul_ok(BH, N * N, ns) || !mul_ok(H, N, hn))
        return fail(RWKV_ERR_SHAPE, "size product overflows%s");
    // workspace: per (b, h), a 64 x 64 fp32 checkpoint every 8 tokens and 64 floats
    const int64_t nblk = (T + 7) / 8;
    int64_t per_head, cells;
    if (!mul_ok(nblk, 4096, &per_head) || !mul_ok(BH, per_head + 64, &cells))
        return fail(RWKV_ERR_SHAPE, "workspace size overflows%s");
    return RWKV_OK;
}

int wkv6_bwd_entry(int64_t B, int64_t T, int64_t H, int64_t N, const void *r, const void *k, const void *v,
                   const void *w, const float *u, const float *s0, const void *dy, const float *dsT, float *dr,
                   float *dk, float *dv, float *dw, float *du, float *ds0, void *workspace, size_t wbytes,
                   bool bf16, bool omega)
{
    tl_err[0] = 0;
    int64_t n, ns, hn;
    int rc = wkv6_bwd_sizes(B, T, H, N, &n, &ns, &hn);
    if (rc) return rc;
    if (n == 0 && hn == 0 && !(ds0 && ns > 0)) return RWKV_OK;
    if (N != 64) return fail(RWKV_ERR_UNSUPPORTED, "head size N must be 64%s");
    if (n > 0 && (!r || !k || !v || !w || !dy))
        return fail(RWKV_ERR_NULL, "r, k, v, w (or omega) and dy must be non-null%s");
    if (n > 0 && (!dr || !dk || !dv || !dw)) return fail(RWKV_ERR_NULL, "dr, dk, dv and dw must be non-null%s");
    if (hn > 0 && (!u || !du)) return fail(RWKV_ERR_NULL, "u and du must be non-null%s");
    const size_t need = n > 0 ? wkv::wkv6_backward_workspace_bytes(B, T, H) : 0;
    if (need > 0 && !workspace) return fail(RWKV_ERR_NULL, "workspace must be non-null%s");
    if (wbytes < need) {
        snprintf(tl_err, sizeof(tl_err), "workspace holds %zu bytes; this call needs %zu", wbytes, need);
        return RWKV_ERR_ARG;
    }
    const void *ptrs[] = {r, k, v, w, u, s0, dy, dsT, dr, dk, dv, dw, du, ds0, workspace};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return fail(RWKV_ERR_ALIGN, "tensor pointers must be 16-byte aligned%s");
    const int64_t esz = bf16 ? 2 : 4;
    const Span ins[] = {{r, n * esz}, {k, n * esz}, {v, n * esz}, {w, n * esz}, {u, hn * 4}, {s0, ns * 4},
                        {dy, n * esz}, {dsT, ns * 4}};
    const Span outs[] = {{dr, n * 4}, {dk, n * 4}, {dv, n * 4}, {dw, n * 4}, {du, hn * 4},
                         {ds0, ns * 4}, {workspace, static_cast<int64_t>(need)}};
    const int n_outs = sizeof(outs) / sizeof(outs[0]);
    for (int a = 0; a < n_outs; ++a) {
        for (const Span &x : ins) {
            // ds0 may be the very same array as dsT (in place); any other overlap is refused
            if (outs[a].p == ds0 && x.p == dsT && ds0 == dsT) continue;
            if (overlap(outs[a], x)) return fail(RWKV_ERR_ALIAS, "a gradient or the workspace overlaps an input%s");
        }
        for (int c = a + 1; c < n_outs; ++c)
            if (overlap(outs[a], outs[c])) return fail(RWKV_ERR_ALIAS, "two outputs overlap%s");
    }
    int *status = nullptr;
    rc = status_word(&status);
    if (rc) return rc;
    cudaError_t e = cudaSuccess;
    if (n == 0) {  // no token: du = 0, ds0 = dsT (or 0)
        if (hn > 0) e = cudaMemsetAsync(du, 0, hn * 4, tl_stream);
        if (e == cudaSuccess && ds0 && ns > 0 && ds0 != dsT)
            e = dsT ? cudaMemcpyAsync(ds0, dsT, ns * 4, cudaMemcpyDeviceToDevice, tl_stream)
                    : cudaMemsetAsync(ds0, 0, ns * 4, tl_stream);
        return e == cudaSuccess ? RWKV_OK : cuda_fail(e, "wkv6 backward without tokens");
    }
    wkv::Wkv6BwdArgs a{B, T, H, N, r, k, v, w, u, s0, dy, dsT, dr, dk, dv, dw, du, ds0, workspace, bf16, omega};
    a.chunked = bf16 && tl_wkv6_algo != RWKV_WKV6_SERIAL;
    a.status = status;
    e = wkv::wkv6_backward_launch(a, tl_stream);
    if (e != cudaSuccess) return cuda_fail(e, "wkv6 backward launch");
    return RWKV_OK;
}

// Allocation-free WKV-6 (bf16): same validation as wkv6_entry, chunked kernel only, the
// split's scratch in the library's fixed device array.
int wkv6_noalloc_entry(int64_t B, int64_t T, int64_t H, int64_t N, const void *r, const void *k,
                       const void *v, const void *w, const float *u, const float *s0, void *y,
                       float *sT, int segments)
{
    tl_err[0] = 0;
    if (segments < 0) return fail(RWKV_ERR_ARG, "segments must be >= 0%s");
    if (B < 0 || T < 0 || H < 0 || N < 0) return fail(RWKV_ERR_SHAPE, "negative size%s");
    int64_t BT, BTH, n, BH, ns;
    if (!mul_ok(B, T, &BT) || !mul_ok(BT, H, &BTH) || !mul_ok(BTH, N, &n) ||
        !mul_ok(B, H, &BH) || !mul_ok(BH, N * N, &ns))
        return fail(RWKV_ERR_SHAPE, "size product overflows%s");
    if (n == 0 && !(sT && ns > 0)) return RWKV_OK;
    if (N != 64) return fail(RWKV_ERR_UNSUPPORTED, "head size N must be 64%s");
    if (n > 0 && (!r || !k || !v || !w || !y))
        return fail(RWKV_ERR_NULL, "r, k, v, w and y must be non-null%s");
    if (BH > 0 && !u) return fail(RWKV_ERR_NULL, "u must be non-null%s");
    const void *ptrs[] = {r, k, v, w, u, s0, y, sT};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return fail(RWKV_ERR_ALIGN, "tensor pointers must be 16-byte aligned%s");
    Span sy{y, n * 2}, sr{r, n * 2}, sk{k, n * 2}, sv{v, n * 2}, sw{w, n * 2};
    Span su{u, H * N * 4}, ss0{s0, ns * 4}, ssT{sT, ns * 4};
    const Span ins[] = {sr, sk, sv, sw, su};
    for (const Span &s : ins)
        if (overlap(sy, s)) return fail(RWKV_ERR_ALIAS, "y overlaps an input%s");
    if (overlap(sy, ss0) || overlap(sy, ssT)) return fail(RWKV_ERR_ALIAS, "y overlaps a state%s");
    if (sT) {
        for (const Span &s : ins)
            if (overlap(ssT, s)) return fail(RWKV_ERR_ALIAS, "sT overlaps an input%s");
        if (s0 && s0 != sT && overlap(ssT, ss0))
            return fail(RWKV_ERR_ALIAS, "sT partially overlaps s0%s");
    }
    int *status = nullptr;
    int rc = status_word(&status);
    if (rc) return rc;
    if (T == 0) {
        if (!sT || sT == s0) return RWKV_OK;
        cudaError_t e = s0 ? cudaMemcpyAsync(sT, s0, ns * 4, cudaMemcpyDeviceToDevice, tl_stream)
                           : cudaMemsetAsync(sT, 0, ns * 4, tl_stream);
        return e == cudaSuccess ? RWKV_OK : cuda_fail(e, "T=0 state copy");
    }
    wkv::Wkv6Args a{B, T, H, N, r, k, v, w, u, s0, y, sT, true, status, segments};
    size_t need = 0;
    cudaError_t e = wkv::wkv6_chunked_launch_noalloc(a, segments, &need, tl_stream);
    if (e == cudaErrorInvalidValue && need > wkv::kNoAllocScratchBytes) {
        snprintf(tl_err, sizeof(tl_err),
                 "the requested sequence split needs %zu bytes of scratch; the fixed no-allocation "
                 "buffer holds %zu (use fewer segments)",
                 need, wkv::kNoAllocScratchBytes);
        return RWKV_ERR_SHAPE;
    }
    if (e != cudaSuccess) return cuda_fail(e, "wkv6 no-allocation launch");
    return RWKV_OK;
}

// ---- gated delta rule ----------------------------------------------------------------

struct DeltaSizes {
    int64_t n, nk, nh, ns;  // elements of v (and o), of q (and k), of g (and beta), of the states
    int64_t nseq, nslots;
};

// Sizes of a delta-rule call, checked for sign, overflow and what the kernels' grids hold.
int delta_sizes(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N, int64_t nseq, bool packed, int64_t nslots,
                bool slots, DeltaSizes *z)
{
    if (B < 0 || T < 0 || Hk < 0 || H < 0 || N < 0 || (packed && nseq < 0) || (slots && nslots < 0))
        return fail(RWKV_ERR_SHAPE, "negative size%s");
    if (packed && B != 1) return fail(RWKV_ERR_SHAPE, "packed sequences (offsets) need B = 1%s");
    if (H > 0 && (Hk == 0 || H % Hk != 0)) return fail(RWKV_ERR_SHAPE, "Hk must divide H%s");
    z->nseq = packed ? nseq : B;
    z->nslots = slots ? nslots : z->nseq;
    int64_t BT, x;
    if (!mul_ok(B, T, &BT) || !mul_ok(BT, Hk, &x) || !mul_ok(x, N, &z->nk) || !mul_ok(BT, H, &z->nh) ||
        !mul_ok(z->nh, N, &z->n) || !mul_ok(z->nslots, H, &x) || !mul_ok(x, N * N, &z->ns) ||
        !mul_ok(z->nseq, H, &x))
        return fail(RWKV_ERR_SHAPE, "size product overflows%s");
    // blocks are numbered by (sequence, head); token, head and slot indices are 32-bit
    if (x > 0x7fffffffLL || BT > 0x7fffff00LL || z->nslots > 0x7fffffffLL || z->nseq > 0x7ffffffeLL)
        return fail(RWKV_ERR_SHAPE, "more than 2^31 (sequence, head) pairs, tokens or slots%s");
    const int64_t chunks = packed ? T / 64 + nseq : B * ((T + 63) / 64);  // at most 2^32
    if (H > 0 && chunks > 0x7fffffffLL / H) return fail(RWKV_ERR_SHAPE, "more than 2^31 (chunk, head) pairs%s");
    return RWKV_OK;
}

// Shortest mean sequences of bf16 that take the tensor cores; shorter ones and fp32 are walked
// token by token.  A chunk costs the same however few tokens it holds, a walk grows with them.
// Forward, walk against chunked, us (B1 H4, B8 H32, B64 H32): 20 tokens 10 / 12, 16 / 16, 66 / 72; 28
// tokens 12 / 12, 20 / 18, 86 / 74.  Backward: 8 tokens 16 / 24, 22 / 37, 106 / 164; 9 tokens 20 / 25,
// 39 / 35, 174 / 164 (beyond one segment of 8 two walks come first).  The host knows a packed call's mean
// length alone, so one long sequence among many short ones is walked with them: 2048 tokens and 127 single
// ones, H16, 631 us where the two kinds apart take 73 and 15; backward of 4000 and 600, H32, 2.8 ms
// (the 4000 alone 0.28).
constexpr int64_t kDeltaChunkedTokens = 24, kDeltaBwdChunkedTokens = 9;

bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }

// A DeltaArgs with the sizes alone, for the workspace of a call.
wkv::DeltaArgs delta_shape(int64_t B, int64_t T, int64_t Hk, int64_t H, const DeltaSizes &z, bool packed, bool bf16)
{
    static const int32_t any = 0;
    wkv::DeltaArgs a{};
    a.B = B, a.T = T, a.Hk = Hk, a.H = H, a.nseq = z.nseq, a.bf16 = bf16;
    a.offsets = packed ? &any : nullptr;  // only its being there counts
    return a;
}

bool delta_chunked(int64_t T, const DeltaSizes &z, bool packed, bool bf16, int64_t least)
{
    return bf16 && z.n > 0 && z.nseq > 0 && (packed ? T / z.nseq : T) >= least;
}

int delta_fwd_bytes(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N, int64_t nseq, bool packed, int64_t nslots,
                    bool slots, bool bf16, DeltaSizes *z, size_t *bytes)
{
    int rc = delta_sizes(B, T, Hk, H, N, nseq, packed, nslots, slots, z);
    if (rc) return rc;
    const wkv::DeltaArgs a = delta_shape(B, T, Hk, H, *z, packed, bf16);
    *bytes = N == 64 && delta_chunked(T, *z, packed, bf16, kDeltaChunkedTokens) ? wkv::delta_t_bytes(a) : 0;
    return RWKV_OK;
}

int delta_entry(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N, const void *q, const void *k, const void *v,
                const void *g, const void *beta, float scale, int64_t nseq, const int32_t *offsets, int64_t nslots,
                const int32_t *slots, const float *s0, void *o, float *sT, void *workspace, size_t wbytes, bool bf16)
{
    tl_err[0] = 0;
    DeltaSizes z;
    size_t need = 0;
    int rc = delta_fwd_bytes(B, T, Hk, H, N, nseq, offsets != nullptr, nslots, slots != nullptr, bf16, &z, &need);
    if (rc) return rc;
    if (z.nseq == 0 || H == 0 || N == 0 || (z.n == 0 && !(sT && z.ns > 0))) return RWKV_OK;
    if (N != 64) return fail(RWKV_ERR_UNSUPPORTED, "head size N must be 64%s");
    if (!(scale >= -3.0e38f && scale <= 3.0e38f)) return fail(RWKV_ERR_ARG, "scale must be finite%s");
    if (z.n > 0 && (!q || !k || !v || !g || !beta || !o))
        return fail(RWKV_ERR_NULL, "q, k, v, g, beta and o must be non-null%s");
    if (need > 0 && !workspace) return fail(RWKV_ERR_NULL, "workspace must be non-null%s");
    if (wbytes < need) {
        snprintf(tl_err, sizeof(tl_err), "workspace holds %zu bytes; this call needs %zu", wbytes, need);
        return RWKV_ERR_ARG;
    }
    const void *ptrs[] = {q, k, v, g, beta, s0, o, sT, workspace};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return fail(RWKV_ERR_ALIGN, "tensor pointers must be 16-byte aligned%s");
    if (!aligned4(offsets) || !aligned4(slots)) return fail(RWKV_ERR_ALIGN, "index arrays must be 4-byte aligned%s");
    const int64_t esz = bf16 ? 2 : 4;
    const Span so{o, z.n * esz}, ss0{s0, z.ns * 4}, ssT{sT, z.ns * 4}, sw{workspace, static_cast<int64_t>(need)};
    const Span ins[] = {{q, z.nk * esz}, {k, z.nk * esz}, {v, z.n * esz}, {g, z.nh * esz}, {beta, z.nh * esz},
                        {offsets, (z.nseq + 1) * 4}, {slots, z.nseq * 4}};
    for (const Span &x : ins) {
        if (overlap(so, x)) return fail(RWKV_ERR_ALIAS, "o overlaps an input%s");
        if (overlap(ssT, x)) return fail(RWKV_ERR_ALIAS, "sT overlaps an input%s");
        if (overlap(sw, x)) return fail(RWKV_ERR_ALIAS, "the workspace overlaps an input%s");
    }
    if (overlap(sw, so) || overlap(sw, ss0) || overlap(sw, ssT))
        return fail(RWKV_ERR_ALIAS, "the workspace overlaps an output or a state%s");
    if (overlap(so, ss0) || overlap(so, ssT)) return fail(RWKV_ERR_ALIAS, "o overlaps a state%s");
    if (s0 != sT && overlap(ssT, ss0)) return fail(RWKV_ERR_ALIAS, "sT partially overlaps s0%s");
    int *status = nullptr;
    rc = status_word(&status);
    if (rc) return rc;
    const wkv::DeltaArgs a{B, T, Hk, H, z.nseq, offsets, z.nslots, slots, q, k, v, g, beta, scale, s0, o, sT, bf16, status};
    cudaError_t e;
    if (need > 0) {
        e = wkv::delta_prep_launch(a, workspace, tl_stream);
        if (e == cudaSuccess) e = wkv::delta_chunked_launch(a, workspace, tl_stream);
    } else {
        e = wkv::delta_recurrent_launch(a, tl_stream);
    }
    return e == cudaSuccess ? RWKV_OK : cuda_fail(e, "delta launch");
}

int delta_bwd_bytes(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N, int64_t nseq, bool packed, bool bf16,
                    DeltaSizes *z, size_t *bytes)
{
    int rc = delta_sizes(B, T, Hk, H, N, nseq, packed, 0, false, z);
    if (rc) return rc;
    // No overflow here: 2^31 (chunk, head) pairs at most are 2^34 segments of 8 tokens, and neither layout
    // takes 2^16 bytes for one.
    const wkv::DeltaArgs a = delta_shape(B, T, Hk, H, *z, packed, bf16);
    *bytes = z->nseq == 0 || z->nh == 0 || N != 64 ? 0
             : delta_chunked(T, *z, packed, bf16, kDeltaBwdChunkedTokens) ? wkv::delta_backward_tc_workspace_bytes(a)
                                                                          : wkv::delta_walks_workspace_bytes(a);
    return RWKV_OK;
}

int delta_bwd_entry(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N, const void *q, const void *k,
                    const void *v, const void *g, const void *beta, float scale, int64_t nseq, const int32_t *offsets,
                    const float *s0, const void *dout, const float *dsT, void *dq, void *dk, void *dv, void *dg,
                    void *dbeta, float *ds0, void *workspace, size_t wbytes, bool bf16)
{
    tl_err[0] = 0;
    DeltaSizes z;
    size_t need = 0;
    int rc = delta_bwd_bytes(B, T, Hk, H, N, nseq, offsets != nullptr, bf16, &z, &need);
    if (rc) return rc;
    if (z.nseq == 0 || H == 0 || N == 0 || (z.n == 0 && !(ds0 && z.ns > 0))) return RWKV_OK;
    if (N != 64) return fail(RWKV_ERR_UNSUPPORTED, "head size N must be 64%s");
    if (!(scale >= -3.0e38f && scale <= 3.0e38f)) return fail(RWKV_ERR_ARG, "scale must be finite%s");
    if (z.n > 0 && (!q || !k || !v || !g || !beta || !dout))
        return fail(RWKV_ERR_NULL, "q, k, v, g, beta and dout must be non-null%s");
    if (z.n > 0 && (!dq || !dk || !dv || !dg || !dbeta))
        return fail(RWKV_ERR_NULL, "dq, dk, dv, dg and dbeta must be non-null%s");
    if (need > 0 && !workspace) return fail(RWKV_ERR_NULL, "workspace must be non-null%s");
    if (wbytes < need) {
        snprintf(tl_err, sizeof(tl_err), "workspace holds %zu bytes; this call needs %zu", wbytes, need);
        return RWKV_ERR_ARG;
    }
    const void *ptrs[] = {q, k, v, g, beta, s0, dout, dsT, dq, dk, dv, dg, dbeta, ds0, workspace};
    for (const void *p : ptrs)
        if (p && !aligned16(p)) return fail(RWKV_ERR_ALIGN, "tensor pointers must be 16-byte aligned%s");
    if (!aligned4(offsets)) return fail(RWKV_ERR_ALIGN, "index arrays must be 4-byte aligned%s");
    const int64_t e = bf16 ? 2 : 4;
    const Span ins[] = {{q, z.nk * e}, {k, z.nk * e}, {v, z.n * e}, {g, z.nh * e}, {beta, z.nh * e}, {s0, z.ns * 4},
                        {dout, z.n * e}, {dsT, z.ns * 4}, {offsets, (z.nseq + 1) * 4}};
    const Span outs[] = {{dq, z.nk * e}, {dk, z.nk * e}, {dv, z.n * e}, {dg, z.nh * e}, {dbeta, z.nh * e},
                         {ds0, z.ns * 4}, {workspace, static_cast<int64_t>(need)}};
    const int n_outs = sizeof(outs) / sizeof(outs[0]);
    for (int i = 0; i < n_outs; ++i) {
        for (const Span &x : ins) {
            // ds0 may be the very same array as dsT (in place); any other overlap is refused
            if (outs[i].p == ds0 && x.p == dsT && ds0 == dsT) continue;
            if (overlap(outs[i], x)) return fail(RWKV_ERR_ALIAS, "a gradient or the workspace overlaps an input%s");
        }
        for (int c = i + 1; c < n_outs; ++c)
            if (overlap(outs[i], outs[c])) return fail(RWKV_ERR_ALIAS, "two outputs overlap%s");
    }
    int *status = nullptr;
    rc = status_word(&status);
    if (rc) return rc;
    wkv::DeltaBwdArgs a{};
    a.f = wkv::DeltaArgs{B, T, Hk, H, z.nseq, offsets, z.nseq, nullptr, q, k, v, g, beta, scale, s0, nullptr, nullptr, bf16, status};
    a.dout = dout, a.dsT = dsT, a.dq = dq, a.dk = dk, a.dv = dv, a.dg = dg, a.dbeta = dbeta, a.ds0 = ds0;
    a.workspace = workspace;
    const cudaError_t err = delta_chunked(T, z, offsets != nullptr, bf16, kDeltaBwdChunkedTokens)
                                ? wkv::delta_backward_tc_launch(a, tl_stream)
                                : wkv::delta_backward_walks_launch(a, tl_stream);
    return err == cudaSuccess ? RWKV_OK : cuda_fail(err, "delta backward launch");
}

// ---- state pools ----------------------------------------------------------------------

int pool_sizes(int64_t layers, int64_t nslots, int64_t slot_bytes, const void *pool, int64_t *bytes)
{
    int64_t per;
    if (layers < 0 || nslots < 0 || slot_bytes < 0) return fail(RWKV_ERR_SHAPE, "negative size%s");
    if (!mul_ok(nslots, slot_bytes, &per) || !mul_ok(layers, per, bytes))
        return fail(RWKV_ERR_SHAPE, "size product overflows%s");
    if (nslots > 0x7fffffffLL) return fail(RWKV_ERR_SHAPE, "more than 2^31 slots%s");
    if (*bytes > 0 && !pool) return fail(RWKV_ERR_NULL, "pool must be non-null%s");
    if (slot_bytes % 16 != 0 || !aligned16(pool))
        return fail(RWKV_ERR_ALIGN, "the pool must be 16-byte aligned and slot_bytes a multiple of 16%s");
    return RWKV_OK;
}

}  // namespace

extern "C" {

int rwkv_wkv4_forward(int64_t B, int64_t T, int64_t C, const float *w, const float *u,
                      const float *k, const float *v, float *y)
{
    return wkv4_entry(B, T, C, w, u, k, v, nullptr, y, nullptr, false, false);
}

int rwkv_wkv4_forward_bf16(int64_t B, int64_t T, int64_t C, const float *w, const float *u,
                           const uint16_t *k, const uint16_t *v, uint16_t *y)
{
    return wkv4_entry(B, T, C, w, u, k, v, nullptr, y, nullptr, true, false);
}

int rwkv_wkv4_forward_state(int64_t B, int64_t T, int64_t C, const float *w, const float *u,
                            const float *k, const float *v, const float *s0, float *y,
                            float *sT)
{
    return wkv4_entry(B, T, C, w, u, k, v, s0, y, sT, false, true);
}

int rwkv_wkv4_forward_state_bf16(int64_t B, int64_t T, int64_t C, const float *w,
                                 const float *u, const uint16_t *k, const uint16_t *v,
                                 const float *s0, uint16_t *y, float *sT)
{
    return wkv4_entry(B, T, C, w, u, k, v, s0, y, sT, true, true);
}

int rwkv_wkv6_forward(int64_t B, int64_t T, int64_t H, int64_t N, const float *r,
                      const float *k, const float *v, const float *w, const float *u,
                      const float *s0, float *y, float *sT)
{
    return wkv6_entry(B, T, H, N, r, k, v, w, u, s0, y, sT, false);
}

int rwkv_wkv6_forward_bf16(int64_t B, int64_t T, int64_t H, int64_t N, const uint16_t *r,
                           const uint16_t *k, const uint16_t *v, const uint16_t *w,
                           const float *u, const float *s0, uint16_t *y, float *sT)
{
    return wkv6_entry(B, T, H, N, r, k, v, w, u, s0, y, sT, true);
}

extern "C" int rwkv_wkv6_forward_gated_bf16(int64_t B, int64_t T, int64_t H, int64_t N, const uint16_t *r,
                                            const uint16_t *k, const uint16_t *v, const uint16_t *w,
                                            const float *u, const float *s0, const uint16_t *g,
                                            const float *ln_w, const float *ln_b, float eps, uint16_t *y,
                                            float *sT)
{
    return wkv6_entry(B, T, H, N, r, k, v, w, u, s0, y, sT, true, g, ln_w, ln_b, eps, true);
}

int rwkv_wkv6_forward_omega_bf16(int64_t B, int64_t T, int64_t H, int64_t N, const uint16_t *r,
                                 const uint16_t *k, const uint16_t *v, const uint16_t *omega,
                                 const float *u, const float *s0, const uint16_t *g, const float *ln_w,
                                 const float *ln_b, float eps, uint16_t *y, float *sT)
{
    // the output stage is fused when any of its three tensors is given; the gated checks then
    // reject a missing one
    const bool gated = g || ln_w || ln_b;
    return wkv6_entry(B, T, H, N, r, k, v, omega, u, s0, y, sT, true, g, ln_w, ln_b, gated ? eps : 0.f, gated,
                      true);
}

int rwkv_wkv6_forward_bf16_noalloc(int64_t B, int64_t T, int64_t H, int64_t N, const uint16_t *r,
                                   const uint16_t *k, const uint16_t *v, const uint16_t *w,
                                   const float *u, const float *s0, uint16_t *y, float *sT,
                                   int segments)
{
    return wkv6_noalloc_entry(B, T, H, N, r, k, v, w, u, s0, y, sT, segments);
}

int rwkv_wkv6_backward_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t N, size_t *bytes)
{
    tl_err[0] = 0;
    if (!bytes) return fail(RWKV_ERR_NULL, "bytes must be non-null%s");
    int64_t n, ns, hn;
    int rc = wkv6_bwd_sizes(B, T, H, N, &n, &ns, &hn);
    if (rc) return rc;
    *bytes = n > 0 ? wkv::wkv6_backward_workspace_bytes(B, T, H) : 0;
    return RWKV_OK;
}

int rwkv_wkv6_backward(int64_t B, int64_t T, int64_t H, int64_t N, const float *r, const float *k,
                       const float *v, const float *w, const float *u, const float *s0, const float *dy,
                       const float *dsT, float *dr, float *dk, float *dv, float *dw, float *du, float *ds0,
                       void *workspace, size_t workspace_bytes)
{
    return wkv6_bwd_entry(B, T, H, N, r, k, v, w, u, s0, dy, dsT, dr, dk, dv, dw, du, ds0, workspace,
                          workspace_bytes, false, false);
}

int rwkv_wkv6_backward_bf16(int64_t B, int64_t T, int64_t H, int64_t N, const uint16_t *r, const uint16_t *k,
                            const uint16_t *v, const uint16_t *w, const float *u, const float *s0,
                            const uint16_t *dy, const float *dsT, float *dr, float *dk, float *dv, float *dw,
                            float *du, float *ds0, void *workspace, size_t workspace_bytes)
{
    return wkv6_bwd_entry(B, T, H, N, r, k, v, w, u, s0, dy, dsT, dr, dk, dv, dw, du, ds0, workspace,
                          workspace_bytes, true, false);
}

int rwkv_wkv6_backward_omega_bf16(int64_t B, int64_t T, int64_t H, int64_t N, const uint16_t *r,
                                  const uint16_t *k, const uint16_t *v, const uint16_t *omega, const float *u,
                                  const float *s0, const uint16_t *dy, const float *dsT, float *dr, float *dk,
                                  float *dv, float *domega, float *du, float *ds0, void *workspace,
                                  size_t workspace_bytes)
{
    return wkv6_bwd_entry(B, T, H, N, r, k, v, omega, u, s0, dy, dsT, dr, dk, dv, domega, du, ds0, workspace,
                          workspace_bytes, true, true);
}

int rwkv_delta_forward(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N, const float *q, const float *k,
                       const float *v, const float *g, const float *beta, float scale, int64_t nseq,
                       const int32_t *offsets, int64_t nslots, const int32_t *slots, const float *s0, float *o,
                       float *sT, void *workspace, size_t workspace_bytes)
{
    return delta_entry(B, T, Hk, H, N, q, k, v, g, beta, scale, nseq, offsets, nslots, slots, s0, o, sT, workspace,
                       workspace_bytes, false);
}

int rwkv_delta_forward_bf16(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N, const uint16_t *q,
                            const uint16_t *k, const uint16_t *v, const uint16_t *g, const uint16_t *beta,
                            float scale, int64_t nseq, const int32_t *offsets, int64_t nslots, const int32_t *slots,
                            const float *s0, uint16_t *o, float *sT, void *workspace, size_t workspace_bytes)
{
    return delta_entry(B, T, Hk, H, N, q, k, v, g, beta, scale, nseq, offsets, nslots, slots, s0, o, sT, workspace,
                       workspace_bytes, true);
}

int rwkv_delta_forward_workspace_bytes(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N, int64_t nseq,
                                       int packed, int bf16, size_t *bytes)
{
    tl_err[0] = 0;
    if (!bytes) return fail(RWKV_ERR_NULL, "bytes must be non-null%s");
    DeltaSizes z;
    return delta_fwd_bytes(B, T, Hk, H, N, nseq, packed != 0, 0, false, bf16 != 0, &z, bytes);
}

int rwkv_delta_backward_workspace_bytes(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N, int64_t nseq,
                                        int packed, int bf16, size_t *bytes)
{
    tl_err[0] = 0;
    if (!bytes) return fail(RWKV_ERR_NULL, "bytes must be non-null%s");
    DeltaSizes z;
    return delta_bwd_bytes(B, T, Hk, H, N, nseq, packed != 0, bf16 != 0, &z, bytes);
}

int rwkv_delta_backward(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N, const float *q, const float *k,
                        const float *v, const float *g, const float *beta, float scale, int64_t nseq,
                        const int32_t *offsets, const float *s0, const float *dout, const float *dsT, float *dq,
                        float *dk, float *dv, float *dg, float *dbeta, float *ds0, void *workspace,
                        size_t workspace_bytes)
{
    return delta_bwd_entry(B, T, Hk, H, N, q, k, v, g, beta, scale, nseq, offsets, s0, dout, dsT, dq, dk, dv, dg,
                           dbeta, ds0, workspace, workspace_bytes, false);
}

int rwkv_delta_backward_bf16(int64_t B, int64_t T, int64_t Hk, int64_t H, int64_t N, const uint16_t *q,
                             const uint16_t *k, const uint16_t *v, const uint16_t *g, const uint16_t *beta,
                             float scale, int64_t nseq, const int32_t *offsets, const float *s0,
                             const uint16_t *dout, const float *dsT, uint16_t *dq, uint16_t *dk, uint16_t *dv,
                             uint16_t *dg, uint16_t *dbeta, float *ds0, void *workspace, size_t workspace_bytes)
{
    return delta_bwd_entry(B, T, Hk, H, N, q, k, v, g, beta, scale, nseq, offsets, s0, dout, dsT, dq, dk, dv, dg,
                           dbeta, ds0, workspace, workspace_bytes, true);
}

int rwkv_state_copy(int64_t layers, int64_t nslots, int64_t slot_bytes, void *pool, int64_t n, const int32_t *src,
                    const int32_t *dst)
{
    tl_err[0] = 0;
    int64_t bytes;
    int rc = pool_sizes(layers, nslots, slot_bytes, pool, &bytes);
    if (rc) return rc;
    if (n < 0 || n > wkv::kMaxCopyPairs) return fail(RWKV_ERR_SHAPE, "n must be 0 .. 4096 pairs%s");
    if (n == 0 || bytes == 0) return RWKV_OK;
    if (!src || !dst) return fail(RWKV_ERR_NULL, "src and dst must be non-null%s");
    if (!aligned4(src) || !aligned4(dst)) return fail(RWKV_ERR_ALIGN, "index arrays must be 4-byte aligned%s");
    if (overlap({pool, bytes}, {src, n * 4}) || overlap({pool, bytes}, {dst, n * 4}))
        return fail(RWKV_ERR_ALIAS, "the pool overlaps an index array%s");
    int *status = nullptr;
    rc = status_word(&status);
    if (rc) return rc;
    const cudaError_t e = wkv::state_copy_launch(
        {layers, nslots, slot_bytes, static_cast<unsigned char *>(pool), n, src, dst, status}, tl_stream);
    return e == cudaSuccess ? RWKV_OK : cuda_fail(e, "state copy launch");
}

int rwkv_state_compact(int64_t layers, int64_t nslots, int64_t slot_bytes, void *pool, const uint8_t *live,
                       int32_t *new_index, int32_t *count)
{
    tl_err[0] = 0;
    int64_t bytes;
    int rc = pool_sizes(layers, nslots, slot_bytes, pool, &bytes);
    if (rc) return rc;
    if (nslots > wkv::kMaxCompactSlots) return fail(RWKV_ERR_SHAPE, "a compacted pool has at most 16384 slots%s");
    if (!count || (nslots > 0 && (!live || !new_index)))
        return fail(RWKV_ERR_NULL, "live, new_index and count must be non-null%s");
    if (!aligned4(new_index) || !aligned4(count)) return fail(RWKV_ERR_ALIGN, "index arrays must be 4-byte aligned%s");
    const Span sp{pool, bytes}, sl{live, nslots}, sn{new_index, nslots * 4}, sc{count, 4};
    if (overlap(sp, sl) || overlap(sp, sn) || overlap(sp, sc) || overlap(sl, sn) || overlap(sl, sc) || overlap(sn, sc))
        return fail(RWKV_ERR_ALIAS, "the pool, live, new_index and count must not overlap%s");
    int *status = nullptr;
    rc = status_word(&status);
    if (rc) return rc;
    const cudaError_t e = wkv::state_compact_launch(
        {layers, nslots, slot_bytes, static_cast<unsigned char *>(pool), live, new_index, count, status}, tl_stream);
    return e == cudaSuccess ? RWKV_OK : cuda_fail(e, "state compact launch");
}

int rwkv_set_wkv6_algo(int algo)
{
    if (algo != RWKV_WKV6_AUTO && algo != RWKV_WKV6_SERIAL && algo != RWKV_WKV6_CHUNKED)
        return RWKV_ERR_ARG;
    tl_wkv6_algo = algo;
    return RWKV_OK;
}

int rwkv_get_wkv6_algo(void) { return tl_wkv6_algo; }

int rwkv_set_wkv6_segments(int segments)
{
    if (segments < 0) return RWKV_ERR_ARG;
    tl_wkv6_segments = segments;
    return RWKV_OK;
}

int rwkv_get_wkv6_segments(void) { return tl_wkv6_segments; }

int rwkv_debug_inject_timeout(int enable)
{
    int prev = wkv::g_chunked_inject_timeout;
    wkv::g_chunked_inject_timeout = enable ? 1 : 0;
    return prev;
}

void rwkv_set_stream(void *cuda_stream) { tl_stream = static_cast<cudaStream_t>(cuda_stream); }

void *rwkv_get_stream(void) { return tl_stream; }

int rwkv_get_device_status(void)
{
    int *p = nullptr;
    int rc = status_word(&p);
    if (rc) return rc;
    cudaError_t e = cudaStreamSynchronize(tl_stream);
    if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
    int value = 0, zero = 0;
    e = cudaMemcpy(&value, p, sizeof(int), cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_fail(e, "status read");
    e = cudaMemcpy(p, &zero, sizeof(int), cudaMemcpyHostToDevice);
    if (e != cudaSuccess) return cuda_fail(e, "status clear");
    return value;
}

const char *rwkv_status_string(int status)
{
    switch (status) {
    case RWKV_OK: return "ok";
    case RWKV_ERR_NULL: return "required pointer is null";
    case RWKV_ERR_SHAPE: return "invalid size";
    case RWKV_ERR_UNSUPPORTED: return "unsupported configuration";
    case RWKV_ERR_ALIAS: return "output overlaps an input";
    case RWKV_ERR_CUDA: return "CUDA error";
    case RWKV_ERR_TIMEOUT: return "device-side wait timed out";
    case RWKV_ERR_ALIGN: return "pointer not 16-byte aligned";
    case RWKV_ERR_ARG: return "invalid argument";
    case RWKV_ERR_BOUNDS: return "index check failed (debug build)";
    default: return "unknown status";
    }
}

const char *rwkv_last_error(void) { return tl_err; }

int rwkv_abi_version(void) { return RWKV_ABI_VERSION; }

int rwkv_debug_bounds(void) { return wkv::kDebugBounds ? 1 : 0; }

}  // extern "C"
