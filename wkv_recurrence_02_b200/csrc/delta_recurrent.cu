// delta_recurrent.cu -- the gated delta rule token by token (decode, a few tokens, fp32).
//
// Per sequence and value head, state S (64 x 64, row i = key channel, column j = value channel):
//   S' = exp(g_t) S,   u_t = beta_t (v_t - k_t S'),   S = S' + k_t^T u_t,   o_t = scale q_t S.
// The two products with the state are taken in one walk over it, before the update:
//   k_t S' = a (k_t S),   q_t S = a (q_t S_prev) + (q_t . k_t) u_t,   a = exp(g_t).
//
// The columns of S are independent of one another given k, so a warp owns 16 columns of one
// head and keeps them in registers for the whole sequence.  One block is the four warps of one
// (sequence, head).
//
// Two kernels.  A few tokens (decode) are bound by the state's bytes, 16 KB in and 16 KB out
// for each head, all of a warp's 4 KB loaded at once: 256 sequences of 64 heads take 94 us, 5.8
// TB/s.  There lane (rg, cq) holds rows 8 rg .. 8 rg + 7 of columns 4 cq .. 4 cq + 3, 16-byte
// loads and stores of the state; sums over rows are three shuffles; no shared memory.  More
// tokens are bound by the chain and the instructions of one token: see delta_walk_kernel.
#include "wkv_internal.cuh"

namespace wkv {
namespace {

constexpr int kN = 64;
constexpr int kThreads = 128;

template <typename T> __device__ __forceinline__ void ld_n(const T *p, float (&x)[4]);
template <> __device__ __forceinline__ void ld_n<float>(const float *p, float (&x)[4])
{
    const float4 q = *reinterpret_cast<const float4 *>(p);
    x[0] = q.x, x[1] = q.y, x[2] = q.z, x[3] = q.w;
}
template <> __device__ __forceinline__ void ld_n<__nv_bfloat16>(const __nv_bfloat16 *p, float (&x)[4])
{
    const uint2 q = *reinterpret_cast<const uint2 *>(p);
    x[0] = __uint_as_float(q.x << 16), x[1] = __uint_as_float(q.x & 0xFFFF0000u);
    x[2] = __uint_as_float(q.y << 16), x[3] = __uint_as_float(q.y & 0xFFFF0000u);
}
template <typename T> __device__ __forceinline__ void ld8(const T *p, float (&x)[8]);
template <> __device__ __forceinline__ void ld8<float>(const float *p, float (&x)[8])
{
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
template <> __device__ __forceinline__ void ld8<__nv_bfloat16>(const __nv_bfloat16 *p, float (&x)[8])
{
    const uint4 q = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ float ld1(const float *p) { return *p; }
__device__ __forceinline__ float ld1(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st_n(float *p, const float (&x)[4])
{
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void st_n(__nv_bfloat16 *p, const float (&x)[4])
{
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                               *reinterpret_cast<const uint32_t *>(&b));
}

// Inputs of one token for one lane: its 8 rows of q and k, its 4 columns of v, the two scalars.
struct Token {
    float q[8], k[8], v[4], g, b;
};

template <typename T>
__global__ void __launch_bounds__(kThreads)
delta_recurrent_kernel(int64_t B, int64_t Tn, int64_t Hk, int64_t H, int64_t nseq, const int32_t *__restrict__ offsets,
                       int64_t nslots, const int32_t *__restrict__ slots, const T *__restrict__ q,
                       const T *__restrict__ k, const T *__restrict__ v, const T *__restrict__ g,
                       const T *__restrict__ beta, float scale, const float *s0, T *__restrict__ o, float *sT,
                       int *status)
{
    const int64_t n = blockIdx.x, seq = n / H, h = n % H, hk = h / (H / Hk);
    const int lane = threadIdx.x & 31, rg = lane >> 2;
    const int col = 16 * (threadIdx.x >> 5) + 4 * (lane & 3);
    int64_t first, len;
    sequence_span(offsets, seq, Tn, &first, &len);
    const int64_t slot = sequence_slot(slots, seq, nslots, status);
    const int64_t at = ((slot * H + h) * kN + 8 * rg) * kN + col;  // this lane's first state element
    const bool has = slot >= 0 && in_bounds(status, (slot * H + h) * kN * kN, kN * kN, nslots * H * kN * kN);

    const int64_t ntok = B * Tn;
    auto load = [&](int64_t t, Token &x) {
        if (!in_bounds(status, first + t, 1, ntok)) return;
        const T *pq = q + ((first + t) * Hk + hk) * kN + 8 * rg, *pk = k + ((first + t) * Hk + hk) * kN + 8 * rg;
        const int64_t th = (first + t) * H + h;
        ld8(pq, x.q);
        ld8(pk, x.k);
        ld_n(v + th * kN + col, x.v);
        x.g = ld1(g + th);
        x.b = ld1(beta + th);
    };

    float S[8][4];
    if (s0 && has) {
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            const float4 x = *reinterpret_cast<const float4 *>(s0 + at + m * kN);
            S[m][0] = x.x, S[m][1] = x.y, S[m][2] = x.z, S[m][3] = x.w;
        }
    } else {
#pragma unroll
        for (int m = 0; m < 8; ++m)
#pragma unroll
            for (int c = 0; c < 4; ++c) S[m][c] = 0.f;
    }
    Token x, y;
    if (len > 0) load(0, x);
    for (int64_t t = 0; t < len; ++t) {
        if (t + 1 < len) load(t + 1, y);  // the next token's inputs load under this one's sums
        const float a = expf(x.g);
        float ks[4] = {}, qs[4] = {}, qk = 0.f;
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            qk = fmaf(x.q[m], x.k[m], qk);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                ks[c] = fmaf(x.k[m], S[m][c], ks[c]);
                qs[c] = fmaf(x.q[m], S[m][c], qs[c]);
            }
        }
#pragma unroll
        for (int d = 4; d < 32; d *= 2) {
            qk += __shfl_xor_sync(0xffffffffu, qk, d);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                ks[c] += __shfl_xor_sync(0xffffffffu, ks[c], d);
                qs[c] += __shfl_xor_sync(0xffffffffu, qs[c], d);
            }
        }
        float u[4], out[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            u[c] = x.b * (x.v[c] - a * ks[c]);
            out[c] = scale * fmaf(qk, u[c], a * qs[c]);
        }
#pragma unroll
        for (int m = 0; m < 8; ++m)
#pragma unroll
            for (int c = 0; c < 4; ++c) S[m][c] = fmaf(x.k[m], u[c], a * S[m][c]);
        if (rg == 0 && in_bounds(status, first + t, 1, ntok)) st_n(o + ((first + t) * H + h) * kN + col, out);
        x = y;
    }
    if (sT && has) {
#pragma unroll
        for (int m = 0; m < 8; ++m)
            *reinterpret_cast<float4 *>(sT + at + m * kN) = make_float4(S[m][0], S[m][1], S[m][2], S[m][3]);
    }
}

// ---------------------------------------------------------------- many tokens
// The same walk for longer sequences, bound by instructions and by the chain of one token (k S,
// two rounds of shuffles, u, the update).  A lane holds 16 rows of two columns (COLS; of one, where
// there are few heads), the rows in pairs, so that the products are two-wide instructions
// (fma.rn.f32x2) and a sum over rows has two rounds of shuffles: 64 fma2 and 10 shuffles a token
// where the layout above has 128 fma and 27.  Inputs come through shared memory (cp.async), kGroups - 1 groups of kGroup tokens
// ahead, a ring to each warp: no barrier.  Measured, one sequence of 4 heads, 256 tokens fp32: 61 us
// a call (0.23 us a token: one warp on each scheduler, a third of its cycles issue), against 127 with the
// kernel above (one token ahead, a miss's latency each).
constexpr int kGroup = 4, kGroups = 4, kRing = kGroup * kGroups;
template <int COLS> constexpr int kRow = 2 * kN + 8 * COLS;  // a token in the ring: q, k, the warp's columns of v

template <typename T> __device__ __forceinline__ void copy16(T *smem, const T *gmem)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(smem))),
                 "l"(gmem)
                 : "memory");
}
__device__ __forceinline__ uint64_t pack2(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float sum2(uint64_t x)
{
    float lo, hi;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
    return lo + hi;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// Rows 16 i + 4 rg + 0 .. 3, i = 0 .. 3, of a vector, in pairs (lanes side by side read side by side).
__device__ __forceinline__ void ld_rows(const float *p, int rg, uint64_t (&x)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const ulonglong2 w = *reinterpret_cast<const ulonglong2 *>(p + 16 * i + 4 * rg);
        x[2 * i] = w.x, x[2 * i + 1] = w.y;
    }
}
__device__ __forceinline__ void ld_rows(const __nv_bfloat16 *p, int rg, uint64_t (&x)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float f[4];
        ld_n(p + 16 * i + 4 * rg, f);
        x[2 * i] = pack2(f[0], f[1]), x[2 * i + 1] = pack2(f[2], f[3]);
    }
}
__device__ __forceinline__ void ldc(const float *p, float (&x)[1]) { x[0] = *p; }
__device__ __forceinline__ void ldc(const __nv_bfloat16 *p, float (&x)[1]) { x[0] = __bfloat162float(*p); }
__device__ __forceinline__ void ldc(const float *p, float (&x)[2])
{
    const float2 w = *reinterpret_cast<const float2 *>(p);
    x[0] = w.x, x[1] = w.y;
}
__device__ __forceinline__ void ldc(const __nv_bfloat16 *p, float (&x)[2])
{
    const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
    x[0] = __uint_as_float(w << 16), x[1] = __uint_as_float(w & 0xFFFF0000u);
}
__device__ __forceinline__ void stc(float *p, const float (&x)[1]) { *p = x[0]; }
__device__ __forceinline__ void stc(__nv_bfloat16 *p, const float (&x)[1]) { *p = __float2bfloat16_rn(x[0]); }
__device__ __forceinline__ void stc(float *p, const float (&x)[2])
{
    *reinterpret_cast<float2 *>(p) = make_float2(x[0], x[1]);
}
__device__ __forceinline__ void stc(__nv_bfloat16 *p, const float (&x)[2])
{
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(x[0], x[1]);
}

// One token for one lane: its rows of q and k, its columns of v, exp(g) and beta.
template <int COLS> struct WalkToken {
    uint64_t q[8], k[8];
    float v[COLS], a, b;
};

// What a walk is for.  kStates: the state before every segment of the backward pass (q and o unused).
// kGradients: the walk back for the gradient D of the state (v: the outputs' gradients, s0: the last
// state's), D after every segment:
//   D += scale q_t^T do_t,   du = k_t D,   D = exp(g_t) (D - beta_t k_t^T du)
enum { kOutputs, kStates, kGradients };

template <typename T, int COLS, int MODE>
__global__ void __launch_bounds__(kThreads)
delta_walk_kernel(int64_t B, int64_t Tn, int64_t Hk, int64_t H, int64_t nseq, const int32_t *__restrict__ offsets,
                  int64_t nslots, const int32_t *__restrict__ slots, const T *__restrict__ q, const T *__restrict__ k,
                  const T *__restrict__ v, const T *__restrict__ g, const T *__restrict__ beta, float scale,
                  const float *s0, T *__restrict__ o, float *sT, float *ckpt, int64_t nckpt, int *status)
{
    if (MODE == kStates) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the other walk
    constexpr int kParts = 2 / COLS;  // blocks of a (sequence, head)
    const int64_t n = blockIdx.x / kParts, seq = n / H, h = n % H, hk = h / (H / Hk);
    const int lane = threadIdx.x & 31, rg = lane >> 3, warp = threadIdx.x >> 5;
    const int col0 = 8 * COLS * (4 * static_cast<int>(blockIdx.x % kParts) + warp);  // the warp's first column
    const int col = col0 + COLS * (lane & 7);
    int64_t first, len64;
    sequence_span(offsets, seq, Tn, &first, &len64);
    const int tokens = in_bounds(status, first, len64, B * Tn) ? static_cast<int>(len64) : 0;
    const int nseg = (tokens + kDeltaSeg - 1) / kDeltaSeg;
    // tokens to walk; the i-th of them is token_at(i)
    const int len = MODE == kOutputs ? tokens : nseg < 2 ? 0 : MODE == kStates ? (nseg - 1) * kDeltaSeg : tokens - kDeltaSeg;
    auto token_at = [&](int i) { return MODE == kGradients ? tokens - 1 - i : i; };
    const int64_t slot = sequence_slot(slots, seq, nslots, status);
    const int64_t at = 4 * rg * kN + col;  // this lane's first element of a state
    const int64_t state = (slot * H + h) * kN * kN;
    const bool has = slot >= 0 && in_bounds(status, state, kN * kN, nslots * H * kN * kN);

    __shared__ __align__(16) T ring[kThreads / 32][kRing][kRow<COLS>];
    // Copies: chunks of 16 bytes; q and k of kTok tokens at a time, a chunk a lane, then v.
    constexpr int kE = 16 / static_cast<int>(sizeof(T)), kQ = kN / kE, kTok = 32 / (2 * kQ), kV = 8 * COLS / kE;
    const int xq = lane / (2 * kQ), cq = lane % (2 * kQ), xv = lane / kV;
    const T *pq = (cq < kQ ? q : k) + (first * Hk + hk) * kN + (cq % kQ) * kE;
    const T *pv = v + (first * H + h) * kN + col0 + (lane % kV) * kE;
    auto fetch = [&](int t0) {  // tokens t0 .. t0 + kGroup - 1; always one commit: groups are counted by them
#pragma unroll
        for (int x = 0; x < kGroup; x += kTok) {
            const int t = t0 + x + xq;
            if (t < len && (MODE != kStates || cq >= kQ))
                copy16(&ring[warp][t % kRing][cq * kE], pq + token_at(t) * (Hk * kN));
        }
        if (xv < kGroup && t0 + xv < len)
            copy16(&ring[warp][(t0 + xv) % kRing][2 * kN + (lane % kV) * kE], pv + token_at(t0 + xv) * (H * kN));
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // At most kGroups - 2 groups are under way after this.
    auto arrived = [&] {
        asm volatile("cp.async.wait_group %0;" ::"n"(kGroups - 2) : "memory");
        __syncwarp();
    };
    // Lane i's g and beta of the 32 tokens from t, loaded 32 tokens ahead.
    const T *gh = g + first * H + h, *bh = beta + first * H + h;
    float ac = 0.f, bc = 0.f, gn = 0.f, bn = 0.f;
    auto scalars = [&](int t) {
        const bool in = t + lane < len;
        gn = in ? ld1(gh + token_at(t + lane) * H) : 0.f;
        bn = in ? ld1(bh + token_at(t + lane) * H) : 0.f;
    };
    auto load = [&](int t, WalkToken<COLS> &x) {  // t = 0, 1, ... in turn, its group complete
        const T *row = ring[warp][t % kRing];
        if (MODE != kStates) ld_rows(row, rg, x.q);
        ld_rows(row + kN, rg, x.k);
        ldc(row + 2 * kN + COLS * (lane & 7), x.v);
        if (t % 32 == 0) {
            ac = expf(gn), bc = bn;
            scalars(t + 32);
        }
        x.a = __shfl_sync(0xffffffffu, ac, t % 32);
        x.b = __shfl_sync(0xffffffffu, bc, t % 32);
    };

    scalars(0);
#pragma unroll
    for (int j = 0; j < kGroups - 1; ++j) fetch(j * kGroup);
    uint64_t S[COLS][8];  // [column][pair of rows]
#pragma unroll
    for (int m = 0; m < 8; ++m) {
        float x[COLS] = {}, y[COLS] = {};
        if (s0 && has) {
            const float *p = s0 + state + at + (16 * (m / 2) + 2 * (m % 2)) * kN;
            ldc(p, x);
            ldc(p + kN, y);
        }
#pragma unroll
        for (int c = 0; c < COLS; ++c) S[c][m] = pack2(x[c], y[c]);
    }
    auto put = [&](float *p0) {  // the state to memory
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            float *p = p0 + at + (16 * (m / 2) + 2 * (m % 2)) * kN;
            float x[COLS], y[COLS];
#pragma unroll
            for (int c = 0; c < COLS; ++c) asm("mov.b64 {%0, %1}, %2;" : "=f"(x[c]), "=f"(y[c]) : "l"(S[c][m]));
            stc(p, x);
            stc(p + kN, y);
        }
    };
    auto checkpoint = [&](int sg) {
        const int64_t id = delta_first_segment(offsets != nullptr, seq, first, Tn) + sg;
        if (in_bounds(status, id, 1, nckpt)) put(ckpt + (id * H + h) * kN * kN);
    };
    if (MODE == kGradients && nseg > 1) checkpoint(nseg - 1);
    T *po = MODE == kOutputs ? o + (first * H + h) * kN + col : nullptr;
    auto step = [&](int t, const WalkToken<COLS> &x) {
        if constexpr (MODE == kGradients) {
            uint64_t du2[COLS] = {};
            float du[COLS];
#pragma unroll
            for (int c = 0; c < COLS; ++c) {
                const float d = scale * x.v[c];
                const uint64_t d2 = pack2(d, d);
#pragma unroll
                for (int m = 0; m < 8; ++m) S[c][m] = fma2(x.q[m], d2, S[c][m]);
            }
#pragma unroll
            for (int m = 0; m < 8; ++m)
#pragma unroll
                for (int c = 0; c < COLS; ++c) du2[c] = fma2(x.k[m], S[c][m], du2[c]);
#pragma unroll
            for (int c = 0; c < COLS; ++c) du[c] = sum2(du2[c]);
#pragma unroll
            for (int d = 8; d < 32; d *= 2)
#pragma unroll
                for (int c = 0; c < COLS; ++c) du[c] += __shfl_xor_sync(0xffffffffu, du[c], d);
            const uint64_t a2 = pack2(x.a, x.a);
#pragma unroll
            for (int c = 0; c < COLS; ++c) {
                const uint64_t w2 = pack2(-x.b * du[c], -x.b * du[c]);
#pragma unroll
                for (int m = 0; m < 8; ++m) S[c][m] = mul2(a2, fma2(x.k[m], w2, S[c][m]));
            }
            const int token = token_at(t);
            if (token % kDeltaSeg == 0) checkpoint(token / kDeltaSeg - 1);
            return;
        }
        uint64_t ks[COLS] = {}, qs[COLS] = {}, qk2 = 0;
#pragma unroll
        for (int m = 0; m < 8; ++m) {
#pragma unroll
            for (int c = 0; c < COLS; ++c) ks[c] = fma2(x.k[m], S[c][m], ks[c]);
        }
        float r[COLS], w[COLS];
#pragma unroll
        for (int c = 0; c < COLS; ++c) r[c] = sum2(ks[c]);
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            if (MODE == kStates) break;
            qk2 = fma2(x.q[m], x.k[m], qk2);
#pragma unroll
            for (int c = 0; c < COLS; ++c) qs[c] = fma2(x.q[m], S[c][m], qs[c]);
        }
        float qk = sum2(qk2);
#pragma unroll
        for (int c = 0; c < COLS; ++c) w[c] = sum2(qs[c]);
        const uint64_t a2 = pack2(x.a, x.a);
#pragma unroll
        for (int m = 0; m < 8; ++m)
#pragma unroll
            for (int c = 0; c < COLS; ++c) S[c][m] = mul2(a2, S[c][m]);
#pragma unroll
        for (int d = 8; d < 32; d *= 2) {
#pragma unroll
            for (int c = 0; c < COLS; ++c) r[c] += __shfl_xor_sync(0xffffffffu, r[c], d);
            if (MODE == kStates) continue;
            qk += __shfl_xor_sync(0xffffffffu, qk, d);
#pragma unroll
            for (int c = 0; c < COLS; ++c) w[c] += __shfl_xor_sync(0xffffffffu, w[c], d);
        }
        float out[COLS];
#pragma unroll
        for (int c = 0; c < COLS; ++c) {
            const float u = x.b * (x.v[c] - x.a * r[c]);
            const uint64_t u2 = pack2(u, u);
#pragma unroll
            for (int m = 0; m < 8; ++m) S[c][m] = fma2(x.k[m], u2, S[c][m]);
            out[c] = scale * fmaf(qk, u, x.a * w[c]);
        }
        if (MODE == kOutputs && rg == 0) stc(po + t * (H * kN), out);
        if (MODE == kStates && t % kDeltaSeg == kDeltaSeg - 1) checkpoint(t / kDeltaSeg + 1);
    };
    WalkToken<COLS> x, y;
    arrived();  // group 0
    if (len > 0) load(0, x);
    for (int t = 0; t < len; t += kGroup) {
        __syncwarp();  // every lane has read the group whose place is taken
        fetch(t + (kGroups - 1) * kGroup);
        arrived();  // the group after this one
#pragma unroll
        for (int i = 0; i < kGroup; i += 2) {  // the next token's inputs load under this one's sums
            if (t + i >= len) break;
            if (t + i + 1 < len) load(t + i + 1, y);
            step(t + i, x);
            if (t + i + 1 >= len) break;
            if (t + i + 2 < len) load(t + i + 2, x);
            step(t + i + 1, y);
        }
    }
    if (MODE == kOutputs && sT && has) put(sT + state);
    if (MODE == kGradients) asm volatile("griddepcontrol.wait;" ::: "memory");  // see the launch
}

// Shortest mean sequence that takes the second kernel.  First against second, bf16, us (B1 H4, B64
// H32): 4 tokens 8.2 / 8.2, 28.7 / 30.7; 6 tokens 10.2 / 8.2, 34.8 / 34.8; 8 tokens 12.3 / 10.2,
// 41.0 / 38.9.
constexpr int64_t kWalkTokens = 5;

// Most (sequence, head) pairs whose walks take one column a lane, in two blocks each: fewer
// instructions in a token's chain, as long as the blocks have an SM each.  Two columns against one,
// us for 128 tokens: 64 pairs fp32 37 / 35, bf16 47 / 39; 128 pairs 39 / 45, 47 / 47; 256 pairs 53 / 80,
// 64 / 72.
constexpr int64_t kNarrowPairs = 74;

template <typename T> cudaError_t launch(const DeltaArgs &a, cudaStream_t s)
{
    const int64_t pairs = a.nseq * a.H;
    const bool walk = (a.offsets ? a.T / a.nseq : a.T) >= kWalkTokens, narrow = walk && pairs <= kNarrowPairs;
    if (!walk) {
        delta_recurrent_kernel<T><<<static_cast<unsigned>(pairs), kThreads, 0, s>>>(
            a.B, a.T, a.Hk, a.H, a.nseq, a.offsets, a.nslots, a.slots, static_cast<const T *>(a.q),
            static_cast<const T *>(a.k), static_cast<const T *>(a.v), static_cast<const T *>(a.g),
            static_cast<const T *>(a.beta), a.scale, a.s0, static_cast<T *>(a.o), a.sT, a.status);
        return cudaGetLastError();
    }
    const auto kernel = narrow ? delta_walk_kernel<T, 1, kOutputs> : delta_walk_kernel<T, 2, kOutputs>;
    kernel<<<static_cast<unsigned>(narrow ? 2 * pairs : pairs), kThreads, 0, s>>>(
        a.B, a.T, a.Hk, a.H, a.nseq, a.offsets, a.nslots, a.slots, static_cast<const T *>(a.q),
        static_cast<const T *>(a.k), static_cast<const T *>(a.v), static_cast<const T *>(a.g),
        static_cast<const T *>(a.beta), a.scale, a.s0, static_cast<T *>(a.o), a.sT, nullptr, 0, a.status);
    return cudaGetLastError();
}

template <typename T> cudaError_t launch_checkpoints(const DeltaBwdArgs &b, float *states, float *grads, cudaStream_t s)
{
    const DeltaArgs &a = b.f;
    const int64_t pairs = a.nseq * a.H, ntok = a.B * a.T;
    const int64_t nckpt = delta_first_segment(a.offsets != nullptr, a.nseq, ntok, a.T);  // where one more would start
    const bool narrow = 2 * pairs <= kNarrowPairs;  // two grids at a time
    const T *q = static_cast<const T *>(a.q), *k = static_cast<const T *>(a.k), *v = static_cast<const T *>(a.v);
    const T *g = static_cast<const T *>(a.g), *beta = static_cast<const T *>(a.beta);
    const unsigned grid = static_cast<unsigned>(narrow ? 2 * pairs : pairs);
    (narrow ? delta_walk_kernel<T, 1, kStates> : delta_walk_kernel<T, 2, kStates>)<<<grid, kThreads, 0, s>>>(
        a.B, a.T, a.Hk, a.H, a.nseq, a.offsets, a.nseq, nullptr, q, k, v, g, beta, a.scale, a.s0, nullptr, nullptr, states,
        nckpt, a.status);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // The walk back needs nothing of the other and may start beside it (a programmatic launch); it ends
    // only after the other has, so that the next kernel, launched as usual, follows both.
    cudaLaunchAttribute beside[1];
    beside[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    beside[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = beside;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, narrow ? delta_walk_kernel<T, 1, kGradients> : delta_walk_kernel<T, 2, kGradients>, a.B,
                              a.T, a.Hk, a.H, a.nseq, a.offsets, a.nseq, static_cast<const int32_t *>(nullptr), q, k,
                              static_cast<const T *>(b.dout), g, beta, a.scale, b.dsT, static_cast<T *>(nullptr),
                              static_cast<float *>(nullptr), grads, nckpt, a.status);
}

}  // namespace

cudaError_t delta_checkpoints_launch(const DeltaBwdArgs &a, float *states, float *grads, cudaStream_t s)
{
    return a.f.bf16 ? launch_checkpoints<__nv_bfloat16>(a, states, grads, s) : launch_checkpoints<float>(a, states, grads, s);
}

cudaError_t delta_recurrent_launch(const DeltaArgs &a, cudaStream_t s)
{
    if (a.nseq * a.H == 0) return cudaSuccess;
    return a.bf16 ? launch<__nv_bfloat16>(a, s) : launch<float>(a, s);
}

}  // namespace wkv
