// delta_recurrent.cu -- the gated delta rule token by token (decode, a few tokens, fp32).
//
// Per sequence and value head, state S (64 x 64, row i = key channel, column j = value channel):
//   S' = exp(g_t) S,   u_t = beta_t (v_t - k_t S'),   S = S' + k_t^T u_t,   o_t = scale q_t S.
// The two products with the state are taken in one walk over it, before the update:
//   k_t S' = a (k_t S),   q_t S = a (q_t S_prev) + (q_t . k_t) u_t,   a = exp(g_t).
//
// The columns of S are independent of one another given k, so a warp owns 16 columns of one
// head and keeps them in registers for the whole sequence: lane (rg, cq) holds rows 8 rg ..
// 8 rg + 7 of columns 4 cq .. 4 cq + 3.  Sums over rows are three shuffles; no barrier, no
// shared memory.  One block is the four warps of one (sequence, head).
//
// One decoded token is bound by the state's bytes: 16 KB in and 16 KB out for each head, all of
// a warp's 4 KB loaded at once.  Long fp32 sequences are bound by the chain of one token
// (two rounds of shuffles).
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

template <typename T> cudaError_t launch(const DeltaArgs &a, cudaStream_t s)
{
    delta_recurrent_kernel<T><<<static_cast<unsigned>(a.nseq * a.H), kThreads, 0, s>>>(
        a.B, a.T, a.Hk, a.H, a.nseq, a.offsets, a.nslots, a.slots, static_cast<const T *>(a.q),
        static_cast<const T *>(a.k), static_cast<const T *>(a.v), static_cast<const T *>(a.g),
        static_cast<const T *>(a.beta), a.scale, a.s0, static_cast<T *>(a.o), a.sT, a.status);
    return cudaGetLastError();
}

}  // namespace

cudaError_t delta_recurrent_launch(const DeltaArgs &a, cudaStream_t s)
{
    if (a.nseq * a.H == 0) return cudaSuccess;
    return a.bf16 ? launch<__nv_bfloat16>(a, s) : launch<float>(a, s);
}

}  // namespace wkv
