// delta_backward.cu -- gradients of the gated delta rule by exact fp32 walks (CUDA cores).
//
// Forward, per sequence and value head (a_t = exp(g_t)):
//   S' = a_t S,   r_t = v_t - k_t S',   u_t = beta_t r_t,   S = S' + k_t^T u_t,   o_t = scale q_t S.
// With D the gradient of the state after token t, walked backwards in time:
//   D += scale q_t^T do_t
//   dq_t = scale S do_t^T,   du = k_t D,   dbeta_t = du . r_t,   dv_t = beta_t du
//   dk_t = D u_t^T - S' dv_t^T,   D' = D - k_t^T dv_t,   dg_t = <D', S'>,   D = a_t D'.
//
// In segments of 8 tokens.  Two walks side by side (delta_recurrent.cu) leave the state before every
// segment and D after it; then a block for each (segment, value head), all at once, forms the
// segment's states and updates again and walks them in reverse.  Each thread keeps its own 16
// elements of every fourth state in shared memory and forms those between once more: with the
// updates known that takes no sums, and three blocks fit on an SM where all eight states leave room
// for one.  Warp w owns columns 8 w .. 8 w + 7; lane (rg, cq) rows 8 rg .. 8 rg + 7
// of columns 2 cq, 2 cq + 1 of those.  Sums over rows are shuffles; sums over columns (dq, dk,
// dbeta, dg) leave the block's eight warps through shared memory once, added in a fixed order.
// Value heads that share a key head write their shares of dq and dk to the workspace and a second
// kernel adds them, also in a fixed order.
//
// Bound by the chain of one token in the two walks: 0.24 us a token (1024 tokens of 4 heads fp32 249
// us, where one block walking all segments of a head in turn took 1366).  With many heads, by the
// segments' instructions: 4 sequences of 128 tokens, 32 heads 147 us (181 with every state kept).  The
// tensor-core path serves longer bf16 sequences.
#include "wkv_internal.cuh"

namespace wkv {
namespace {

constexpr int kN = 64;
constexpr int kThreads = 256;
constexpr int kSeg = kDeltaSeg;
constexpr int kPart = 2 * kN + 2;  // dq, dk, dbeta, dg of one token
constexpr int kKeep = 4;  // tokens between states kept
// shared memory, floats: states [kSeg / kKeep][4][256][4], r [kSeg][64], partial sums [kSeg][8][kPart],
// exp(g) and beta [kSeg][2]; then k, v, q, do [kSeg][4][64] of T
constexpr int kStates = kSeg / kKeep * 4096;
constexpr int kSmemFloats = kStates + kSeg * kN + kSeg * 8 * kPart + kSeg * 2;
template <typename T> constexpr int kSmemBytes = kSmemFloats * 4 + kSeg * 4 * kN * static_cast<int>(sizeof(T));
static_assert(kSmemFloats % 4 == 0, "the inputs start on 16 bytes");

__device__ __forceinline__ float rd(const float *p) { return *p; }
__device__ __forceinline__ float rd(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void rd8(const float *p, float (&x)[8])
{
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void rd8(const __nv_bfloat16 *p, float (&x)[8])
{
    const uint4 w = *reinterpret_cast<const uint4 *>(p);
    const uint32_t y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(y[i] << 16);
        x[2 * i + 1] = __uint_as_float(y[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void wr(float *p, float x) { *p = x; }
__device__ __forceinline__ void wr(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

struct WalkParams {
    int64_t B, T, Hk, H, nseq;
    const int32_t *offsets;
    float scale;
    const float *s0, *dsT;
    float *ds0;
    const float *ckpt, *dckpt;  // the state before each segment, D after it: [segments][H][64][64]
    float *dq_h, *dk_h; // [B,T,H,64] shares of the value heads, or null (no shared key heads)
    int64_t nseg;       // segments of the call, the most there can be
    int *status;
};

// The segment with number id: its place in its sequence (returned, -1 if none has the number) and the
// sequence.
__device__ __forceinline__ int64_t segment_of(const WalkParams &p, int64_t id, int64_t *seq, int64_t *first, int64_t *len)
{
    int64_t i = 0;
    if (p.offsets) {
        int64_t hi = p.nseq;  // last sequence whose run starts at or before id
        while (hi - i > 1) {
            const int64_t mid = (i + hi) / 2, at = min(max(static_cast<int64_t>(p.offsets[mid]), static_cast<int64_t>(0)), p.T);
            if (at / kSeg + mid <= id) i = mid;
            else hi = mid;
        }
    } else {
        i = id / delta_first_segment(false, 1, 0, p.T);
    }
    *seq = i;
    sequence_span(p.offsets, i, p.T, first, len);
    const int64_t sg = id - delta_first_segment(p.offsets != nullptr, i, *first, p.T);
    return sg == 0 || (sg > 0 && sg * kSeg < *len) ? sg : -1;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
delta_segments_kernel(const WalkParams p, const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                      const T *__restrict__ g, const T *__restrict__ beta, const T *__restrict__ dout,
                      T *__restrict__ dq, T *__restrict__ dk, T *__restrict__ dv, T *__restrict__ dg,
                      T *__restrict__ dbeta)
{
    extern __shared__ float sm[];
    float *states = sm, *rs = sm + kStates, *part = rs + kSeg * kN, *scalars = part + kSeg * 8 * kPart;
    T *inputs = reinterpret_cast<T *>(sm + kSmemFloats);
    const int64_t id = blockIdx.x / p.H, h = blockIdx.x % p.H, hk = h / (p.H / p.Hk);
    int64_t seq, first, len;
    const int64_t sg = segment_of(p, id, &seq, &first, &len);
    if (sg < 0) return;  // a number that no segment has
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rg = lane >> 2, row = 8 * rg;
    const int col = 8 * warp + 2 * (lane & 3);
    const int64_t ntok = p.B * p.T, t0 = first + sg * kSeg;
    const int cnt = static_cast<int>(min(static_cast<int64_t>(kSeg), len - sg * kSeg));
    const bool alone = len <= kSeg;  // its sequence's only segment
    if (!in_bounds(p.status, t0, cnt, ntok) || !in_bounds(p.status, id, 1, p.nseg)) return;

    // ---- the segment's inputs to shared memory; thread i < 16 brings g or beta of one token
    {
        constexpr int kE = 16 / static_cast<int>(sizeof(T)), kQ = kN / kE;
        for (int i = tid; i < cnt * 4 * kQ; i += kThreads) {
            const int x = i / (4 * kQ), arr = i % (4 * kQ) / kQ, c = i % kQ * kE;
            const T *src = arr == 0 ? k : arr == 1 ? v : arr == 2 ? q : dout;
            src += ((t0 + x) * (arr == 0 || arr == 2 ? p.Hk : p.H) + (arr == 0 || arr == 2 ? hk : h)) * kN + c;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                             static_cast<uint32_t>(__cvta_generic_to_shared(inputs + (x * 4 + arr) * kN + c))),
                         "l"(src)
                         : "memory");
        }
        if (tid < 2 * cnt) {
            const float x = rd((tid & 1 ? beta : g) + (t0 + tid / 2) * p.H + h);
            scalars[tid] = tid & 1 ? x : expf(x);
        }
    }
    float S[8][2], D[8][2];
    const int64_t base = (seq * p.H + h) * kN * kN, ck = (id * p.H + h) * kN * kN;
    const float *s_in = sg == 0 ? (p.s0 ? p.s0 + base : nullptr) : p.ckpt + ck;
    const float *d_in = alone ? (p.dsT ? p.dsT + base : nullptr) : p.dckpt + ck;
#pragma unroll
    for (int m = 0; m < 8; ++m) {
        const int64_t at = (row + m) * kN + col;
        const float2 x = s_in ? *reinterpret_cast<const float2 *>(s_in + at) : make_float2(0.f, 0.f);
        const float2 y = d_in ? *reinterpret_cast<const float2 *>(d_in + at) : make_float2(0.f, 0.f);
        S[m][0] = x.x, S[m][1] = x.y, D[m][0] = y.x, D[m][1] = y.y;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    // ---- forward: the state before each token, r
    for (int i = 0; i < cnt; ++i) {
        if (i % kKeep == 0) {
            float4 *mine = reinterpret_cast<float4 *>(states) + i / kKeep * 1024 + tid;
#pragma unroll
            for (int m = 0; m < 4; ++m)
                mine[m * 256] = make_float4(S[2 * m][0], S[2 * m][1], S[2 * m + 1][0], S[2 * m + 1][1]);
        }
        const T *in = inputs + i * 4 * kN;
        const float a = scalars[2 * i], b = scalars[2 * i + 1];
        float kk[8], ks[2] = {}, r[2];
        rd8(in + row, kk);
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            ks[0] = fmaf(kk[m], S[m][0], ks[0]);
            ks[1] = fmaf(kk[m], S[m][1], ks[1]);
        }
#pragma unroll
        for (int d = 4; d < 32; d *= 2) {
            ks[0] += __shfl_xor_sync(0xffffffffu, ks[0], d);
            ks[1] += __shfl_xor_sync(0xffffffffu, ks[1], d);
        }
        r[0] = rd(in + kN + col) - a * ks[0];
        r[1] = rd(in + kN + col + 1) - a * ks[1];
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            S[m][0] = fmaf(kk[m], b * r[0], a * S[m][0]);
            S[m][1] = fmaf(kk[m], b * r[1], a * S[m][1]);
        }
        if (rg == 0) *reinterpret_cast<float2 *>(rs + i * kN + col) = make_float2(r[0], r[1]);
    }
    __syncwarp();
    // ---- and back
    for (int i = cnt - 1; i >= 0; --i) {
        const int64_t th = (t0 + i) * p.H + h;
        const float4 *mine = reinterpret_cast<const float4 *>(states) + i / kKeep * 1024 + tid;
        const T *in = inputs + i * 4 * kN;
        const float a = scalars[2 * i], b = scalars[2 * i + 1], d0 = rd(in + 3 * kN + col), d1 = rd(in + 3 * kN + col + 1);
        const float2 rr = *reinterpret_cast<const float2 *>(rs + i * kN + col);
        float kk[8], qq[8], pdq[8], sp[8][2], du[2] = {};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float4 x = mine[m * 256];
            sp[2 * m][0] = x.x, sp[2 * m][1] = x.y, sp[2 * m + 1][0] = x.z, sp[2 * m + 1][1] = x.w;
        }
        for (int j = i / kKeep * kKeep; j < i; ++j) {  // the state before token i
            const float aj = scalars[2 * j], bj = scalars[2 * j + 1];
            const float2 rj = *reinterpret_cast<const float2 *>(rs + j * kN + col);
            rd8(inputs + j * 4 * kN + row, kk);
#pragma unroll
            for (int m = 0; m < 8; ++m) {
                sp[m][0] = fmaf(kk[m], bj * rj.x, aj * sp[m][0]);
                sp[m][1] = fmaf(kk[m], bj * rj.y, aj * sp[m][1]);
            }
        }
#pragma unroll
        for (int m = 0; m < 8; ++m) sp[m][0] *= a, sp[m][1] *= a;
        rd8(in + row, kk);
        rd8(in + 2 * kN + row, qq);
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            D[m][0] = fmaf(p.scale * qq[m], d0, D[m][0]);
            D[m][1] = fmaf(p.scale * qq[m], d1, D[m][1]);
            du[0] = fmaf(kk[m], D[m][0], du[0]);
            du[1] = fmaf(kk[m], D[m][1], du[1]);
            pdq[m] = p.scale * (fmaf(kk[m], b * rr.x, sp[m][0]) * d0 + fmaf(kk[m], b * rr.y, sp[m][1]) * d1);
        }
#pragma unroll
        for (int d = 4; d < 32; d *= 2) {
            du[0] += __shfl_xor_sync(0xffffffffu, du[0], d);
            du[1] += __shfl_xor_sync(0xffffffffu, du[1], d);
        }
        const float v0 = b * du[0], v1 = b * du[1];
        float pdb = rg == 0 ? du[0] * rr.x + du[1] * rr.y : 0.f, pdg = 0.f, pdk[8];
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            pdk[m] = D[m][0] * (b * rr.x) + D[m][1] * (b * rr.y) - sp[m][0] * v0 - sp[m][1] * v1;
            const float e0 = fmaf(-kk[m], v0, D[m][0]), e1 = fmaf(-kk[m], v1, D[m][1]);
            pdg = fmaf(e0, sp[m][0], fmaf(e1, sp[m][1], pdg));
            D[m][0] = a * e0;
            D[m][1] = a * e1;
        }
#pragma unroll
        for (int d = 1; d < 4; d *= 2)
#pragma unroll
            for (int m = 0; m < 8; ++m) {
                pdq[m] += __shfl_xor_sync(0xffffffffu, pdq[m], d);
                pdk[m] += __shfl_xor_sync(0xffffffffu, pdk[m], d);
            }
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            pdb += __shfl_xor_sync(0xffffffffu, pdb, d);
            pdg += __shfl_xor_sync(0xffffffffu, pdg, d);
        }
        float *pp = part + (i * 8 + warp) * kPart;
        if ((lane & 3) == 0) {
#pragma unroll
            for (int m = 0; m < 8; ++m) {
                pp[row + m] = pdq[m];
                pp[kN + row + m] = pdk[m];
            }
        }
        if (lane == 0) {
            pp[2 * kN] = pdb;
            pp[2 * kN + 1] = pdg;
        }
        if (rg == 0) {
            wr(dv + th * kN + col, v0);
            wr(dv + th * kN + col + 1, v1);
        }
    }
    __syncthreads();
    for (int e = tid; e < cnt * kPart; e += kThreads) {
        const int i = e / kPart, x = e % kPart;
        float sum = 0.f;
        for (int w = 0; w < 8; ++w) sum += part[(i * 8 + w) * kPart + x];
        const int64_t t = t0 + i, th = t * p.H + h;
        if (x >= 2 * kN) wr((x == 2 * kN ? dbeta : dg) + th, sum);
        else if (p.dq_h) (x < kN ? p.dq_h : p.dk_h)[th * kN + (x & (kN - 1))] = sum;
        else wr((x < kN ? dq : dk) + th * kN + (x & (kN - 1)), sum);
    }
    if (p.ds0 && sg == 0) {
#pragma unroll
        for (int m = 0; m < 8; ++m)
            *reinterpret_cast<float2 *>(p.ds0 + base + (row + m) * kN + col) = make_float2(D[m][0], D[m][1]);
    }
}

// dq and dk of a key head: the shares of its value heads, added in order.  With offsets, only
// the tokens some sequence holds (the shares of the others were never written).
template <typename T>
__global__ void __launch_bounds__(256)
delta_sum_heads_kernel(int64_t ntok, int64_t Hk, int64_t H, int64_t nseq, const int32_t *__restrict__ offsets,
                       const float *__restrict__ dq_h, const float *__restrict__ dk_h, T *__restrict__ dq,
                       T *__restrict__ dk)
{
    const int64_t e = blockIdx.x * 256LL + threadIdx.x;  // token, key head, channel
    const int64_t t = e / (Hk * kN), hk = e / kN % Hk;
    if (t >= ntok) return;
    if (offsets) {  // the last sequence that starts at or before t
        int64_t lo = 0, hi = nseq;
        while (lo < hi) {
            const int64_t mid = (lo + hi) / 2;
            if (offsets[mid] <= t) lo = mid + 1;
            else hi = mid;
        }
        if (lo == 0 || t >= offsets[lo]) return;
    }
    const int64_t G = H / Hk;
    float a = 0.f, b = 0.f;
    for (int64_t i = 0; i < G; ++i) {
        const int64_t x = (t * H + hk * G + i) * kN + e % kN;
        a += dq_h[x];
        b += dk_h[x];
    }
    wr(dq + e, a);
    wr(dk + e, b);
}

// Numbers of segments in use and unused: where those of one more sequence would start.
int64_t segments(const DeltaArgs &a) { return delta_first_segment(a.offsets != nullptr, a.nseq, a.B * a.T, a.T); }
// Whether every sequence is known to be of one segment: no walks, no checkpoints.
bool single(const DeltaArgs &a) { return !a.offsets && a.T <= kSeg; }
int64_t checkpoint_floats(const DeltaArgs &a) { return single(a) ? 0 : segments(a) * a.H * kN * kN; }

template <typename T> cudaError_t launch(const DeltaBwdArgs &a, cudaStream_t s)
{
    const DeltaArgs &f = a.f;
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!done[dev]) {  // racing first calls set the same attribute: harmless
        e = cudaFuncSetAttribute(delta_segments_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes<T>);
        if (e != cudaSuccess) return e;
        done[dev] = true;
    }
    const int64_t ntok = f.B * f.T, nseg = segments(f), nck = checkpoint_floats(f);
    if (nseg * f.H > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    float *ck = static_cast<float *>(a.workspace), *dck = ck + nck;
    float *share = f.H == f.Hk ? nullptr : dck + nck;
    if (!single(f)) {
        e = delta_checkpoints_launch(a, ck, dck, s);
        if (e != cudaSuccess) return e;
    }
    const WalkParams p{f.B, f.T, f.Hk, f.H, f.nseq, f.offsets, f.scale, f.s0, a.dsT, a.ds0, ck, dck,
                       share, share ? share + ntok * f.H * kN : nullptr, nseg, f.status};
    delta_segments_kernel<T><<<static_cast<unsigned>(nseg * f.H), kThreads, kSmemBytes<T>, s>>>(
        p, static_cast<const T *>(f.q), static_cast<const T *>(f.k), static_cast<const T *>(f.v),
        static_cast<const T *>(f.g), static_cast<const T *>(f.beta), static_cast<const T *>(a.dout),
        static_cast<T *>(a.dq), static_cast<T *>(a.dk), static_cast<T *>(a.dv), static_cast<T *>(a.dg),
        static_cast<T *>(a.dbeta));
    e = cudaGetLastError();
    if (e == cudaSuccess && share) e = delta_sum_heads_launch(a, share, share + ntok * f.H * kN, s);
    return e;
}

}  // namespace

cudaError_t delta_sum_heads_launch(const DeltaBwdArgs &a, const float *dq_h, const float *dk_h, cudaStream_t s)
{
    const DeltaArgs &f = a.f;
    const int64_t ntok = f.B * f.T, blocks = (ntok * f.Hk * kN + 255) / 256;
    if (blocks == 0) return cudaSuccess;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (f.bf16)
        delta_sum_heads_kernel<<<static_cast<unsigned>(blocks), 256, 0, s>>>(
            ntok, f.Hk, f.H, f.nseq, f.offsets, dq_h, dk_h, static_cast<__nv_bfloat16 *>(a.dq),
            static_cast<__nv_bfloat16 *>(a.dk));
    else
        delta_sum_heads_kernel<<<static_cast<unsigned>(blocks), 256, 0, s>>>(
            ntok, f.Hk, f.H, f.nseq, f.offsets, dq_h, dk_h, static_cast<float *>(a.dq), static_cast<float *>(a.dk));
    return cudaGetLastError();
}

size_t delta_walks_workspace_bytes(const DeltaArgs &a)
{
    const int64_t shares = a.H == a.Hk ? 0 : 2 * a.B * a.T * a.H * kN;
    return static_cast<size_t>(2 * checkpoint_floats(a) + shares) * sizeof(float);
}

cudaError_t delta_backward_walks_launch(const DeltaBwdArgs &a, cudaStream_t s)
{
    if (a.f.nseq * a.f.H == 0) return cudaSuccess;
    return a.f.bf16 ? launch<__nv_bfloat16>(a, s) : launch<float>(a, s);
}

}  // namespace wkv
