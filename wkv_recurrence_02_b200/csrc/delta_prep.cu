// delta_prep.cu -- T = (I + L)^-1 of every 64-token chunk of the gated delta rule, all chunks at
// once (bf16 inputs).  delta_tc.cuh has the chunk's algebra.
//
// One block of four warps per (chunk, value head).  K arrives by TMA; K K^T and everything after
// it are 16-wide blocks in registers (mma.sync): the inverse is a chain of 16 x 16 x 16 products,
// each too small for a tcgen05 tile and each waiting for the last, and blocks that stay in
// registers from K K^T on need no trip through tensor memory.  What carries it instead is that
// five or so blocks share an SM and nothing waits for another chunk.
//
//   L       warp w forms block column w of L from the blocks of K K^T right of the diagonal in block
//           row w (K K^T is symmetric), which puts L in the register order of a B operand.
//   D[w]    inverse of the diagonal block by substitution in fp32, a column per lane, two blocks a warp.
//   T       T10 = -(D1 L10) D0              T21 = -Z D1, Z = D2 L21     T20 = -(D2 L20 D0 + Z T10)
//           T32 = -(D3 L32) D2              T31 = -Y D1, Y = D3 L31 + T32 L21
//           T30 = -((D3 L30 + T32 L20) D0 + Y T10)
//           with both operands split into two bf16 terms, hi and lo, three products each (the
//           error left is that of lo, 2^-16): T enters the fp32 state.
//
// T is written as its two terms in the order in which the walking kernels hold it in shared memory;
// a warp's store is one 128-byte line.
//
// Measured: 158 thousand cycles, 84 to 91 us by the clock, for B8 T4096 H32 (402 MB, 4.4 to 4.8 TB/s;
// 168 thousand before D's places were chosen against bank conflicts and the diagonal blocks of K K^T
// took their B operand from the A one).  Issue is 60 % active, the shared-memory pipe about as busy
// (24 block operands and the substitution's columns a chunk).
#include "delta_tc.cuh"

namespace wkv {
namespace {
using namespace dtc;

constexpr int kThreads = 128;
// shared memory: K tile, L blocks, per warp the diagonal block of L by columns and then D, T10
// (a block of L, D or T is 1 KB: hi, then lo, 16 bytes for every lane as a B operand), decays
// a diagonal block: L by columns of 20 floats (no two of a warp's stores meet in a bank), then D
constexpr int kXRow = 20, kXBytes = 16 * kXRow * 4;
constexpr int OFF_L = kTile, OFF_X = OFF_L + 6 * 1024, OFF_T10 = OFF_X + 4 * kXBytes;
constexpr int OFF_PN = OFF_T10 + 1024;     // [64] sums of log2 decays inside the block: integer part
constexpr int OFF_PF = OFF_PN + 256;       // [64] fraction part
constexpr int OFF_CF = OFF_PF + 256;       // [64] decay from after the token to its block's end
constexpr int OFF_PB = OFF_CF + 256;       // [64] beta times the decay from the block's start to the token
constexpr int OFF_BETA = OFF_PB + 256;     // [64]
constexpr int OFF_BS = OFF_BETA + 256;     // [4] integer, [4] fraction parts of the blocks' sums
constexpr int OFF_BAR = OFF_BS + 32;
constexpr int kSmemBytes = OFF_BAR + 16 + 1024;  // + alignment slack

struct Params {
    int64_t B, T, Hk, H, nseq;
    const int32_t *offsets;
    const __nv_bfloat16 *g, *beta;
    unsigned char *t_out;   // [chunks][H][kTBytes]
    int64_t nchunks;        // chunks of the call, the most there can be
    int *status;
    uint32_t spin_limit;
    int inject_timeout;
};

// One 16 x 16 operand in two bf16 terms.  As A (and as the accumulators of two n = 8 products lie):
// h[i] holds columns 8 (i / 2) + 2 t, + 1 of row g + 8 (i % 2), with g = lane / 4, t = lane % 4.  As
// B: h[i] holds rows 8 (i % 2) + 2 t, + 1 of column g + 8 (i / 2).
struct Frag {
    uint32_t h[4], l[4];
};
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at)
                 : "memory");
}
// A operand <-> B operand of the same block: the four 8 x 8 matrices transposed in place.
__device__ __forceinline__ Frag turn(const Frag &f)
{
    Frag o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(o.h[i]) : "r"(f.h[i]));
        asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(o.l[i]) : "r"(f.l[i]));
    }
    return o;
}
// Where lane (g, t)'s 16 bytes of D lie: written column by column and read lane by lane, both without
// two accesses in a bank.
__device__ __forceinline__ int d_slot(int g, int t) { return 16 * (8 * t + (g ^ (2 * t))); }
__device__ __forceinline__ Frag ld_at(const unsigned char *block, int at)
{
    const uint4 h = *reinterpret_cast<const uint4 *>(block + at);
    const uint4 l = *reinterpret_cast<const uint4 *>(block + 512 + at);
    return {{h.x, h.y, h.z, h.w}, {l.x, l.y, l.z, l.w}};
}
__device__ __forceinline__ Frag ld_block(const unsigned char *block, int lane) { return ld_at(block, 16 * lane); }
__device__ __forceinline__ void put_block(unsigned char *block, int lane, const Frag &f)
{
    *reinterpret_cast<uint4 *>(block + 16 * lane) = make_uint4(f.h[0], f.h[1], f.h[2], f.h[3]);
    *reinterpret_cast<uint4 *>(block + 512 + 16 * lane) = make_uint4(f.l[0], f.l[1], f.l[2], f.l[3]);
}
// acc += A B; the cross terms go to accumulators of their own, so that they do not wait for hi hi
__device__ __forceinline__ void mul_block(float (&acc)[2][2][4], const Frag &a, const Frag &b)
{
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        mma16816(acc[0][n], a.h, b.h[2 * n], b.h[2 * n + 1]);
        mma16816(acc[1][n], a.h, b.l[2 * n], b.l[2 * n + 1]);
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) mma16816(acc[1][n], a.l, b.h[2 * n], b.h[2 * n + 1]);
}
__device__ __forceinline__ Frag sum_frag(const float (&acc)[2][2][4], float sign)
{
    Frag f;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const P2 s = mul2(add2(pk(acc[0][n][2 * r], acc[0][n][2 * r + 1]), pk(acc[1][n][2 * r], acc[1][n][2 * r + 1])),
                              pk(sign, sign));
            split2(s, &f.h[2 * n + r], &f.l[2 * n + r]);
        }
    return f;
}
__device__ __forceinline__ Frag times(const Frag &a, const Frag &b, float sign)
{
    float acc[2][2][4] = {};
    mul_block(acc, a, b);
    return sum_frag(acc, sign);
}
__device__ __forceinline__ Frag times2(const Frag &a, const Frag &b, const Frag &a2, const Frag &b2, float sign)
{
    float acc[2][2][4] = {};
    mul_block(acc, a, b);
    mul_block(acc, a2, b2);
    return sum_frag(acc, sign);
}

__global__ void __launch_bounds__(kThreads)
delta_prep_kernel(const __grid_constant__ CUtensorMap map_k, const Params p)
{
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, lane = tid & 31;
    const int w = __shfl_sync(0xffffffffu, tid >> 5, 0);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the walk waits for this grid itself
    const uint32_t heads = static_cast<uint32_t>(p.H), id = blockIdx.x / heads;
    const int64_t h = blockIdx.x % heads, hk = static_cast<uint32_t>(h) / (heads / static_cast<uint32_t>(p.Hk));
    int64_t seq, first, len;
    const int c = chunk_of(p.offsets, p.nseq, p.T, id, &seq, &first, &len);
    if (c < 0) return;  // a number that no chunk has
    const int64_t t0 = first + static_cast<int64_t>(c) * kC, ntok = p.B * p.T;
    const int tv = static_cast<int>(len - (t0 - first) < kC ? len - (t0 - first) : kC);
    const uint32_t bar = smem_u32(sm + OFF_BAR);
    if (p.inject_timeout) {  // no copy is started that the barrier could tell of
        if (tid == 0) {
            bar_init(bar, 1);
            if (!bar_wait(bar, 0, p.spin_limit)) record_status(p.status, kStatusTimeout);
        }
        return;
    }
    if (tid == 0) {
        bar_init(bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        const int row_b = p.offsets ? 0 : static_cast<int>(seq), row_t = static_cast<int>(p.offsets ? t0 : t0 - first);
        if (tma_coord_ok(p.status, 0, 2, kN, row_t, p.T)) {
            bar_expect_tx(bar, kTile);
            tma_load_4d(smem_u32(sm), &map_k, 0, static_cast<int>(hk), row_t, row_b, bar);
        }
    }
    float *pn = reinterpret_cast<float *>(sm + OFF_PN), *pf = reinterpret_cast<float *>(sm + OFF_PF);
    float *cf = reinterpret_cast<float *>(sm + OFF_CF), *pb = reinterpret_cast<float *>(sm + OFF_PB);
    float *bt = reinterpret_cast<float *>(sm + OFF_BETA), *bs = reinterpret_cast<float *>(sm + OFF_BS);
    if (tid < 64) {
        float g = 0.f, b = 0.f;
        if (tid < tv && in_bounds(p.status, t0 + tid, 1, ntok)) {
            g = __bfloat162float(p.g[(t0 + tid) * p.H + h]);
            b = __bfloat162float(p.beta[(t0 + tid) * p.H + h]);
        }
        const BlockSums s = block_sums(g, tid);
        pn[tid] = s.n;
        pf[tid] = s.f;
        cf[tid] = ex2_approx((s.bn - s.n) + (s.bf - s.f));
        pb[tid] = b * ex2_approx(s.n + s.f);
        bt[tid] = b;
        if ((tid & 15) == 15) {
            bs[tid >> 4] = s.n;
            bs[4 + (tid >> 4)] = s.f;
        }
    }
    __syncthreads();
    int ok = bar_wait(bar, 0, p.spin_limit);
    if (tv < kC) {
        zero_rows(sm, tv, tid, kThreads);
        __syncthreads();
    }
    // ---- K K^T: block row w from the diagonal to the right
    float acc[4][2][4] = {};
    {
        const uint32_t base = smem_u32(sm);
        const int g8 = lane & 7, sel = lane >> 3;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            uint32_t a[4];
            ldmatrix4(a, base + swz(16 * w + g8 + 8 * (sel & 1), 32 * ks + 16 * (sel >> 1)));
#pragma unroll
            for (int nn = 0; nn < 2; ++nn) mma16816(acc[0][nn], a, a[nn], a[2 + nn]);  // as B: the same rows of K
#pragma unroll
            for (int j = 1; j < 4; ++j)  // acc[j]: block column w + j
                if (w + j < 4) {
                    uint32_t b[4];
                    ldmatrix4(b, base + swz(16 * (w + j) + g8 + 8 * (sel >> 1), 32 * ks + 16 * (sel & 1)));
                    mma16816(acc[j][0], a, b[0], b[1]);
                    mma16816(acc[j][1], a, b[2], b[3]);
                }
        }
    }
    const int g = lane >> 2, t = lane & 3, r0 = 16 * w + g;
    // ---- L: the diagonal block by columns
    {
        float *xt = reinterpret_cast<float *>(sm + OFF_X + kXBytes * w);
        const float n0 = pn[r0], n1 = pn[r0 + 8], f0 = pf[r0], f1 = pf[r0 + 8], b0 = bt[r0], b1 = bt[r0 + 8];
#pragma unroll
        for (int nn = 0; nn < 2; ++nn) {
            const float2 cn = *reinterpret_cast<const float2 *>(pn + 16 * w + 8 * nn + 2 * t);
            const float2 ff = *reinterpret_cast<const float2 *>(pf + 16 * w + 8 * nn + 2 * t);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int col = 8 * nn + 2 * t + (e & 1), row = g + 8 * (e >> 1);
                const float gam = ex2_approx(((e >> 1 ? n1 : n0) - (e & 1 ? cn.y : cn.x)) + ((e >> 1 ? f1 : f0) - (e & 1 ? ff.y : ff.x)));
                xt[col * kXRow + row] = col < row ? (e >> 1 ? b1 : b0) * gam * acc[0][nn][e] : 0.f;
            }
        }
    }
    // ---- L[j][w], j > w, turned: rows i to the block's end, the blocks between, columns t from
    // their block's start
    {
        const float cf0 = cf[r0], cf1 = cf[r0 + 8];
        float mn = 0.f, mf = 0.f;
#pragma unroll
        for (int jj = 1; jj < 4; ++jj) {
            const int j = w + jj;
            if (j > 3) break;
            const float mid = ex2_approx(mn + mf);
            mn += bs[j];
            mf += bs[4 + j];
            Frag f;
#pragma unroll
            for (int nn = 0; nn < 2; ++nn) {
                const P2 cc = ld_p2(pb + 16 * j + 8 * nn + 2 * t);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float s = mid * (r ? cf1 : cf0);
                    split2(mul2(mul2(cc, pk(s, s)), pk(acc[jj][nn][2 * r], acc[jj][nn][2 * r + 1])), &f.h[2 * r + nn],
                           &f.l[2 * r + nn]);
                }
            }
            put_block(sm + OFF_L + 1024 * (j * (j - 1) / 2 + w), lane, f);
        }
    }
    __syncthreads();
    // ---- D: warps 2 and 3 (which had the least of L to form), a block in each half-warp, a column in
    // each lane, by substitution in registers; the next column of L loads under the current one's
    // updates
    if (w >= 2) {
        const int blk = 2 * (w - 2) + (lane >> 4), j = lane & 15;
        const float4 *xt = reinterpret_cast<const float4 *>(sm + OFF_X + kXBytes * blk);
        P2 x[8], la[8], lb[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = pk(2 * i == j ? 1.f : 0.f, 2 * i + 1 == j ? 1.f : 0.f);
        auto fetch = [&](int k, P2 (&l)[8]) {
#pragma unroll
            for (int q = (k + 1) / 4; q < 4; ++q) {
                const float4 v = xt[kXRow / 4 * k + q];
                l[2 * q] = pk(v.x, v.y);
                l[2 * q + 1] = pk(v.z, v.w);
            }
        };
        // rows of L at or above k are zero in column k: the pair that holds row k is updated whole
        auto update = [&](int k, const P2 (&l)[8]) {
            const float xk = k & 1 ? hi(x[k / 2]) : lo(x[k / 2]);
            const P2 m = pk(-xk, -xk);
#pragma unroll
            for (int i = (k + 1) / 2; i < 8; ++i) x[i] = fma2(l[i], m, x[i]);
        };
        fetch(0, la);
#pragma unroll
        for (int k = 0; k < 15; k += 2) {
            if (k + 1 < 15) fetch(k + 1, lb);
            update(k, la);
            if (k + 2 < 15) fetch(k + 2, la);
            if (k + 1 < 15) update(k + 1, lb);
        }
        uint32_t dh[8], dl[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) split2(x[i], &dh[i], &dl[i]);
        __syncwarp();
        unsigned char *at = sm + OFF_X + kXBytes * blk + 8 * (j >> 3);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            *reinterpret_cast<uint2 *>(at + d_slot(j & 7, q)) = make_uint2(dh[q], dh[4 + q]);
            *reinterpret_cast<uint2 *>(at + 512 + d_slot(j & 7, q)) = make_uint2(dl[q], dl[4 + q]);
        }
    }
    if (__syncthreads_or(!ok)) {
        if (tid == 0) {
            record_status(p.status, kStatusTimeout);
            bar_wait_spin(bar, 0, 64u * p.spin_limit);  // the copy in flight
        }
        return;
    }
    // ---- T
    unsigned char *const tout = p.t_out + (static_cast<int64_t>(id) * p.H + h) * kTBytes;
    if (!in_bounds(p.status, id, 1, p.nchunks)) return;
    auto L = [&](int k, int j) { return ld_block(sm + OFF_L + 1024 * (k * (k - 1) / 2 + j), lane); };
    auto D = [&](int j) { return ld_at(sm + OFF_X + kXBytes * j, d_slot(g, t)); };
    auto put = [&](int i, int j, const Frag &f) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            unsigned char *at = tout + (2 * j + (q >> 1)) * 1024 + (2 * i + (q & 1)) * 128 + 4 * lane;
            *reinterpret_cast<uint32_t *>(at) = f.h[q];
            *reinterpret_cast<uint32_t *>(at + kTile) = f.l[q];
        }
    };
    if (tid < 96) {  // the blocks above the diagonal: core columns 2 .. 7, the rows above 16 (c / 2)
        const int c = 2 + tid / 16, at = 1024 * c + 16 * (tid % 16);
#pragma unroll
        for (int r = 0; r < 3; ++r)
            if (r < c / 2) {
                *reinterpret_cast<uint4 *>(tout + at + 256 * r) = make_uint4(0u, 0u, 0u, 0u);
                *reinterpret_cast<uint4 *>(tout + kTile + at + 256 * r) = make_uint4(0u, 0u, 0u, 0u);
            }
    }
    if (w == 0) {
        const Frag d0 = D(0), d1 = D(1), l10 = L(1, 0), a1 = turn(d1);
        const Frag t10 = times(times(a1, l10, 1.f), d0, -1.f);
        put_block(sm + OFF_T10, lane, turn(t10));
        group_sync<1, 96>();
        put(0, 0, turn(d0));
        put(1, 0, t10);
        put(1, 1, a1);
    } else if (w == 1) {
        const Frag l21 = L(2, 1), l20 = L(2, 0), d0 = D(0), d1 = D(1), a2 = turn(D(2));
        const Frag z = times(a2, l21, 1.f), y = times(a2, l20, 1.f);
        put(2, 1, times(z, d1, -1.f));
        put(2, 2, a2);
        group_sync<1, 96>();
        put(2, 0, times2(y, d0, z, ld_block(sm + OFF_T10, lane), -1.f));
    } else {
        const Frag a3 = turn(D(3)), l32 = L(3, 2), d2 = D(2);
        const Frag t32 = times(times(a3, l32, 1.f), d2, -1.f);
        const Frag y = times2(a3, L(3, 1), t32, L(2, 1), 1.f);
        if (w == 2) {
            put(3, 3, a3);
            put(3, 2, t32);
            put(3, 1, times(y, D(1), -1.f));
        } else {
            const Frag z = times2(a3, L(3, 0), t32, L(2, 0), 1.f);
            group_sync<1, 96>();
            put(3, 0, times2(z, D(0), y, ld_block(sm + OFF_T10, lane), -1.f));
        }
    }
}

}  // namespace

// Chunks a call is numbered with, the most there can be.
int64_t delta_chunks(const DeltaArgs &a)
{
    return a.offsets ? a.T / kC + a.nseq : a.B * ((a.T + kC - 1) / kC);
}
size_t delta_t_bytes(const DeltaArgs &a) { return static_cast<size_t>(delta_chunks(a) * a.H) * kTBytes; }

cudaError_t delta_prep_launch(const DeltaArgs &a, void *t_out, cudaStream_t s)
{
    const int64_t chunks = delta_chunks(a);
    if (chunks * a.H == 0) return cudaSuccess;
    if (chunks * a.H > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    CUtensorMap mk;
    if (!make_map(&mk, a.k, a.B, a.T, a.Hk)) return cudaErrorInvalidValue;
    const Params p{a.B, a.T, a.Hk, a.H, a.nseq, a.offsets, static_cast<const __nv_bfloat16 *>(a.g),
                   static_cast<const __nv_bfloat16 *>(a.beta), static_cast<unsigned char *>(t_out), chunks, a.status,
                   g_chunked_inject_timeout ? 100u : 100000u, g_chunked_inject_timeout};
    delta_prep_kernel<<<static_cast<unsigned>(chunks * a.H), kThreads, kSmemBytes, s>>>(mk, p);
    return cudaGetLastError();
}

}  // namespace wkv
