// Device code shared by the tensor-core kernels of the gated delta rule (forward and backward):
// the state-free part of a 64-token chunk.  Internal: not part of the public ABI.
//
// With G_t the sum of the chunk's log decays up to token t, gamma_t = exp(G_t) and the ratios
// Gamma[t][i] = exp(G_t - G_i) (i <= t), the updates u of a chunk solve a unit lower triangular
// system, so with T = (I + L)^-1, L[t][i] = beta_t Gamma[t][i] k_t.k_i (i < t):
//   U = T W,   W_t = beta_t (v_t - gamma_t k_t S_prev)
//   O = scale diag(gamma) Q S_prev + P U,   P[t][i] = scale Gamma[t][i] q_t.k_i (i <= t)
//   S = gamma_63 S_prev + K^T diag(tail) U,  tail_i = exp(G_63 - G_i)
//
// Decays.  Every exponent is formed from sums over whole 16-token blocks and inside one block,
// never as a difference of two long sums, so a token that forgets everything (g of -inf or of
// a large size) costs the tokens after it no accuracy.  Inside a block log2 decays are kept as
// an integer and a fraction, which makes their differences accurate too.
//
// T.  The four 16 x 16 diagonal blocks are inverted by substitution in fp32, one warp each.  The
// rest follows from T (I + L) = I, a block row at a time from the diagonal to the left:
//   T[w][j] = -(sum_{k=j+1..w} T[w][k] L[k][j]) D[j],   D[j] = (I + L[j][j])^-1,
// which needs only L and D of other warps, never their T.  These 16-wide products are too
// small for a tcgen05 tile (and each depends on the last): they are warp-level mma.sync with
// both operands split into two bf16 terms, hi and lo, three products each (the error left is
// that of lo, 2^-16).
#pragma once

#include "tc_common.cuh"

namespace wkv {
namespace dtc {
using namespace tc;

constexpr int kC = 64;  // tokens per chunk
constexpr int kN = 64;  // head size
constexpr float kLog2e = 1.4426950408889634f;

// Shared-memory scratch of the prep group (byte offsets from its own base, 16-byte aligned).
constexpr int PR_L = 0;                         // L[k][j], k > j: six 16 x 16 blocks, hi then lo, bf16
constexpr int PR_D = PR_L + 6 * 1024;           // D[j], j < 3: hi then lo, bf16
constexpr int PR_X = PR_D + 3 * 1024;           // per warp 16 x 16 fp32: L transposed, then D
constexpr int PR_PN = PR_X + 4 * 1024;          // [64] sums of log2 decays inside the block: integer part
constexpr int PR_PF = PR_PN + 256;              // [64] fraction part
constexpr int PR_CF = PR_PF + 256;              // [64] decay from after the token to its block's end
constexpr int PR_BS = PR_CF + 256;              // [4] integer, [4] fraction parts of the blocks' sums
constexpr int PR_ARR = PR_BS + 32;              // [2 chunk parities][gamma, tail, beta][64]
constexpr int PR_BYTES = PR_ARR + 2 * 3 * 256;

__device__ __forceinline__ const float *arr(const unsigned char *pr, int c, int which)
{
    return reinterpret_cast<const float *>(pr + PR_ARR + (c & 1) * 768 + which * 256);
}
constexpr int kGamma = 0, kTail = 1, kBeta = 2;

// fp32 pair -> bf16 pair hi and the bf16 pair of what hi leaves
__device__ __forceinline__ void split2(P2 x, uint32_t *hi, uint32_t *lo)
{
    *hi = pack2(x);
    *lo = pack2(fma2(unpack2(*hi), pk(-1.f, -1.f), x));
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A 16 x 16 bf16 block (32-byte rows) as the B operand of two n = 8 products: b[0], b[1] for
// columns 0-7, b[2], b[3] for columns 8-15.
__device__ __forceinline__ void ld_b16(uint32_t (&b)[4], uint32_t block, int lane)
{
    const uint32_t at = block + (lane & 15) * 32 + (lane >> 4) * 16;
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
                 : "r"(at)
                 : "memory");
}

// One 16 x 16 operand in two bf16 terms, as the A operand of m16n8k16 (which is also where the
// accumulators of two n = 8 products lie).
struct Frag {
    uint32_t h[4], l[4];
};
__device__ __forceinline__ Frag to_frag(const float (&c)[2][4])
{
    Frag f;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) split2(pk(c[n][2 * r], c[n][2 * r + 1]), &f.h[2 * n + r], &f.l[2 * n + r]);
    return f;
}
// acc += A B, B a block held as hi then lo
__device__ __forceinline__ void mul_block(float (&acc)[2][4], const Frag &a, uint32_t block, int lane)
{
    uint32_t bh[4], bl[4];
    ld_b16(bh, block, lane);
    ld_b16(bl, block + 512, lane);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        mma16816(acc[n], a.h, bh[2 * n], bh[2 * n + 1]);
        mma16816(acc[n], a.h, bl[2 * n], bl[2 * n + 1]);
        mma16816(acc[n], a.l, bh[2 * n], bh[2 * n + 1]);
    }
}
__device__ __forceinline__ uint32_t l_block(uint32_t pr, int k, int j) { return pr + PR_L + 1024 * (k * (k - 1) / 2 + j); }

// 16 TMEM lanes x 64 columns in the layout of mma accumulators: v[n] holds columns 8 n + 2 t,
// 8 n + 2 t + 1 of row g, then of row g + 8 (g = lane / 4, t = lane % 4).
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float (&v)[8][4])
{
    uint32_t r[32];
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x8.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
                   "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
                   "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[n][e] = __uint_as_float(r[4 * n + e]);
}

// log2 of the decay as integer and fraction.  Below 2^-1000 a decay is zero in fp32 whatever
// it is multiplied by, so -inf and very large drops are cut there and sums stay exact.
__device__ __forceinline__ void split_decay(float g, float *n, float *f)
{
    float x = g * kLog2e;
    x = x < -1000.f ? -1000.f : x;
    *n = floorf(x);
    *f = x - *n;
}

// First step of a chunk, threads 0-127 of the prep group: thread t < 64 holds token t's g (0
// past the end), thread 64 + t its beta.  Writes the in-block sums, block sums, cf and beta; the
// caller's group barrier follows.
__device__ __forceinline__ void prep_scan(unsigned char *pr, int c, int tid, float x)
{
    if (tid < 64) {
        float n, f;
        split_decay(x, &n, &f);
#pragma unroll
        for (int d = 1; d < 16; d *= 2) {
            const float n1 = __shfl_up_sync(0xffffffffu, n, d, 16), f1 = __shfl_up_sync(0xffffffffu, f, d, 16);
            if ((tid & 15) >= d) {
                n += n1;
                f += f1;
            }
        }
        const float bn = __shfl_sync(0xffffffffu, n, 15, 16), bf = __shfl_sync(0xffffffffu, f, 15, 16);
        reinterpret_cast<float *>(pr + PR_PN)[tid] = n;
        reinterpret_cast<float *>(pr + PR_PF)[tid] = f;
        reinterpret_cast<float *>(pr + PR_CF)[tid] = ex2_approx((bn - n) + (bf - f));
        if ((tid & 15) == 15) {
            reinterpret_cast<float *>(pr + PR_BS)[tid >> 4] = n;
            reinterpret_cast<float *>(pr + PR_BS)[4 + (tid >> 4)] = f;
        }
    } else {
        const_cast<float *>(arr(pr, c, kBeta))[tid - 64] = x;
    }
}

// After the barrier: gamma and tail of token t (threads 0-63).
__device__ __forceinline__ void prep_decays(unsigned char *pr, int c, int tid)
{
    if (tid >= 64) return;
    const float *bs = reinterpret_cast<const float *>(pr + PR_BS);
    const int w = tid >> 4;
    const float n = reinterpret_cast<const float *>(pr + PR_PN)[tid], f = reinterpret_cast<const float *>(pr + PR_PF)[tid];
    float gn = n, gf = f, tn = bs[w] - n, tf = bs[4 + w] - f;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        if (m < w) gn += bs[m], gf += bs[4 + m];
        if (m > w) tn += bs[m], tf += bs[4 + m];
    }
    const_cast<float *>(arr(pr, c, kGamma))[tid] = ex2_approx(gn + gf);
    const_cast<float *>(arr(pr, c, kTail))[tid] = ex2_approx(tn + tf);
}

// Block row w (this warp's) of L and, with WANT_P, of P from the raw products in tensor memory
// (columns kk and qk).  Leaves L in the scratch and returns P as bf16 pairs: ph[n] holds columns
// 8 n + 2 t, + 1 of rows g and g + 8 of the block row (and pl what ph leaves, with P_LO).
template <bool WANT_P, bool P_LO>
__device__ __forceinline__ void prep_scores(unsigned char *pr, int c, int w, int lane, uint32_t kk_addr, uint32_t qk_addr,
                                            float scale, uint32_t (&ph)[8][2], uint32_t (&pl)[8][2])
{
    const float *pn = reinterpret_cast<const float *>(pr + PR_PN), *pf = reinterpret_cast<const float *>(pr + PR_PF);
    const float *cf = reinterpret_cast<const float *>(pr + PR_CF), *bs = reinterpret_cast<const float *>(pr + PR_BS);
    const float *bet = arr(pr, c, kBeta);
    const int g = lane >> 2, t = lane & 3;
    float kk[8][4], qk[8][4];
    tmem_ld_frag(kk_addr, kk);
    if (WANT_P) tmem_ld_frag(qk_addr, qk);
    const int r0 = 16 * w + g;
    const float n0 = pn[r0], n1 = pn[r0 + 8], f0 = pf[r0], f1 = pf[r0 + 8], b0 = bet[r0], b1 = bet[r0 + 8];
    float *xt = reinterpret_cast<float *>(pr + PR_X + 1024 * w);
    // decay of the whole blocks between block j and this one, from the diagonal to the left
    float mn = 0.f, mf = 0.f;
#pragma unroll
    for (int j = 3; j >= 0; --j) {
        if (j > w) {
#pragma unroll
            for (int nn = 0; nn < 2; ++nn)
#pragma unroll
                for (int r = 0; r < 2; ++r) ph[2 * j + nn][r] = pl[2 * j + nn][r] = 0;
            continue;
        }
        float l[2][4], p[2][4];
        if (j == w) {
#pragma unroll
            for (int nn = 0; nn < 2; ++nn)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int col = 8 * nn + 2 * t + (e & 1), row = g + 8 * (e >> 1);
                    const float gn = (e >> 1 ? n1 : n0) - pn[16 * w + col], gf = (e >> 1 ? f1 : f0) - pf[16 * w + col];
                    const float gam = col <= row ? ex2_approx(gn + gf) : 0.f;
                    l[nn][e] = col < row ? (e >> 1 ? b1 : b0) * gam * kk[2 * j + nn][e] : 0.f;
                    if (WANT_P) p[nn][e] = col <= row ? scale * gam * qk[2 * j + nn][e] : 0.f;
                    xt[col * 16 + row] = l[nn][e];  // transposed, for the substitution
                }
        } else {
            const float e0 = ex2_approx((n0 + mn) + (f0 + mf)), e1 = ex2_approx((n1 + mn) + (f1 + mf));
            mn += bs[j];
            mf += bs[4 + j];
            unsigned char *blk = pr + PR_L + 1024 * (w * (w - 1) / 2 + j);
#pragma unroll
            for (int nn = 0; nn < 2; ++nn) {
                const float2 cc = *reinterpret_cast<const float2 *>(cf + 16 * j + 8 * nn + 2 * t);
                const float g4[4] = {e0 * cc.x, e0 * cc.y, e1 * cc.x, e1 * cc.y};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    l[nn][e] = (e >> 1 ? b1 : b0) * g4[e] * kk[2 * j + nn][e];
                    if (WANT_P) p[nn][e] = scale * g4[e] * qk[2 * j + nn][e];
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    uint32_t hi, lo;
                    split2(pk(l[nn][2 * r], l[nn][2 * r + 1]), &hi, &lo);
                    const int at = (g + 8 * r) * 32 + (8 * nn + 2 * t) * 2;
                    *reinterpret_cast<uint32_t *>(blk + at) = hi;
                    *reinterpret_cast<uint32_t *>(blk + 512 + at) = lo;
                }
            }
        }
        if (WANT_P) {
#pragma unroll
            for (int nn = 0; nn < 2; ++nn)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    if (P_LO) {
                        split2(pk(p[nn][2 * r], p[nn][2 * r + 1]), &ph[2 * j + nn][r], &pl[2 * j + nn][r]);
                    } else {
                        ph[2 * j + nn][r] = pack_bf16(p[nn][2 * r], p[nn][2 * r + 1]);
                    }
                }
        }
    }
}

// Inverse of this warp's diagonal block: column (lane % 16) by substitution in registers.  Leaves
// D as fp32 in the warp's scratch and, for w < 3, as two bf16 terms for the other warps.
__device__ __forceinline__ void prep_diag(unsigned char *pr, int w, int lane)
{
    float *xt = reinterpret_cast<float *>(pr + PR_X + 1024 * w);
    const int j = lane & 15;
    __syncwarp();
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = i == j ? 1.f : 0.f;
#pragma unroll
    for (int k = 0; k < 15; ++k) {
        float lk[16];
#pragma unroll
        for (int q = (k + 1) / 4; q < 4; ++q) {
            const float4 v = *reinterpret_cast<const float4 *>(xt + 16 * k + 4 * q);
            lk[4 * q] = v.x, lk[4 * q + 1] = v.y, lk[4 * q + 2] = v.z, lk[4 * q + 3] = v.w;
        }
#pragma unroll
        for (int i = k + 1; i < 16; ++i) x[i] = fmaf(-lk[i], x[k], x[i]);
    }
    __syncwarp();
    unsigned char *blk = pr + PR_D + 1024 * w;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const __nv_bfloat16 hi = __float2bfloat16_rn(x[i]);
        if (lane < 16) {
            xt[16 * i + j] = x[i];
            if (w < 3) *reinterpret_cast<__nv_bfloat16 *>(blk + 32 * i + 2 * j) = hi;
        } else if (w < 3) {
            *reinterpret_cast<__nv_bfloat16 *>(blk + 512 + 32 * i + 2 * j) = __float2bfloat16_rn(x[i] - __bfloat162float(hi));
        }
    }
    __syncwarp();
}

// Block row W of T (blocks 0 .. W), in two bf16 terms; the caller's group barrier has made L
// and D of all warps visible.
template <int W> __device__ __forceinline__ void prep_inverse(const unsigned char *pr, int lane, Frag (&T)[4])
{
    const float *xt = reinterpret_cast<const float *>(pr + PR_X + 1024 * W);
    const uint32_t base = smem_u32(pr);
    const int g = lane >> 2, t = lane & 3;
    float d[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float2 x = *reinterpret_cast<const float2 *>(xt + 16 * (g + 8 * r) + 8 * n + 2 * t);
            d[n][2 * r] = x.x;
            d[n][2 * r + 1] = x.y;
        }
    T[W] = to_frag(d);
#pragma unroll
    for (int j = W - 1; j >= 0; --j) {
        float acc[2][4] = {}, out[2][4] = {};
#pragma unroll
        for (int k = W; k > j; --k) mul_block(acc, T[k], l_block(base, k, j), lane);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][e] = -acc[n][e];
        mul_block(out, to_frag(acc), base + PR_D + 1024 * j, lane);
        T[j] = to_frag(out);
    }
}

// Block row w of a swizzled 64 x 64 tile, from the layout of the fragments: columns 8 n + 2 t.
__device__ __forceinline__ void st_frag(unsigned char *tile, int w, int lane, int n, const uint32_t x0, const uint32_t x1)
{
    const int g = lane >> 2, t = lane & 3;
    *reinterpret_cast<uint32_t *>(tile + swz(16 * w + g, 16 * n + 4 * t)) = x0;
    *reinterpret_cast<uint32_t *>(tile + swz(16 * w + g + 8, 16 * n + 4 * t)) = x1;
}
template <int W> __device__ __forceinline__ void store_t(unsigned char *hi, unsigned char *lo, int lane, const Frag (&T)[4])
{
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            st_frag(hi, W, lane, 2 * j + n, T[j].h[2 * n], T[j].h[2 * n + 1]);
            st_frag(lo, W, lane, 2 * j + n, T[j].l[2 * n], T[j].l[2 * n + 1]);
        }
}

// Rows tv .. 63 of a tile to zero: a sequence's last chunk may hold tokens of the next one.
__device__ __forceinline__ void zero_rows(unsigned char *tile, int tv, int tid, int threads)
{
    for (int i = tv * 8 + tid; i < 64 * 8; i += threads)
        *reinterpret_cast<uint4 *>(tile + i * 16) = make_uint4(0u, 0u, 0u, 0u);
}

}  // namespace dtc
}  // namespace wkv
