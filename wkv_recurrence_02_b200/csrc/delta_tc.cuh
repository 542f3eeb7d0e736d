// Device code shared by the tensor-core kernels of the gated delta rule.  Internal: not part of
// the public ABI.
//
// The algebra of a 64-token chunk.  With G_t the sum of the chunk's log decays up to token t,
// gamma_t = exp(G_t) and the ratios Gamma[t][i] = exp(G_t - G_i) (i <= t), the updates u of a chunk
// solve a unit lower triangular system, so with T = (I + L)^-1, L[t][i] = beta_t Gamma[t][i] k_t.k_i
// (i < t):
//   U = T W,   W_t = beta_t (v_t - gamma_t k_t S_prev)
//   O = scale diag(gamma) Q S_prev + P U,   P[t][i] = scale Gamma[t][i] q_t.k_i (i <= t)
//   S = gamma_63 S_prev + K^T diag(tail) U,  tail_i = exp(G_63 - G_i)
// T does not depend on the state: one kernel forms it for all chunks at once (delta_prep.cu) and
// the kernels that walk the chunks read it.
//
// Decays.  Every exponent is formed from sums over whole 16-token blocks and inside one block,
// never as a difference of two long sums, so a token that forgets everything (g of -inf or of
// a large size) costs the tokens after it no accuracy.  Inside a block log2 decays are kept as
// an integer and a fraction, which makes their differences accurate too.
#pragma once

#include "tc_common.cuh"

namespace wkv {
namespace dtc {
using namespace tc;

constexpr int kC = 64;  // tokens per chunk
constexpr int kN = 64;  // head size
constexpr float kLog2e = 1.4426950408889634f;

// A barrier of part of the block.
template <int ID, int COUNT> __device__ __forceinline__ void group_sync()
{
    asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(COUNT) : "memory");
}

// One lane of a warp whose control flow is uniform.  Products are issued under this, never under a
// test of the thread index: the compiler then keeps descriptors in uniform registers, and eight
// products take 134 cycles to issue instead of 497 (measured, M = N = 64).
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(p));
    return p != 0;
}

// D (+)= A B over K = 64, from the descriptors of the first of four K steps of 16.  SA, SB: a step
// in 16-byte units, 32 bytes of a swizzled K-major tile, 2048 bytes of an MN-major one.
constexpr uint32_t kStepK = 2, kStepMn = 128;
template <uint32_t SA, uint32_t SB, bool ACC>
__device__ __forceinline__ void mma_tile(uint32_t d, uint64_t a, uint64_t b, uint32_t id)
{
#pragma unroll
    for (uint32_t ks = 0; ks < 4; ++ks) mma(d, a + SA * ks, b + SB * ks, id, ACC || ks > 0);
}

// T as an operand: 8 x 8 core matrices of 128 bytes (8 rows of 16 bytes), core (r, c) of rows 8 r ..,
// columns 8 c .. at 1024 c + 128 r, no swizzle; hi, then lo.  It is stored as it lies in shared
// memory, zero blocks included: one copy of 16 KB.  (Leaving the zeros out saves 6 KB a chunk but
// takes 16 copies, which hold the warp that issues them for some 1000 cycles.)
constexpr int kTBytes = 2 * kTile;  // per chunk and head
constexpr uint32_t kStepTK = 2 * 1024 / 16, kStepTMn = 2 * 128 / 16;
__device__ __forceinline__ uint64_t udesc_plain(uint32_t addr, uint32_t lbo, uint32_t sbo)
{
    return static_cast<uint64_t>((addr >> 4) & 0x3FFF) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFF) << 16) |
           (static_cast<uint64_t>((sbo >> 4) & 0x3FFF) << 32) | (1ull << 46);
}
// read along its rows (T W): K steps of 16 columns are 2048 bytes
__device__ __forceinline__ uint64_t desc_t(uint32_t addr) { return udesc_plain(addr, 1024, 128); }
// read across them (T^T dU): K steps of 16 rows are 256 bytes
__device__ __forceinline__ uint64_t desc_tt(uint32_t addr) { return udesc_plain(addr, 128, 1024); }
// A grid (the backward pass's two walks together) that leaves every CTA an SM of its own asks for more
// shared memory than half of one: else some are put in pairs where the kernel before still holds
// other SMs (B1 T2048 H148 forward: 142 us, so 122).
constexpr int64_t kLoneCtas = 148;
constexpr int kLoneSmemBytes = 120 * 1024;

// Chunks of a call are numbered through: sequences take disjoint runs, since each needs at most
// one more than its share of the tokens.
__host__ __device__ __forceinline__ int64_t first_chunk(bool packed, int64_t seq, int64_t first, int64_t T)
{
    return packed ? first / kC + seq : seq * ((T + kC - 1) / kC);
}

// The chunk with number id: its place in its sequence (returned, -1 if no chunk has the number) and
// the sequence.  32-bit arithmetic: there are fewer than 2^31 tokens, sequences and chunks.
__device__ __forceinline__ int chunk_of(const int32_t *offsets, int64_t nseq, int64_t T, uint32_t id, int64_t *seq,
                                        int64_t *first, int64_t *len)
{
    const uint32_t tokens = static_cast<uint32_t>(T);
    if (offsets) {
        uint32_t lo = 0, hi = static_cast<uint32_t>(nseq);  // last sequence whose run starts at or before id
        while (hi - lo > 1) {
            const uint32_t mid = (lo + hi) / 2;
            const int at = min(max(offsets[mid], 0), static_cast<int>(tokens));
            if (static_cast<uint32_t>(at) / kC + mid <= id) lo = mid;
            else hi = mid;
        }
        *seq = lo;
        sequence_span(offsets, lo, T, first, len);
        const int c = static_cast<int>(id - (static_cast<uint32_t>(*first) / kC + lo));
        return c >= 0 && static_cast<int64_t>(c) * kC < *len ? c : -1;
    }
    const uint32_t per = (tokens + kC - 1) / kC;
    *seq = id / per;
    *first = *seq * T;
    *len = T;
    return static_cast<int>(id % per);
}

// fp32 pair -> bf16 pair hi and the bf16 pair of what hi leaves
__device__ __forceinline__ void split2(P2 x, uint32_t *hi, uint32_t *lo)
{
    *hi = pack2(x);
    *lo = pack2(fma2(unpack2(*hi), pk(-1.f, -1.f), x));
}

// A value loaded from tensor memory may be read only after the wait: this keeps the compiler from
// moving even a copy of it before.
__device__ __forceinline__ void after_wait(float &x) { asm volatile("" : "+f"(x)); }
__device__ __forceinline__ void after_wait(uint32_t &x) { asm volatile("" : "+r"(x)); }

// 16 TMEM lanes x 16 columns in the layout of mma.sync accumulators: v[n] holds columns 8 n + 2 t,
// 8 n + 2 t + 1 of row g, then of row g + 8 (g = lane / 4, t = lane % 4).  No wait.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float (&v)[2][4])
{
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e >> 2][e & 3] = __uint_as_float(r[e]);
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Two accumulators, APART columns apart, added: threads 0-15 hold columns c .. c + 15, threads 16-31
// those HALF further on, each thread one lane, as pairs.
template <int HALF = 32, int APART = 64> __device__ __forceinline__ void tmem_ld_sum16(uint32_t taddr, P2 (&x)[8])
{
    uint32_t a[16], b[16];
#define WKV_LD16(r, at)                                                                                              \
    asm volatile("tcgen05.ld.sync.aligned.16x32bx2.x16.b32 "                                                         \
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16], %17;"                              \
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),   \
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),          \
                   "=r"(r[15])                                                                                       \
                 : "r"(at), "n"(HALF))
    WKV_LD16(a, taddr);
    WKV_LD16(b, taddr + APART);
#undef WKV_LD16
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        after_wait(a[i]);
        after_wait(b[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = add2(pk(__uint_as_float(a[2 * i]), __uint_as_float(a[2 * i + 1])),
                    pk(__uint_as_float(b[2 * i]), __uint_as_float(b[2 * i + 1])));
}

// 16 TMEM lanes x 64 columns: threads 0-15 hold columns 0-31, threads 16-31 32-63, each thread one
// lane, as pairs.
__device__ __forceinline__ void tmem_ld_row(uint32_t taddr, P2 (&x)[16])
{
    float v[32];
    tmem_ld32(taddr, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = pk(v[2 * i], v[2 * i + 1]);
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

// Sums of the log2 decays of a 16-token block up to this token, and of the block: threads of a
// half-warp hold the block's tokens in order.
struct BlockSums {
    float n, f, bn, bf;  // to the token, of the block: integer and fraction parts
};
__device__ __forceinline__ BlockSums block_sums(float g, int t)
{
    float n, f;
    split_decay(g, &n, &f);
#pragma unroll
    for (int d = 1; d < 16; d *= 2) {
        const float n1 = __shfl_up_sync(0xffffffffu, n, d, 16), f1 = __shfl_up_sync(0xffffffffu, f, d, 16);
        if ((t & 15) >= d) {
            n += n1;
            f += f1;
        }
    }
    return {n, f, __shfl_sync(0xffffffffu, n, 15, 16), __shfl_sync(0xffffffffu, f, 15, 16)};
}

// Decays of one chunk, as a group of warps keeps them in shared memory.
struct Decays {
    float pn[kC], pf[kC];  // sums of log2 decays inside the block: integer and fraction part
    float cf[kC];          // decay from after the token to its block's end
    float pre[kC];         // decay from the block's start up to the token
    float bs[8];           // integer, fraction parts of the blocks' sums
};
struct ChunkArrays {
    float gamma[kC], tail[kC], beta[kC];
};
// Written by 64 threads (two whole warps), thread t with token t's g and beta (0 past the end);
// named barrier ID among them.
template <int ID> __device__ __forceinline__ void scan_decays(Decays &d, ChunkArrays &a, int t, float g, float beta)
{
    const int wb = t >> 4;
    const BlockSums s = block_sums(g, t);
    d.pn[t] = s.n;
    d.pf[t] = s.f;
    d.cf[t] = ex2_approx((s.bn - s.n) + (s.bf - s.f));
    d.pre[t] = ex2_approx(s.n + s.f);
    a.beta[t] = beta;
    if ((t & 15) == 15) {
        d.bs[wb] = s.n;
        d.bs[4 + wb] = s.f;
    }
    group_sync<ID, 64>();
    float gn = s.n, gf = s.f, tn = s.bn - s.n, tf = s.bf - s.f;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        if (m < wb) gn += d.bs[m], gf += d.bs[4 + m];
        if (m > wb) tn += d.bs[m], tf += d.bs[4 + m];
    }
    a.gamma[t] = ex2_approx(gn + gf);
    a.tail[t] = ex2_approx(tn + tf);
}
__device__ __forceinline__ float widen(uint16_t bf16) { return __uint_as_float(static_cast<uint32_t>(bf16) << 16); }

// Block row w of P from Q K^T in tensor memory (this warp's lanes), as bf16 pairs in the layout of
// mma.sync accumulators; pl: what ph leaves, with LO.  Blocks right of the diagonal are zero.
template <bool LO>
__device__ __forceinline__ void form_p(const Decays &d, int w, int lane, uint32_t qk, float scale, uint32_t (&ph)[4][4],
                                       uint32_t (&pl)[4][4])
{
    const int g = lane >> 2, t = lane & 3, r0 = 16 * w + g;
    const float n0 = d.pn[r0], n1 = d.pn[r0 + 8], f0 = d.pf[r0], f1 = d.pf[r0 + 8];
    const float p0 = scale * d.pre[r0], p1 = scale * d.pre[r0 + 8];
    float mn = 0.f, mf = 0.f;  // decay of the whole blocks between block j and this one
#pragma unroll
    for (int j = 3; j >= 0; --j) {
        if (j > w) {
#pragma unroll
            for (int i = 0; i < 4; ++i) ph[j][i] = pl[j][i] = 0;
            continue;
        }
        float x[2][4];
        tmem_ld_frag(qk + 16 * j, x);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) after_wait(x[i >> 2][i & 3]);
        const float mid = ex2_approx(mn + mf);
        if (j < w) mn += d.bs[j], mf += d.bs[4 + j];
#pragma unroll
        for (int nn = 0; nn < 2; ++nn) {
            P2 gam[2];
            if (j == w) {
                const int col = 8 * nn + 2 * t;
                const P2 cn = ld_p2(d.pn + 16 * j + col), ff = ld_p2(d.pf + 16 * j + col);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float e0 = ex2_approx(((r ? n1 : n0) - tc::lo(cn)) + ((r ? f1 : f0) - tc::lo(ff)));
                    const float e1 = ex2_approx(((r ? n1 : n0) - tc::hi(cn)) + ((r ? f1 : f0) - tc::hi(ff)));
                    gam[r] = pk(scale * e0, scale * e1);
                }
            } else {
                const P2 cc = ld_p2(d.cf + 16 * j + 8 * nn + 2 * t);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float f = mid * (r ? p1 : p0);
                    gam[r] = mul2(cc, pk(f, f));
                }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                P2 y = mul2(gam[r], pk(x[nn][2 * r], x[nn][2 * r + 1]));
                if (j == w) {  // masked by choice, not by a zero factor: there may be no number there
                    const int col = 8 * nn + 2 * t;
                    y = pk(col <= g + 8 * r ? tc::lo(y) : 0.f, col + 1 <= g + 8 * r ? tc::hi(y) : 0.f);
                }
                if (LO) split2(y, &ph[j][2 * nn + r], &pl[j][2 * nn + r]);
                else ph[j][2 * nn + r] = pack2(y);
            }
        }
    }
}

// A block of a swizzled 64 x 64 tile (rows 16 w, columns 16 j) from mma.sync accumulators' layout.
__device__ __forceinline__ void st_block(unsigned char *tile, int w, int j, int lane, const uint32_t (&x)[4])
{
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint32_t *>(tile + swz(16 * w + g + 8 * (i & 1), 32 * j + 16 * (i >> 1) + 4 * t)) = x[i];
}

// Rows tv .. 63 of a tile to zero: a sequence's last chunk may hold tokens of the next one.
__device__ __forceinline__ void zero_rows(unsigned char *tile, int tv, int tid, int threads)
{
    for (int i = tv * 8 + tid; i < 64 * 8; i += threads)
        *reinterpret_cast<uint4 *>(tile + i * 16) = make_uint4(0u, 0u, 0u, 0u);
}

}  // namespace dtc
}  // namespace wkv
