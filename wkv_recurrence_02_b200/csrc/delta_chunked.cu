// delta_chunked.cu -- the gated delta rule in 64-token chunks on B200 tensor cores (tcgen05 +
// TMA + TMEM), bf16 inputs.
//
// One CTA owns one (sequence, value head) and walks it chunk by chunk with the state S (64 x 64
// fp32) in registers.  delta_tc.cuh has the chunk's algebra; T of every chunk was formed before, in
// delta_prep.cu.  (Forming T here too, in the same warps, was slower: T's code and the chain's
// together do not stay in the instruction caches, and each ran at half its speed.)  Two CTAs
// share an SM.  Per chunk:
//   chain group (warps 4-7)  S -> K S -> W -> T W = U -> K^T diag(tail) U -> S: three products,
//                            each waiting for the last; beside them scale diag(gamma) Q S + P U;
//   P group (warps 0-3)      Q K^T on the tensor core, decay ratios, P; runs ahead.
//
// Accuracy.  The state is an fp32 result, so every operand between S and the next S is two bf16
// terms, hi and lo (K and V are exact): S, W, T and diag(tail) U, three products where both
// sides are split.  What that leaves is 2^-16 of each operand.  The output is rounded to bf16,
// and there P, U and the S of Q S are single bf16.
//
// Shared memory (13 tiles of 8 KB): K, Q and T (hi, lo) of two chunks, V of one (it is read early
// in the chain), P, and three chain tiles A, B, C that take S hi/lo (A, B), W hi/lo (C, B),
// diag(tail) U hi/lo (A, B) and U (C) in turn.  Tensor memory (256 columns): Q K^T, one accumulator
// that takes K S, U and K^T U in turn, and the outputs of two chunks.
//
// Every mbarrier wait is bounded; on expiry the CTA records RWKV_ERR_TIMEOUT in the device
// status word, waits (bounded) for its own copies and MMAs, frees its tensor memory and returns.
#include "delta_tc.cuh"

namespace wkv {
namespace {
using namespace dtc;

constexpr int kThreads = 256;
constexpr int OFF_K = 0, OFF_Q = 2 * kTile, OFF_V = 4 * kTile, OFF_P = 5 * kTile, OFF_T = 6 * kTile;
constexpr int OFF_A = 10 * kTile, OFF_B = 11 * kTile, OFF_CC = 12 * kTile;
constexpr int OFF_PN = 13 * kTile;         // [64] sums of log2 decays inside the block: integer part
constexpr int OFF_PF = OFF_PN + 256;       // [64] fraction part
constexpr int OFF_CF = OFF_PF + 256;       // [64] decay from after the token to its block's end
constexpr int OFF_PRE = OFF_CF + 256;      // [64] decay from the block's start up to the token
constexpr int OFF_BS = OFF_PRE + 256;      // [4] integer, [4] fraction parts of the blocks' sums
constexpr int OFF_ARR = OFF_BS + 32;       // [chunk % 3][gamma, tail, beta][64]
constexpr int OFF_BAR = OFF_ARR + 3 * 768;
constexpr int OFF_MISC = OFF_BAR + 20 * 8;
constexpr int kSmemBytes = OFF_MISC + 32 + 1024;  // + alignment slack
static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM do not fit");
constexpr uint32_t COL_QK = 0, COL_X = 64, COL_O = 128, kTmemCols = 256;

struct Params {
    int64_t B, T, Hk, H, nseq, nslots;
    const int32_t *offsets, *slots;
    const __nv_bfloat16 *g, *beta;
    const unsigned char *t;  // [chunks][H][kTBytes]
    int64_t nchunks;         // chunks behind t
    float scale;
    const float *s0;
    __nv_bfloat16 *o;
    float *sT;
    int *status;
    uint32_t spin_limit;
    int inject_timeout;
};

__global__ void __launch_bounds__(kThreads, 2)
delta_chunked_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const Params p)
{
    extern __shared__ unsigned char smem_raw[];
    // aligned by an offset on the __shared__ array itself (not through an integer), so the
    // compiler keeps the shared state space
    unsigned char *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + OFF_BAR);
    volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(sm + OFF_MISC);  // TMEM base, abort
    const uint32_t bar_k0 = smem_u32(&bars[0]);  // K, Q, T there: + 8 * (chunk % 2)
    const uint32_t bar_q0 = smem_u32(&bars[2]);
    const uint32_t bar_t0 = smem_u32(&bars[4]);
    const uint32_t bar_v = smem_u32(&bars[6]);
    const uint32_t bar_a = smem_u32(&bars[7]);   // Q K^T done
    const uint32_t bar_x = smem_u32(&bars[8]);   // K S, U, K^T U done (three phases a chunk)
    const uint32_t bar_qs = smem_u32(&bars[9]);  // Q S done
    const uint32_t bar_o = smem_u32(&bars[10]);  // P U done
    const uint32_t bar_p = smem_u32(&bars[11]);  // P written
    const uint32_t bar_never = smem_u32(&bars[12]);
    const uint32_t bar_drain = smem_u32(&bars[13]);
    // decays written, tail rows of K and Q zeroed: + 8 * (chunk % 3), since the P group may pass
    // two more chunks here before the chain waits for this one
    const uint32_t bar_s0 = smem_u32(&bars[14]);

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform, see elect_one
    const int64_t n = blockIdx.x, seq = n / p.H, h = n % p.H, hk = h / (p.H / p.Hk);
    int64_t first, len;
    sequence_span(p.offsets, seq, p.T, &first, &len);
    const int64_t slot = sequence_slot(p.slots, seq, p.nslots, tid == 0 ? p.status : nullptr);
    const int nchunks = static_cast<int>((len + kC - 1) / kC);
    const int64_t chunk0 = first_chunk(p.offsets != nullptr, seq, first, p.T);
    // tensor-map coordinates of the sequence's first token
    const int row_b = p.offsets ? 0 : static_cast<int>(seq), row_t = p.offsets ? static_cast<int>(first) : 0;
    const uint32_t spin = p.spin_limit;
    const int64_t ntok = p.B * p.T;

    if (tid == 0) {
        for (int i = 0; i < 17; ++i) bar_init(smem_u32(&bars[i]), i == 11 ? 128 : i == 13 ? 3 : i > 13 ? 65 : 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        misc[1] = 0;
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(const_cast<uint32_t *>(misc))),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    // P and T are lower triangular: the blocks above the diagonal are zeroed once
    for (int i = tid; i < 5 * kTile / 16; i += kThreads)
        *reinterpret_cast<uint4 *>(sm + OFF_P + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
    fence_async_smem();
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tbase = misc[0];

    auto load_tile = [&](const CUtensorMap *map, uint32_t off, int64_t head, int c, uint32_t bar) {
        if (!tma_coord_ok(p.status, 0, 2, kN, row_t + static_cast<int64_t>(c) * kC, p.T)) return;
        bar_expect_tx(bar, kTile);
        tma_load_4d(smem_u32(sm + off), map, 0, static_cast<int>(head), row_t + c * kC, row_b, bar);
    };
    // T of chunk c, without its zero blocks: one warp, a copy for each of 8 core columns of each term
    auto load_t = [&](int c) {
        if (!in_bounds(p.status, chunk0 + c, 1, p.nchunks)) return;
        const uint32_t bar = bar_t0 + 8 * (c & 1);
        if (lane == 0) bar_expect_tx(bar, kTBytes);
        __syncwarp();
        if (lane < 16) {
            const int col = lane & 7, term = lane >> 3;
            bulk_load(smem_u32(sm + OFF_T + kTile * (2 * (c & 1) + term) + 1024 * col + 256 * (col >> 1)),
                      p.t + ((chunk0 + c) * p.H + h) * kTBytes + term * kTStored + t_stored_at(col),
                      (8 - 2 * (col >> 1)) * 128, bar);
        }
    };
    if (warp == 7) {
        for (int c = 0; c < 2 && c < nchunks; ++c) {
            if (elect_one()) {
                load_tile(&map_k, OFF_K + kTile * c, hk, c, bar_k0 + 8 * c);
                load_tile(&map_q, OFF_Q + kTile * c, hk, c, bar_q0 + 8 * c);
                if (c < 1) load_tile(&map_v, OFF_V, h, c, bar_v);
            }
            __syncwarp();
            load_t(c);
        }
    }
    int abort = 0;
    if (p.inject_timeout && tid == 0) abort = !bar_wait(bar_never, 0, p.spin_limit);
    abort = __syncthreads_or(abort);
    if (abort) misc[1] = 1;

    if (warp < 4) {
        // --------------------------------------------------------------------- P group
        const int w = warp;
        float *pn = reinterpret_cast<float *>(sm + OFF_PN), *pf = reinterpret_cast<float *>(sm + OFF_PF);
        float *cf = reinterpret_cast<float *>(sm + OFF_CF), *pre = reinterpret_cast<float *>(sm + OFF_PRE);
        float *bs = reinterpret_cast<float *>(sm + OFF_BS);
        // Warps 2 and 3 prepare the decays; the tokens' g and beta are loaded a chunk ahead and
        // widened only when their chunk comes, so that nothing waits for the load before.
        const int st = tid - 64;
        uint16_t g_next = 0, b_next = 0;
        auto fetch = [&](int c) {
            const int64_t t = static_cast<int64_t>(c) * kC + st;
            g_next = b_next = 0;
            if (t >= len || !in_bounds(p.status, first + t, 1, ntok)) return;
            const int64_t at = (first + t) * p.H + h;
            g_next = reinterpret_cast<const uint16_t *>(p.g)[at];
            b_next = reinterpret_cast<const uint16_t *>(p.beta)[at];
        };
        auto scan = [&](int c) {
            const float gv = __uint_as_float(static_cast<uint32_t>(g_next) << 16);
            const float bv = __uint_as_float(static_cast<uint32_t>(b_next) << 16);
            if (c + 1 < nchunks) fetch(c + 1);
            float *out = reinterpret_cast<float *>(sm + OFF_ARR + 768 * (c % 3));
            const int wb = st >> 4;
            const BlockSums s = block_sums(gv, st);
            pn[st] = s.n;
            pf[st] = s.f;
            cf[st] = ex2_approx((s.bn - s.n) + (s.bf - s.f));
            pre[st] = ex2_approx(s.n + s.f);
            out[128 + st] = bv;
            if ((st & 15) == 15) {
                bs[wb] = s.n;
                bs[4 + wb] = s.f;
            }
            group_sync<3, 64>();
            float gn = s.n, gf = s.f, tn = s.bn - s.n, tf = s.bf - s.f;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                if (m < wb) gn += bs[m], gf += bs[4 + m];
                if (m > wb) tn += bs[m], tf += bs[4 + m];
            }
            out[st] = ex2_approx(gn + gf);
            out[64 + st] = ex2_approx(tn + tf);
            bar_arrive(bar_s0 + 8 * (c % 3));
        };
        // Q K^T of chunk c (warp 0)
        auto products = [&](int c) -> int {
            unsigned char *kt = sm + OFF_K + kTile * (c & 1), *qt = sm + OFF_Q + kTile * (c & 1);
            const bool there = bar_wait(bar_k0 + 8 * (c & 1), (c >> 1) & 1, spin) &&
                               bar_wait(bar_q0 + 8 * (c & 1), (c >> 1) & 1, spin);
            if (!__all_sync(0xffffffffu, there)) return 0;
            const int64_t left = len - static_cast<int64_t>(c) * kC;
            if (left < kC) {
                zero_rows(kt, static_cast<int>(left), lane, 32);
                zero_rows(qt, static_cast<int>(left), lane, 32);
                fence_async_smem();
                __syncwarp();
            }
            fence_after();
            const uint64_t dk = desc_k(smem_u32(kt)), dq = desc_k(smem_u32(qt));
            if (elect_one()) {
                mma_tile<kStepK, kStepK, false>(tbase + COL_QK, dq, dk, idesc(64, 0, 0));
                mma_commit(bar_a);
                bar_arrive(bar_s0 + 8 * (c % 3));
            }
            __syncwarp();
            return 1;
        };
        const uint32_t qk = tbase + (static_cast<uint32_t>(32 * w) << 16) + COL_QK;
        const int g = lane >> 2, t = lane & 3, r0 = 16 * w + g;
        int ok = 1;
        if (!abort && nchunks > 0) {
            if (w >= 2) {
                fetch(0);
                scan(0);
            } else if (w == 0) {
                ok = products(0);
            }
        }
        for (int c = 0; c < nchunks && !abort; ++c) {
            group_sync<1, 128>();  // the chunk's decays are there
            if (ok) ok = bar_wait(bar_a, c & 1, spin);
            fence_after();
            float x[4][2][4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j <= w) tmem_ld_frag(qk + 16 * j, x[j]);
            const float n0 = pn[r0], n1 = pn[r0 + 8], f0 = pf[r0], f1 = pf[r0 + 8];
            const float p0 = p.scale * pre[r0], p1 = p.scale * pre[r0 + 8];
            tmem_wait_ld();
            uint32_t ph[4][4];  // block row w of P, bf16 pairs
            float mn = 0.f, mf = 0.f;  // decay of the whole blocks between block j and this one
#pragma unroll
            for (int j = 3; j >= 0; --j) {
                if (j > w) continue;
                if (j == w) {
#pragma unroll
                    for (int nn = 0; nn < 2; ++nn) {
                        const float2 cn = *reinterpret_cast<const float2 *>(pn + 16 * j + 8 * nn + 2 * t);
                        const float2 ff = *reinterpret_cast<const float2 *>(pf + 16 * j + 8 * nn + 2 * t);
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const int col = 8 * nn + 2 * t, row = g + 8 * r;
                            const float e0 = ex2_approx(((r ? n1 : n0) - cn.x) + ((r ? f1 : f0) - ff.x));
                            const float e1 = ex2_approx(((r ? n1 : n0) - cn.y) + ((r ? f1 : f0) - ff.y));
                            ph[j][2 * nn + r] = pack_bf16(col <= row ? p.scale * e0 * x[j][nn][2 * r] : 0.f,
                                                          col + 1 <= row ? p.scale * e1 * x[j][nn][2 * r + 1] : 0.f);
                        }
                    }
                    continue;
                }
                const float mid = ex2_approx(mn + mf);
                mn += bs[j];
                mf += bs[4 + j];
#pragma unroll
                for (int nn = 0; nn < 2; ++nn) {
                    const P2 cc = ld_p2(cf + 16 * j + 8 * nn + 2 * t);
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float f = mid * (r ? p1 : p0);
                        ph[j][2 * nn + r] = pack2(mul2(mul2(cc, pk(f, f)), pk(x[j][nn][2 * r], x[j][nn][2 * r + 1])));
                    }
                }
            }
            fence_before();
            if (named_sync_or(1, 128, !ok || misc[1])) {
                abort = 1;
                misc[1] = 1;
                break;
            }
            if (c + 1 < nchunks) {
                if (w >= 2) scan(c + 1);
                else if (w == 0) ok = products(c + 1);
            }
            if (ok && c > 0) ok = bar_wait(bar_o, (c - 1) & 1, spin);  // the chunk before has read P
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j <= w) st_block(sm + OFF_P, w, j, lane, ph[j]);
            fence_async_smem();
            bar_arrive(bar_p);
        }
    } else {
        // ------------------------------------------------------------------ chain group
        const int q = warp & 3;
        const uint32_t tl = tbase + (static_cast<uint32_t>(32 * q) << 16);
        const int row = 16 * q + (lane & 15), col = 32 * (lane >> 4);  // its row and first of 32 columns
        unsigned char *tA = sm + OFF_A, *tB = sm + OFF_B, *tC = sm + OFF_CC;
        const uint64_t dA = desc_mn(smem_u32(tA)), dB = desc_mn(smem_u32(tB)), dC = desc_mn(smem_u32(tC));
        const uint64_t dP = desc_k(smem_u32(sm + OFF_P));
        constexpr uint32_t kIdK = idesc(64, 0, 1), kIdMn = idesc(64, 1, 1);
        const int64_t nstate = p.nslots * p.H * kN * kN;
        const int64_t sat = ((slot * p.H + h) * kN + row) * kN + col;
        P2 S[16];
        if (p.s0 && slot >= 0 && in_bounds(p.status, sat, 32, nstate)) {
            const float4 *src = reinterpret_cast<const float4 *>(p.s0 + sat);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 x = src[i];
                S[2 * i] = pk(x.x, x.y);
                S[2 * i + 1] = pk(x.z, x.w);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) S[i] = pk(0.f, 0.f);
        }
        uint32_t at[4];  // this thread's 32 columns of a tile
#pragma unroll
        for (int i = 0; i < 4; ++i) at[i] = swz(row, 2 * col + 16 * i);
        auto store_split = [&](const P2 (&x)[16], unsigned char *th, unsigned char *tlo) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t a[4], b[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) split2(x[4 * i + e], &a[e], &b[e]);
                *reinterpret_cast<uint4 *>(th + at[i]) = make_uint4(a[0], a[1], a[2], a[3]);
                *reinterpret_cast<uint4 *>(tlo + at[i]) = make_uint4(b[0], b[1], b[2], b[3]);
            }
        };
        auto rounded = [&](const P2 (&x)[16], int i) {
            return make_uint4(pack2(x[4 * i]), pack2(x[4 * i + 1]), pack2(x[4 * i + 2]), pack2(x[4 * i + 3]));
        };
        // group barrier: what was written is ready for the products issued next.  Whether to stop
        // is voted on once a chunk (an expired wait makes the rest of its chunk's waits pass).
        auto meet = [&]() {
            fence_async_smem();
            fence_before();
            group_sync<2, 128>();
            fence_after();
        };
        auto vote = [&](int ok) -> bool {
            fence_async_smem();
            fence_before();
            const bool stop = named_sync_or(2, 128, !ok || misc[1]);
            fence_after();
            return stop;
        };
        auto store_o = [&](int c) {  // output rows of chunk c from tensor memory
            P2 x[16];
            tmem_ld_row(tl + COL_O + 64 * (c & 1), x);
            const int64_t t = static_cast<int64_t>(c) * kC + row;
            if (t < len && in_bounds(p.status, first + t, 1, ntok)) {
                uint4 *dst = reinterpret_cast<uint4 *>(p.o + ((first + t) * p.H + h) * kN + col);
#pragma unroll
                for (int i = 0; i < 4; ++i) dst[i] = rounded(x, i);
            }
        };

        int ok = 1;
        uint32_t xph = 0;  // phase of bar_x
        for (int c = 0; c < nchunks && !abort; ++c) {
            const uint32_t aK = smem_u32(sm + OFF_K + kTile * (c & 1)), co = COL_O + 64 * (c & 1);
            // ---- S hi, lo; K S and Q S
            store_split(S, tA, tB);
            if (ok) ok = bar_wait(bar_s0 + 8 * (c % 3), (c / 3) & 1, spin);
            if (vote(ok)) {
                abort = 1;
                break;
            }
            if (warp == 4) {
                const uint64_t dK = desc_k(aK);
                if (elect_one()) {
                    mma_tile<kStepK, kStepMn, false>(tbase + COL_X, dK, dA, kIdK);
                    mma_tile<kStepK, kStepMn, true>(tbase + COL_X, dK, dB, kIdK);
                    mma_commit(bar_x);
                }
                __syncwarp();
            } else if (warp == 5) {
                const uint64_t dQ = desc_k(smem_u32(sm + OFF_Q + kTile * (c & 1)));
                if (elect_one()) {
                    mma_tile<kStepK, kStepMn, false>(tbase + co, dQ, dA, kIdK);
                    mma_commit(bar_qs);
                }
                __syncwarp();
            }
            const float *arr = reinterpret_cast<const float *>(sm + OFF_ARR + 768 * (c % 3));
            const float gam = arr[row], tail = arr[64 + row], bet = arr[128 + row], gC = arr[kC - 1];
            if (c > 0) {  // the output of the chunk before, under K S
                if (ok) ok = bar_wait(bar_o, (c - 1) & 1, spin);
                fence_after();
                store_o(c - 1);
            }
            // ---- W = beta (v - gamma K S)
            P2 x[16];
            if (ok) ok = bar_wait(bar_v, c & 1, spin);
            if (ok) ok = bar_wait(bar_x, xph, spin);
            xph ^= 1;
            fence_after();
            tmem_ld_row(tl + COL_X, x);
            {
                const P2 b2 = pk(bet, bet), bg = pk(-bet * gam, -bet * gam);
                const bool token = static_cast<int64_t>(c) * kC + row < len;  // else another sequence's, or nothing
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint4 vv = make_uint4(0u, 0u, 0u, 0u);
                    if (token) vv = *reinterpret_cast<const uint4 *>(sm + OFF_V + at[i]);
                    const uint32_t vw[4] = {vv.x, vv.y, vv.z, vv.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[4 * i + e] = fma2(bg, x[4 * i + e], mul2(b2, unpack2(vw[e])));
                }
                store_split(x, tC, tB);
            }
            if (ok) ok = bar_wait(bar_t0 + 8 * (c & 1), (c >> 1) & 1, spin);
            meet();
            if (warp == 4) {  // ---- U = T W
                const uint64_t dTh = desc_t(smem_u32(sm + OFF_T + kTile * (2 * (c & 1))));
                const uint64_t dTl = desc_t(smem_u32(sm + OFF_T + kTile * (2 * (c & 1) + 1)));
                if (elect_one()) {
                    mma_tile<kStepTK, kStepMn, false>(tbase + COL_X, dTh, dC, kIdK);
                    mma_tile<kStepTK, kStepMn, true>(tbase + COL_X, dTl, dC, kIdK);
                    mma_tile<kStepTK, kStepMn, true>(tbase + COL_X, dTh, dB, kIdK);
                    mma_commit(bar_x);
                }
                __syncwarp();
            } else if (warp == 7 && c + 1 < nchunks) {
                if (elect_one()) load_tile(&map_v, OFF_V, h, c + 1, bar_v);
                __syncwarp();
            }
            // ---- scale diag(gamma) Q S in place, under T W
            if (ok) ok = bar_wait(bar_qs, c & 1, spin);
            fence_after();
            {
                float v[32];
                tmem_ld32(tl + co, v);
                const float sg = p.scale * gam;
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] *= sg;
                tmem_st32(tl + co, v);
            }
            // ---- U, and diag(tail) U hi, lo
            if (ok) ok = bar_wait(bar_x, xph, spin);
            xph ^= 1;
            fence_after();
            tmem_ld_row(tl + COL_X, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4 *>(tC + at[i]) = rounded(x, i);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = mul2(x[i], pk(tail, tail));
            store_split(x, tA, tB);
            // P is there, and so Q K^T has read its tiles; asked before P U is issued, since the P
            // group may then go on to the next phase of this barrier
            if (ok && (warp == 5 || warp == 7)) ok = bar_wait(bar_p, c & 1, spin);
            meet();
            if (warp == 4) {  // ---- K^T diag(tail) U
                const uint64_t dKt = desc_mn(aK);
                if (elect_one()) {
                    mma_tile<kStepMn, kStepMn, false>(tbase + COL_X, dKt, dA, kIdMn);
                    mma_tile<kStepMn, kStepMn, true>(tbase + COL_X, dKt, dB, kIdMn);
                    mma_commit(bar_x);
                }
                __syncwarp();
            } else if (warp == 5) {  // ---- + P U
                if (elect_one()) {
                    mma_tile<kStepK, kStepMn, true>(tbase + co, dP, dC, kIdK);
                    mma_commit(bar_o);
                }
                __syncwarp();
            } else if (warp == 7 && c + 2 < nchunks) {
                if (elect_one()) load_tile(&map_q, OFF_Q + kTile * (c & 1), hk, c + 2, bar_q0 + 8 * (c & 1));
                __syncwarp();
                load_t(c + 2);
            }
            if (ok) ok = bar_wait(bar_x, xph, spin);
            xph ^= 1;
            fence_after();
            tmem_ld_row(tl + COL_X, x);
#pragma unroll
            for (int i = 0; i < 16; ++i) S[i] = fma2(pk(gC, gC), S[i], x[i]);
            if (warp == 7 && c + 2 < nchunks) {
                if (elect_one()) load_tile(&map_k, OFF_K + kTile * (c & 1), hk, c + 2, bar_k0 + 8 * (c & 1));
                __syncwarp();
            }
        }
        if (!abort && nchunks > 0) {
            if (ok) ok = bar_wait(bar_o, (nchunks - 1) & 1, spin);
            if (vote(ok)) abort = 1;
            else store_o(nchunks - 1);
        }
        if (abort) misc[1] = 1;
        if (!abort && p.sT && slot >= 0 && in_bounds(p.status, sat, 32, nstate)) {
            float4 *dst = reinterpret_cast<float4 *>(p.sT + sat);
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i] = make_float4(lo(S[2 * i]), hi(S[2 * i]), lo(S[2 * i + 1]), hi(S[2 * i + 1]));
        }
    }

    // ---- drain after an abort, then release tensor memory
    fence_before();
    abort = __syncthreads_or(abort | misc[1]);
    fence_after();
    if (abort) {
        record_status(p.status, kStatusTimeout);
        if ((warp == 0 || warp == 4 || warp == 5) && elect_one()) mma_commit(bar_drain);  // the three issuers
        if (tid == 0) {
            bar_wait(bar_drain, 0, p.spin_limit);
            for (int i = 0; i < 7; ++i)  // copies in flight: a barrier that nothing will complete runs out
                for (uint32_t ph = 0; ph < 2; ++ph) bar_wait(smem_u32(&bars[i]), ph, 200);
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(kTmemCols));
}

}  // namespace

cudaError_t delta_chunked_launch(const DeltaArgs &a, const void *t, cudaStream_t s)
{
    if (a.nseq * a.H == 0) return cudaSuccess;
    CUtensorMap mq, mk, mv;
    if (!make_map(&mq, a.q, a.B, a.T, a.Hk) || !make_map(&mk, a.k, a.B, a.T, a.Hk) || !make_map(&mv, a.v, a.B, a.T, a.H))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(delta_chunked_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(delta_chunked_kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e != cudaSuccess) return e;
    const Params p{a.B, a.T, a.Hk, a.H, a.nseq, a.nslots, a.offsets, a.slots, static_cast<const __nv_bfloat16 *>(a.g),
                   static_cast<const __nv_bfloat16 *>(a.beta), static_cast<const unsigned char *>(t), delta_chunks(a),
                   a.scale, a.s0, static_cast<__nv_bfloat16 *>(a.o), a.sT, a.status,
                   g_chunked_inject_timeout ? 100u : 100000u, g_chunked_inject_timeout};
    delta_chunked_kernel<<<static_cast<unsigned>(a.nseq * a.H), kThreads, kSmemBytes, s>>>(mq, mk, mv, p);
    return cudaGetLastError();
}

}  // namespace wkv
