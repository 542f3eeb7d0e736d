// delta_chunked.cu -- the gated delta rule in 64-token chunks on B200 tensor cores (tcgen05 +
// TMA + TMEM), bf16 inputs.
//
// One CTA owns one (sequence, value head) and walks it chunk by chunk with the state S (64 x 64
// fp32) in registers.  delta_tc.cuh has the chunk's algebra and its state-free part.  With two
// CTAs per SM, per chunk:
//   prep group (warps 0-3)   Q K^T and K K^T on the tensor core, decay ratios, P, T = (I + L)^-1;
//                            runs ahead, during the chain of the chunk before;
//   chain group (warps 4-7)  S -> K S -> W -> T W = U -> K^T diag(tail) U -> S: three products,
//                            each waiting for the last; beside them scale diag(gamma) Q S + P U.
//
// Accuracy.  The state is an fp32 result, so every operand between S and the next S is two bf16
// terms, hi and lo (K and V are exact): S, W, T and diag(tail) U, three products where both
// sides are split.  What that leaves is 2^-16 of each operand.  The output is rounded to bf16,
// and there P, U and the S of Q S are single bf16.
//
// Shared memory (12 tiles of 8 KB): K of three chunks (the chain's, the prep's, one in flight),
// Q of two, V of one (it is read early in the chain), P, T hi and lo, and three chain tiles A, B,
// C that take S hi/lo (A, B), W hi/lo (C, B), diag(tail) U hi/lo (A, B) and U (C) in turn.
// Tensor memory (256 columns): Q K^T, K K^T, one accumulator that takes K S, U and K^T U in
// turn, and the output's.
//
// Every mbarrier wait is bounded; on expiry the CTA records RWKV_ERR_TIMEOUT in the device
// status word, waits (bounded) for its own copies and MMAs, frees its tensor memory and returns.
#include "delta_tc.cuh"

namespace wkv {
namespace {
using namespace dtc;

constexpr int kThreads = 256;
constexpr int OFF_K = 0, OFF_Q = 3 * kTile, OFF_V = 5 * kTile, OFF_P = 6 * kTile, OFF_T = 7 * kTile;
constexpr int OFF_A = 9 * kTile, OFF_B = 10 * kTile, OFF_CC = 11 * kTile;
constexpr int OFF_PR = 12 * kTile;
constexpr int OFF_BAR = OFF_PR + PR_BYTES;
constexpr int OFF_MISC = OFF_BAR + 16 * 8;
constexpr int kSmemBytes = OFF_MISC + 32 + 1024;  // + alignment slack
static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM do not fit");
constexpr uint32_t COL_QK = 0, COL_KK = 64, COL_X = 128, COL_O = 192, kTmemCols = 256;

struct Params {
    int64_t B, T, Hk, H, nseq, nslots;
    const int32_t *offsets, *slots;
    const __nv_bfloat16 *g, *beta;
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
    unsigned char *pr = sm + OFF_PR;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + OFF_BAR);
    volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(sm + OFF_MISC);  // TMEM base, abort
    const uint32_t bar_k0 = smem_u32(&bars[0]);  // + 8 * (chunk % 3)
    const uint32_t bar_q0 = smem_u32(&bars[3]);  // + 8 * (chunk % 2)
    const uint32_t bar_v = smem_u32(&bars[5]);
    const uint32_t bar_a = smem_u32(&bars[6]);   // Q K^T and K K^T done
    const uint32_t bar_t = smem_u32(&bars[7]);   // P, T and the decays written
    const uint32_t bar_tf = smem_u32(&bars[8]);  // U done: T may be written
    const uint32_t bar_x = smem_u32(&bars[9]);   // K S, U, K^T U done (three phases a chunk)
    const uint32_t bar_qs = smem_u32(&bars[10]); // Q S done
    const uint32_t bar_o = smem_u32(&bars[11]);  // P U done
    const uint32_t bar_never = smem_u32(&bars[12]);
    const uint32_t bar_drain = smem_u32(&bars[13]);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t n = blockIdx.x, seq = n / p.H, h = n % p.H, hk = h / (p.H / p.Hk);
    int64_t first, len;
    sequence_span(p.offsets, seq, p.T, &first, &len);
    const int64_t slot = sequence_slot(p.slots, seq, p.nslots, tid == 0 ? p.status : nullptr);
    const int nchunks = static_cast<int>((len + kC - 1) / kC);
    // tensor-map coordinates of the sequence's first token
    const int row_b = p.offsets ? 0 : static_cast<int>(seq), row_t = p.offsets ? static_cast<int>(first) : 0;
    const uint32_t spin = p.spin_limit * 64u;
    const int64_t ntok = p.B * p.T;

    if (tid == 0) {
        for (int i = 0; i < 14; ++i) bar_init(smem_u32(&bars[i]), i == 7 ? 128 : i == 13 ? 3 : 1);
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
    for (int i = tid; i < 3 * kTile / 16; i += kThreads)
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
    const int tma_thread = 128 + 96;
    if (tid == tma_thread) {
        for (int c = 0; c < 3 && c < nchunks; ++c) {
            load_tile(&map_k, OFF_K + kTile * c, hk, c, bar_k0 + 8 * c);
            if (c < 2) load_tile(&map_q, OFF_Q + kTile * c, hk, c, bar_q0 + 8 * c);
            if (c < 1) load_tile(&map_v, OFF_V, h, c, bar_v);
        }
    }
    int abort = 0;
    if (p.inject_timeout && tid == 0) abort = !bar_wait(bar_never, 0, p.spin_limit);
    abort = __syncthreads_or(abort);
    if (abort) misc[1] = 1;

    if (warp < 4) {
        // ------------------------------------------------------------------ prep group
        auto token = [&](int c) -> float {  // this thread's g (threads 0-63) or beta of chunk c
            const int64_t t = static_cast<int64_t>(c) * kC + (tid & 63);
            if (t >= len || !in_bounds(p.status, first + t, 1, ntok)) return 0.f;
            return __bfloat162float((tid < 64 ? p.g : p.beta)[(first + t) * p.H + h]);
        };
        float next = nchunks > 0 ? token(0) : 0.f;
        for (int c = 0; c < nchunks && !abort; ++c) {
            unsigned char *kt = sm + OFF_K + kTile * (c % 3), *qt = sm + OFF_Q + kTile * (c & 1);
            const int64_t left = len - static_cast<int64_t>(c) * kC;
            const int tv = static_cast<int>(left < kC ? left : kC);
            prep_scan(pr, c, tid, next);
            if (c + 1 < nchunks) next = token(c + 1);
            int ok = bar_wait_spin(bar_k0 + 8 * (c % 3), (c / 3) & 1, spin);
            if (ok) ok = bar_wait_spin(bar_q0 + 8 * (c & 1), (c >> 1) & 1, spin);
            if (tv < kC) {
                if (ok) ok = bar_wait_spin(bar_v, c & 1, spin);
                if (ok) {
                    zero_rows(kt, tv, tid, 128);
                    zero_rows(qt, tv, tid, 128);
                    zero_rows(sm + OFF_V, tv, tid, 128);
                }
                fence_async_smem();
            }
            fence_before();  // the reads of the last chunk's products are done
            if (named_sync_or(1, 128, !ok || misc[1])) {
                abort = 1;
                misc[1] = 1;
                break;
            }
            if (tid == 0) {
                fence_after();
                const uint32_t aK = smem_u32(kt), aQ = smem_u32(qt);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma(tbase + COL_KK, desc_k(aK + 32 * ks), desc_k(aK + 32 * ks), idesc(64, 0, 0), ks > 0);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma(tbase + COL_QK, desc_k(aQ + 32 * ks), desc_k(aK + 32 * ks), idesc(64, 0, 0), ks > 0);
                mma_commit(bar_a);
            }
            prep_decays(pr, c, tid);
            ok = bar_wait_spin(bar_a, c & 1, spin);
            fence_after();
            const uint32_t lanes = tbase + (static_cast<uint32_t>(32 * warp) << 16);
            uint32_t ph[8][2], pl[8][2];
            prep_scores<true, false>(pr, c, warp, lane, lanes + COL_KK, lanes + COL_QK, p.scale, ph, pl);
            prep_diag(pr, warp, lane);
            if (named_sync_or(1, 128, !ok || misc[1])) {
                abort = 1;
                misc[1] = 1;
                break;
            }
            Frag T[4];
            if (warp == 0) prep_inverse<0>(pr, lane, T);
            else if (warp == 1) prep_inverse<1>(pr, lane, T);
            else if (warp == 2) prep_inverse<2>(pr, lane, T);
            else prep_inverse<3>(pr, lane, T);
            // the chunk before has read T (its U) and P (its P U)
            if (c > 0) {
                ok = bar_wait_spin(bar_tf, (c - 1) & 1, spin);
                if (ok) ok = bar_wait_spin(bar_o, (c - 1) & 1, spin);
            }
            if (!ok) misc[1] = 1;
            unsigned char *th = sm + OFF_T, *tl = sm + OFF_T + kTile;
            if (warp == 0) store_t<0>(th, tl, lane, T);
            else if (warp == 1) store_t<1>(th, tl, lane, T);
            else if (warp == 2) store_t<2>(th, tl, lane, T);
            else store_t<3>(th, tl, lane, T);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < 2 * warp + 2) st_frag(sm + OFF_P, warp, lane, j, ph[j][0], ph[j][1]);
            fence_async_smem();
            bar_arrive(bar_t);
        }
    } else {
        // ------------------------------------------------------------------ chain group
        const int q = warp - 4, hi = lane >> 4, lr = lane & 15;
        const uint32_t tl = tbase + (static_cast<uint32_t>(32 * q) << 16);
        const int row = 16 * q + lr, colh = 32 * hi;  // this thread's row and first of 32 columns
        const bool iss = tid == 128, iss2 = tid == 128 + 32, iss_t = tid == tma_thread;
        unsigned char *tA = sm + OFF_A, *tB = sm + OFF_B, *tC = sm + OFF_CC;
        const uint32_t aA = smem_u32(tA), aB = smem_u32(tB), aC = smem_u32(tC);
        const uint32_t aTh = smem_u32(sm + OFF_T), aTl = aTh + kTile, aP = smem_u32(sm + OFF_P);
        const int64_t nstate = p.nslots * p.H * kN * kN;
        const int64_t sat = ((slot * p.H + h) * kN + row) * kN + colh;
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
        // 32 columns of this thread's row as two bf16 terms (and, with `one`, rounded once)
        auto store_split = [&](const P2 (&x)[16], unsigned char *th, unsigned char *tlo) {
#pragma unroll
            for (int v4 = 0; v4 < 4; ++v4) {
                uint32_t a[4], b[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) split2(x[4 * v4 + e], &a[e], &b[e]);
                const uint32_t at = swz(row, 2 * colh + 16 * v4);
                *reinterpret_cast<uint4 *>(th + at) = make_uint4(a[0], a[1], a[2], a[3]);
                *reinterpret_cast<uint4 *>(tlo + at) = make_uint4(b[0], b[1], b[2], b[3]);
            }
        };
        auto load_x = [&](uint32_t col, P2 (&x)[16]) {
            float v[32];
            tmem_ld32(tl + col, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = pk(v[2 * i], v[2 * i + 1]);
        };
        // group barrier with a vote: true if the CTA is to stop
        auto meet = [&](int ok) -> bool {
            fence_async_smem();
            fence_before();
            const bool stop = named_sync_or(2, 128, !ok || misc[1]);
            fence_after();
            return stop;
        };
        auto store_o = [&](int c) {  // output rows of chunk c from tensor memory
            P2 x[16];
            load_x(COL_O, x);
            const int64_t t = static_cast<int64_t>(c) * kC + row;
            if (t < len && in_bounds(p.status, first + t, 1, ntok)) {
                uint4 *dst = reinterpret_cast<uint4 *>(p.o + ((first + t) * p.H + h) * kN + colh);
#pragma unroll
                for (int v4 = 0; v4 < 4; ++v4)
                    dst[v4] = make_uint4(pack2(x[4 * v4]), pack2(x[4 * v4 + 1]), pack2(x[4 * v4 + 2]), pack2(x[4 * v4 + 3]));
            }
        };

        int ok = 1;
        uint32_t xph = 0;  // phase of bar_x
        for (int c = 0; c < nchunks && !abort; ++c) {
            const uint32_t aK = smem_u32(sm + OFF_K + kTile * (c % 3)), aQ = smem_u32(sm + OFF_Q + kTile * (c & 1));
            // ---- S hi, lo; K S
            store_split(S, tA, tB);
            if (iss && ok) ok = bar_wait_spin(bar_t, c & 1, spin);
            if (meet(ok)) {
                abort = 1;
                break;
            }
            if (iss) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma(tbase + COL_X, desc_k(aK + 32 * ks), desc_mn(aA + 2048 * ks), idesc(64, 0, 1), ks > 0);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma(tbase + COL_X, desc_k(aK + 32 * ks), desc_mn(aB + 2048 * ks), idesc(64, 0, 1), 1);
                mma_commit(bar_x);
            }
            bar_try(bar_t, c & 1);  // what the prep group wrote is visible to every thread
            const float gam = arr(pr, c, kGamma)[row], tail = arr(pr, c, kTail)[row], bet = arr(pr, c, kBeta)[row];
            const float gC = arr(pr, c, kGamma)[kC - 1];
            // ---- the output of the chunk before, under K S; then Q S takes its columns
            if (c > 0) {
                ok = bar_wait_spin(bar_o, (c - 1) & 1, spin);
                fence_after();
                store_o(c - 1);
            }
            if (meet(ok)) {
                abort = 1;
                break;
            }
            if (iss2) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma(tbase + COL_O, desc_k(aQ + 32 * ks), desc_mn(aA + 2048 * ks), idesc(64, 0, 1), ks > 0);
                mma_commit(bar_qs);
            }
            // ---- W = beta (v - gamma K S)
            P2 x[16];
            ok = bar_wait_spin(bar_x, xph, spin);
            xph ^= 1;
            if (ok) ok = bar_wait_spin(bar_v, c & 1, spin);
            fence_after();
            load_x(COL_X, x);
            {
                const P2 b2 = pk(bet, bet), bg = pk(-bet * gam, -bet * gam);
#pragma unroll
                for (int v4 = 0; v4 < 4; ++v4) {
                    const uint4 vv = *reinterpret_cast<const uint4 *>(sm + OFF_V + swz(row, 2 * colh + 16 * v4));
                    const uint32_t vw[4] = {vv.x, vv.y, vv.z, vv.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        x[4 * v4 + e] = fma2(bg, x[4 * v4 + e], mul2(b2, unpack2(vw[e])));
                }
                store_split(x, tC, tB);
            }
            if (meet(ok)) {
                abort = 1;
                break;
            }
            if (iss) {  // ---- U = T W
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma(tbase + COL_X, desc_k(aTh + 32 * ks), desc_mn(aC + 2048 * ks), idesc(64, 0, 1), ks > 0);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma(tbase + COL_X, desc_k(aTl + 32 * ks), desc_mn(aC + 2048 * ks), idesc(64, 0, 1), 1);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma(tbase + COL_X, desc_k(aTh + 32 * ks), desc_mn(aB + 2048 * ks), idesc(64, 0, 1), 1);
                mma_commit(bar_x);
                mma_commit(bar_tf);
            }
            if (iss_t && c + 1 < nchunks) load_tile(&map_v, OFF_V, h, c + 1, bar_v);
            // ---- scale diag(gamma) Q S, in place, under T W
            ok = bar_wait_spin(bar_qs, c & 1, spin);
            fence_after();
            {
                float v[32];
                tmem_ld32(tl + COL_O, v);
                const float sg = p.scale * gam;
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] *= sg;
                tmem_st32(tl + COL_O, v);
            }
            if (iss_t && c + 2 < nchunks) load_tile(&map_q, OFF_Q + kTile * (c & 1), hk, c + 2, bar_q0 + 8 * (c & 1));
            // ---- U, and diag(tail) U hi, lo
            if (ok) ok = bar_wait_spin(bar_x, xph, spin);
            xph ^= 1;
            fence_after();
            load_x(COL_X, x);
#pragma unroll
            for (int v4 = 0; v4 < 4; ++v4)
                *reinterpret_cast<uint4 *>(tC + swz(row, 2 * colh + 16 * v4)) =
                    make_uint4(pack2(x[4 * v4]), pack2(x[4 * v4 + 1]), pack2(x[4 * v4 + 2]), pack2(x[4 * v4 + 3]));
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = mul2(x[i], pk(tail, tail));
            store_split(x, tA, tB);
            if (meet(ok)) {
                abort = 1;
                break;
            }
            if (iss) {  // ---- K^T diag(tail) U
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma(tbase + COL_X, desc_mn(aK + 2048 * ks), desc_mn(aA + 2048 * ks), idesc(64, 1, 1), ks > 0);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma(tbase + COL_X, desc_mn(aK + 2048 * ks), desc_mn(aB + 2048 * ks), idesc(64, 1, 1), 1);
                mma_commit(bar_x);
            } else if (iss2) {  // ---- + P U
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    mma(tbase + COL_O, desc_k(aP + 32 * ks), desc_mn(aC + 2048 * ks), idesc(64, 0, 1), 1);
                mma_commit(bar_o);
            }
            ok = bar_wait_spin(bar_x, xph, spin);
            xph ^= 1;
            fence_after();
            load_x(COL_X, x);
#pragma unroll
            for (int i = 0; i < 16; ++i) S[i] = fma2(pk(gC, gC), S[i], x[i]);
            if (iss_t && ok && c + 3 < nchunks) load_tile(&map_k, OFF_K + kTile * (c % 3), hk, c + 3, bar_k0 + 8 * (c % 3));
        }
        if (!abort && nchunks > 0) {
            if (ok) ok = bar_wait_spin(bar_o, (nchunks - 1) & 1, spin);
            fence_after();
            if (meet(ok)) abort = 1;
            else store_o(nchunks - 1);
        }
        if (abort) misc[1] = 1;
        if (!abort && p.sT && slot >= 0 && in_bounds(p.status, sat, 32, nstate)) {
            float4 *dst = reinterpret_cast<float4 *>(p.sT + sat);
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i] = make_float4(lo(S[2 * i]), tc::hi(S[2 * i]), lo(S[2 * i + 1]), tc::hi(S[2 * i + 1]));
        }
    }

    // ---- drain after an abort, then release tensor memory
    fence_before();
    abort = __syncthreads_or(abort | misc[1]);
    fence_after();
    if (abort) {
        record_status(p.status, kStatusTimeout);
        if (tid == 0 || tid == 128 || tid == 128 + 32) mma_commit(bar_drain);  // the three issuers
        if (tid == 0) {
            bar_wait(bar_drain, 0, p.spin_limit);
            for (int i = 0; i < 6; ++i) {  // copies in flight: each ring barrier's last issued phase
                for (uint32_t ph = 0; ph < 2; ++ph) bar_wait(smem_u32(&bars[i]), ph, 200);
            }
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(kTmemCols));
}

}  // namespace

cudaError_t delta_chunked_launch(const DeltaArgs &a, cudaStream_t s)
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
                   static_cast<const __nv_bfloat16 *>(a.beta), a.scale, a.s0, static_cast<__nv_bfloat16 *>(a.o), a.sT,
                   a.status, g_chunked_inject_timeout ? 100u : 100000u, g_chunked_inject_timeout};
    delta_chunked_kernel<<<static_cast<unsigned>(a.nseq * a.H), kThreads, kSmemBytes, s>>>(mq, mk, mv, p);
    return cudaGetLastError();
}

}  // namespace wkv
