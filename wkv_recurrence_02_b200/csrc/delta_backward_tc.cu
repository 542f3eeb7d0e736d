// delta_backward_tc.cu -- gradients of the gated delta rule on B200 tensor cores, bf16 inputs.
//
// delta_tc.cuh has the chunk's forward algebra (T, P, U, gamma, tail).  Reversed, with dS the
// gradient of the state after the chunk and dO that of its outputs:
//   dU = P^T dO + diag(tail) K dS            dW = T^T dU (the whole gradient of u)
//   dS_prev = gamma_63 dS + Q^T diag(scale gamma) dO - K^T diag(beta gamma) dW
//   A1[t][i] = scale Gamma[t][i] dO_t.U_i (i <= t)      A2[t][i] = -beta_t Gamma[t][i] dW_t.U_i (i < t)
//   dQ = scale diag(gamma) dO S_prev^T + A1 K
//   dK = diag(tail) U dS^T - diag(beta gamma) dW S_prev^T + A1^T Q + (A2 + A2^T) K
//   dV = diag(beta) dW
//   dbeta_t = dW_t.V_t - x_t,  x_t = gamma_t K_t.(dW S_prev^T)_t + sum_{i<t} Gamma[t][i] (k_t.k_i) dW_t.U_i
//   dg_t = sum_{j>=t} e_j + sum_{i<t} tail_i K_i.(U dS^T)_i + gamma_63 <dS, S_prev>,
//   e_t = Q_t.dQ'_t - K_t.dK'_t - 2 beta_t x_t
// where dQ' and dK' leave out what no decay stands before: the diagonal of A1 and, in dK, diag(tail)
// U dS^T (it enters through the second sum).  Every pair of tokens i < j of the chunk enters e_j with
// one sign and e_i with the other, formed from the same rounded operands, and what is left out keeps
// fast decays (whose dg is far below the other gradients) out of the rounding of slow terms.
//
// Four kernels: T of all chunks (delta_prep.cu); the forward walk for S_prev and U of every chunk
// (delta_chunked.cu); delta_bwd_state_kernel, the walk back for dS and dW; delta_bwd_grad_kernel, all
// chunks at once, for the gradients.  S_prev, U, dS and dW pass between them in bf16, as images of
// their swizzled tiles.  ds0 is an fp32 result: between dS and dS_prev every operand is two bf16
// terms, as the state's are in the forward walk.
//
// Every mbarrier wait is bounded; on expiry the CTA records RWKV_ERR_TIMEOUT in the device
// status word, waits (bounded) for its own copies and MMAs, frees its tensor memory and returns.
#include "delta_tc.cuh"

#include <algorithm>

namespace wkv {
namespace {
using namespace dtc;

// ------------------------------------------------------------------------ the walk back
// As the forward walk (two CTAs per SM, the same groups and the same hand-overs):
//   chain group (warps 4-7)  dS -> K dS -> dU -> T^T dU = dW -> K^T diag(-beta gamma) dW -> dS
//   side group (warps 0-3)   what the chain adds but does not wait for: Q K^T, P, P^T dO, and
//                            Q^T diag(scale gamma) dO, where the chain's last product accumulates
// Measured: B8 T4096 H32 245 us; bound by the chain as the forward walk is (B8 T1024 H32: 70 us, tensor
// pipe 35 % active, DRAM 37 %, issue 31 %).
constexpr int kThreads = 256;
// 13 tiles: K, Q and dO of two chunks, T (hi, lo), a pair for P hi/lo and then diag(scale gamma) dO
// hi/lo, and the chain's A, B, C: dS hi/lo (A, B), dU hi/lo (B, C), diag(-beta gamma) dW hi/lo (A, B)
// and dW (C)
constexpr int OFF_K = 0, OFF_Q = 2 * kTile, OFF_DO = 4 * kTile, OFF_T = 6 * kTile, OFF_PG = 8 * kTile;
constexpr int OFF_A = 10 * kTile, OFF_B = 11 * kTile, OFF_CC = 12 * kTile;
constexpr int OFF_DEC = 13 * kTile;
constexpr int OFF_ARR = OFF_DEC + static_cast<int>(sizeof(Decays));
constexpr int OFF_BAR = OFF_ARR + 3 * static_cast<int>(sizeof(ChunkArrays));
constexpr int OFF_MISC = OFF_BAR + 26 * 8;
constexpr int kSmemBytes = OFF_MISC + 32 + 1024;  // + alignment slack
static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM do not fit");
// the chain's accumulators (128); Q K^T and then P^T dO; the sum that becomes dS_prev
constexpr uint32_t COL_X = 0, COL_R = 128, COL_Y = 192, kTmemCols = 256;

struct StateParams {
    int64_t B, T, Hk, H, nseq;
    const int32_t *offsets;
    const __nv_bfloat16 *g, *beta;
    const unsigned char *t;     // [chunks][H][kTBytes]
    int64_t nchunks;
    float scale;
    const float *dsT;
    float *ds0;
    unsigned char *ds, *dw;     // [chunks][H] tiles: dS after the chunk, dW
    int *status;
    uint32_t spin_limit;
    int inject_timeout;
};

__global__ void __launch_bounds__(kThreads, 2)
delta_bwd_state_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_do, const StateParams p)
{
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + OFF_BAR);
    volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(sm + OFF_MISC);  // TMEM base, abort
    // chunks are counted as they are walked: n = 0 is the last chunk of the sequence
    const uint32_t bar_k0 = smem_u32(&bars[0]);    // K, Q, dO there: + 8 * (n % 2)
    const uint32_t bar_q0 = smem_u32(&bars[2]);
    const uint32_t bar_g0 = smem_u32(&bars[4]);
    const uint32_t bar_t = smem_u32(&bars[6]);     // T there
    const uint32_t bar_a = smem_u32(&bars[7]);     // Q K^T done
    const uint32_t bar_x = smem_u32(&bars[8]);     // K dS, dW, the new dS done (three phases a chunk)
    const uint32_t bar_d0 = smem_u32(&bars[9]);    // P^T dO done
    const uint32_t bar_y = smem_u32(&bars[10]);    // Q^T diag(scale gamma) dO done
    const uint32_t bar_rr = smem_u32(&bars[11]);   // P^T dO read: its columns may take Q K^T
    const uint32_t bar_yr = smem_u32(&bars[12]);   // the new dS read: its columns may be written
    const uint32_t bar_as = smem_u32(&bars[17]);   // the copies of dS, of dW have read them
    const uint32_t bar_cs = smem_u32(&bars[18]);
    // decays written (for n = 0 also the tail rows zeroed): + 8 * (n % 3), since the side group may
    // pass two more chunks here before the chain waits for this one
    const uint32_t bar_s0 = smem_u32(&bars[19]);
    const uint32_t bar_drain = smem_u32(&bars[22]);
    const uint32_t bar_never = smem_u32(&bars[23]);

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform, see elect_one
    const int64_t blk = blockIdx.x, seq = blk / p.H, h = blk % p.H, hk = h / (p.H / p.Hk);
    int64_t first_, len_;
    sequence_span(p.offsets, seq, p.T, &first_, &len_);
    const int first = static_cast<int>(first_), len = static_cast<int>(len_);  // fewer than 2^31 tokens in all
    const int nchunks = (len + kC - 1) / kC;
    const int64_t chunk0 = first_chunk(p.offsets != nullptr, seq, first, p.T);
    const int row_b = p.offsets ? 0 : static_cast<int>(seq), row_t = p.offsets ? first : 0;
    const uint32_t spin = p.spin_limit;
    const int64_t ntok = p.B * p.T;

    if (tid == 0) {
        for (int i = 0; i < 24; ++i)
            bar_init(smem_u32(&bars[i]), i == 11 || i == 12 ? 128 : i == 22 ? 2 : i >= 19 && i < 22 ? 64 : 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        misc[1] = 0;
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(const_cast<uint32_t *>(misc))),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tbase = misc[0];

    auto load_tile = [&](const CUtensorMap *map, uint32_t off, int64_t head, int n, uint32_t bar) {
        const int c = nchunks - 1 - n;
        if (!tma_coord_ok(p.status, 0, 2, kN, row_t + static_cast<int64_t>(c) * kC, p.T)) return;
        bar_expect_tx(bar, kTile);
        tma_load_4d(smem_u32(sm + off), map, 0, static_cast<int>(head), row_t + c * kC, row_b, bar);
    };
    auto load_tiles = [&](int n) {  // K, Q, dO: one thread
        load_tile(&map_k, OFF_K + kTile * (n & 1), hk, n, bar_k0 + 8 * (n & 1));
        load_tile(&map_q, OFF_Q + kTile * (n & 1), hk, n, bar_q0 + 8 * (n & 1));
        load_tile(&map_do, OFF_DO + kTile * (n & 1), h, n, bar_g0 + 8 * (n & 1));
    };
    auto load_t = [&](int n) {  // one thread
        const int64_t id = chunk0 + nchunks - 1 - n;
        if (!in_bounds(p.status, id, 1, p.nchunks)) return;
        bar_expect_tx(bar_t, kTBytes);
        bulk_load(smem_u32(sm + OFF_T), p.t + (id * p.H + h) * kTBytes, kTBytes, bar_t);
    };
    if (warp == 7) {
        for (int n = 0; n < 2 && n < nchunks; ++n) {
            if (elect_one()) {
                load_tiles(n);
                if (n == 0) load_t(0);
            }
            __syncwarp();
        }
    }
    // Drain after a wait that ran out, then release tensor memory.
    auto leave = [&] {
        fence_before();
        const int abort = __syncthreads_or(misc[1] != 0);
        fence_after();
        if (abort) {
            record_status(p.status, kStatusTimeout);
            if ((warp == 0 || warp == 4) && elect_one()) mma_commit(bar_drain);  // the two issuers
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
        // This kernel runs beside the walk launched before it (see the launch); what follows needs both.
        asm volatile("griddepcontrol.wait;" ::: "memory");
    };
    if (p.inject_timeout) {
        if (tid == 0 && !bar_wait(bar_never, 0, p.spin_limit)) misc[1] = 1;
        leave();
        return;
    }
    int ok = 1;
    if (warp < 4) {
        // ------------------------------------------------------------------ side group
        const int w = warp;
        Decays &dec = *reinterpret_cast<Decays *>(sm + OFF_DEC);
        ChunkArrays *arrays = reinterpret_cast<ChunkArrays *>(sm + OFF_ARR);
        const int st = tid - 64;
        uint16_t g_next = 0, b_next = 0;
        auto fetch = [&](int n) {  // g and beta of a token, a chunk ahead
            const int t = (nchunks - 1 - n) * kC + st;
            g_next = b_next = 0;
            if (t >= len || !in_bounds(p.status, first + t, 1, ntok)) return;
            const int64_t at = static_cast<int64_t>(first + t) * p.H + h;
            g_next = reinterpret_cast<const uint16_t *>(p.g)[at];
            b_next = reinterpret_cast<const uint16_t *>(p.beta)[at];
        };
        auto scan = [&](int n) {
            const float gv = widen(g_next), bv = widen(b_next);
            if (n + 1 < nchunks) fetch(n + 1);
            scan_decays<3>(dec, arrays[n % 3], st, gv, bv);
            bar_arrive(bar_s0 + 8 * (n % 3));
        };
        auto products = [&](int n) -> int {  // Q K^T (warp 0)
            unsigned char *kt = sm + OFF_K + kTile * (n & 1), *qt = sm + OFF_Q + kTile * (n & 1), *gt = sm + OFF_DO + kTile * (n & 1);
            const uint32_t ph = (n >> 1) & 1;
            const bool there = bar_wait(bar_k0 + 8 * (n & 1), ph, spin) && bar_wait(bar_q0 + 8 * (n & 1), ph, spin) &&
                               bar_wait(bar_g0 + 8 * (n & 1), ph, spin) &&
                               (n == 0 || bar_wait(bar_rr, (n - 1) & 1, spin));
            if (!__all_sync(0xffffffffu, there)) return 0;
            const int tv = len - (nchunks - 1 - n) * kC;
            if (tv < kC) {
                zero_rows(kt, tv, lane, 32);
                zero_rows(qt, tv, lane, 32);
                zero_rows(gt, tv, lane, 32);
                fence_async_smem();
                __syncwarp();
            }
            fence_after();
            const uint64_t dk = desc_k(smem_u32(kt)), dq = desc_k(smem_u32(qt));
            if (elect_one()) {
                mma_tile<kStepK, kStepK, false>(tbase + COL_R, dq, dk, idesc(64, 0, 0));
                mma_commit(bar_a);
            }
            __syncwarp();
            return 1;
        };
        const uint32_t qk = tbase + (static_cast<uint32_t>(32 * w) << 16) + COL_R;
        const int row = 16 * w + (lane & 15), col = 32 * (lane >> 4);
        unsigned char *ph_t = sm + OFF_PG, *pl_t = sm + OFF_PG + kTile;
        if (nchunks > 0) {
            if (w == 0) ok = products(0);
            group_sync<1, 128>();
            if (w >= 2) {
                fetch(0);
                scan(0);
            }
        }
        for (int n = 0; n < nchunks; ++n) {
            group_sync<1, 128>();  // the chunk's decays are there
            if (ok) ok = bar_wait(bar_a, n & 1, spin);
            fence_after();
            uint32_t ph[4][4], pl[4][4];
            form_p<true>(dec, w, lane, qk, p.scale, ph, pl);
            fence_before();
            if (misc[1]) ok = 0;
            group_sync<1, 128>();
            if (w >= 2 && n + 1 < nchunks) scan(n + 1);
            // ---- P^T dO; the pair of tiles was last read by the product that bar_y stands for
            if (ok && n > 0) ok = bar_wait(bar_y, (n - 1) & 1, spin);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                st_block(ph_t, w, j, lane, ph[j]);
                st_block(pl_t, w, j, lane, pl[j]);
            }
            fence_async_smem();
            group_sync<1, 128>();
            const unsigned char *gt = sm + OFF_DO + kTile * (n & 1);
            if (w == 0) {
                fence_after();
                const uint64_t dp = desc_mn(smem_u32(ph_t)), dl = desc_mn(smem_u32(pl_t)), dg = desc_mn(smem_u32(gt));
                if (elect_one()) {
                    mma_tile<kStepMn, kStepMn, false>(tbase + COL_R, dp, dg, idesc(64, 1, 1));
                    mma_tile<kStepMn, kStepMn, true>(tbase + COL_R, dl, dg, idesc(64, 1, 1));
                    mma_commit(bar_d0);
                }
                __syncwarp();
            }
            // ---- diag(scale gamma) dO hi, lo, then its product with Q^T
            const float sg = p.scale * arrays[n % 3].gamma[row];
            if (ok) ok = bar_wait(bar_g0 + 8 * (n & 1), (n >> 1) & 1, spin);
            uint32_t xh[4][4], xl[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 y = *reinterpret_cast<const uint4 *>(gt + swz(row, 2 * col + 16 * i));
                const uint32_t yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) split2(mul2(unpack2(yw[e]), pk(sg, sg)), &xh[i][e], &xl[i][e]);
            }
            if (ok) ok = bar_wait(bar_d0, n & 1, spin);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t at = swz(row, 2 * col + 16 * i);
                *reinterpret_cast<uint4 *>(ph_t + at) = make_uint4(xh[i][0], xh[i][1], xh[i][2], xh[i][3]);
                *reinterpret_cast<uint4 *>(pl_t + at) = make_uint4(xl[i][0], xl[i][1], xl[i][2], xl[i][3]);
            }
            fence_async_smem();
            group_sync<1, 128>();
            if (w == 0) {
                if (n > 0 && ok) ok = __all_sync(0xffffffffu, bar_wait(bar_yr, (n - 1) & 1, spin));
                fence_after();
                const uint64_t dq = desc_mn(smem_u32(sm + OFF_Q + kTile * (n & 1)));
                const uint64_t dh = desc_mn(smem_u32(ph_t)), dl = desc_mn(smem_u32(pl_t));
                if (elect_one()) {
                    mma_tile<kStepMn, kStepMn, false>(tbase + COL_Y, dq, dh, idesc(64, 1, 1));
                    mma_tile<kStepMn, kStepMn, true>(tbase + COL_Y, dq, dl, idesc(64, 1, 1));
                    mma_commit(bar_y);
                }
                __syncwarp();
                if (n + 1 < nchunks && !products(n + 1)) ok = 0;
            }
            if (!ok) misc[1] = 1;
        }
    } else {
        // ------------------------------------------------------------------ chain group
        const int q = warp & 3;
        const uint32_t tl = tbase + (static_cast<uint32_t>(32 * q) << 16);
        const int row = 16 * q + (lane & 15), col = 32 * (lane >> 4);  // its row, first of 32 columns
        unsigned char *tA = sm + OFF_A, *tB = sm + OFF_B, *tC = sm + OFF_CC;
        const int64_t sat = ((seq * p.H + h) * kN + row) * kN + col, nstate = p.nseq * p.H * kN * kN;
        P2 S[16];
        if (p.dsT && in_bounds(p.status, sat, 32, nstate)) {
            const float4 *src = reinterpret_cast<const float4 *>(p.dsT + sat);
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
        const uint32_t at0 = swz(row, 2 * col);  // this thread's 32 columns of a tile: i-th 16 bytes
        auto at = [&](int i) { return at0 ^ static_cast<uint32_t>(16 * i); };
        auto store_split = [&](const P2 *x, int half, unsigned char *th, unsigned char *tlo) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t a[4], b[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) split2(x[4 * i + e], &a[e], &b[e]);
                *reinterpret_cast<uint4 *>(th + at(2 * half + i)) = make_uint4(a[0], a[1], a[2], a[3]);
                *reinterpret_cast<uint4 *>(tlo + at(2 * half + i)) = make_uint4(b[0], b[1], b[2], b[3]);
            }
        };
        const uint64_t dA = desc_mn(smem_u32(tA)), dB = desc_mn(smem_u32(tB));
        const uint64_t dTh = desc_tt(smem_u32(sm + OFF_T)), dTl = desc_tt(smem_u32(sm + OFF_T + kTile));
        auto meet = [&]() {  // what was written is ready for the products issued next
            fence_async_smem();
            fence_before();
            group_sync<2, 128>();
            fence_after();
        };
        uint32_t xph = 0;  // phase of bar_x
        for (int n = 0; n < nchunks; ++n) {
            const uint32_t aK = smem_u32(sm + OFF_K + kTile * (n & 1));
            const int64_t id = chunk0 + nchunks - 1 - n, tile = (id * p.H + h) * kTile;
            // ---- dS hi, lo; K dS
            if (misc[1]) ok = 0;
            store_split(S, 0, tA, tB);
            store_split(S + 8, 1, tA, tB);
            if (n == 0 && ok) ok = bar_wait(bar_s0, 0, spin);  // tail rows are zeroed
            meet();
            if (warp == 4) {
                const uint64_t dK = desc_k(aK);
                if (ok) ok = bar_wait_spin(bar_k0 + 8 * (n & 1), (n >> 1) & 1, spin * 64u);
                __syncwarp();
                if (elect_one()) {
                    mma_tile<kStepK, kStepMn, false>(tbase + COL_X, dK, dA, idesc(128, 0, 1));
                    mma_commit(bar_x);
                }
            } else if (warp == 5 && lane == 0) {
                if (in_bounds(p.status, id, 1, p.nchunks)) bulk_store(p.ds + tile, smem_u32(tA), kTile);
                bulk_commit();
                bulk_wait_read<0>();
                bar_arrive(bar_as);
            } else if (warp == 7 && n > 0 && n + 1 < nchunks) {  // dS is there: the chunk before is done with its tiles
                if (elect_one() && ok) load_tiles(n + 1);
            }
            __syncwarp();
            // ---- dU = P^T dO + diag(tail) K dS
            if (ok) ok = bar_wait(bar_s0 + 8 * (n % 3), (n / 3) & 1, spin);
            const ChunkArrays &arr = reinterpret_cast<const ChunkArrays *>(sm + OFF_ARR)[n % 3];
            const float bg = -arr.beta[row] * arr.gamma[row], tail = arr.tail[row], gC = arr.gamma[kC - 1];
            if (ok) ok = bar_wait(bar_d0, n & 1, spin);
            if (ok && n > 0) ok = bar_wait(bar_cs, (n - 1) & 1, spin);
            if (ok) ok = bar_wait(bar_t, n & 1, spin);
            if (ok) ok = bar_wait(bar_x, xph, spin);
            xph ^= 1;
            fence_after();
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                P2 x[8];
                tmem_ld_sum16(tl + COL_X + 16 * half, x);
                float d0[16];
                tmem_ld16(tl + COL_R + 16 * half, d0);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = fma2(pk(tail, tail), x[i], pk(d0[2 * i], d0[2 * i + 1]));
                store_split(x, half, tB, tC);
            }
            meet();
            bar_arrive(bar_rr);
            if (warp == 4) {  // ---- dW = T^T dU
                if (elect_one()) {
                    mma_tile<kStepTMn, kStepMn, false>(tbase + COL_X, dTh, dB, idesc(128, 1, 1));
                    mma_tile<kStepTMn, kStepMn, true>(tbase + COL_X, dTl, dB, idesc(64, 1, 1));
                    mma_commit(bar_x);
                }
                __syncwarp();
            }
            // ---- dW, and diag(-beta gamma) dW hi, lo
            if (ok) ok = bar_wait(bar_as, n & 1, spin);
            if (ok) ok = bar_wait(bar_y, n & 1, spin);
            if (ok) ok = bar_wait(bar_x, xph, spin);
            xph ^= 1;
            fence_after();
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                P2 x[8];
                tmem_ld_sum16(tl + COL_X + 16 * half, x);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    *reinterpret_cast<uint4 *>(tC + at(2 * half + i)) =
                        make_uint4(pack2(x[4 * i]), pack2(x[4 * i + 1]), pack2(x[4 * i + 2]), pack2(x[4 * i + 3]));
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = mul2(x[i], pk(bg, bg));
                store_split(x, half, tA, tB);
            }
            meet();
            if (warp == 4) {  // ---- + K^T diag(-beta gamma) dW
                const uint64_t dKt = desc_mn(aK);
                if (elect_one()) {
                    mma_tile<kStepMn, kStepMn, true>(tbase + COL_Y, dKt, dA, idesc(64, 1, 1));
                    mma_tile<kStepMn, kStepMn, true>(tbase + COL_Y, dKt, dB, idesc(64, 1, 1));
                    mma_commit(bar_x);
                }
            } else if (warp == 5 && lane == 0) {
                if (in_bounds(p.status, id, 1, p.nchunks)) bulk_store(p.dw + tile, smem_u32(tC), kTile);
                bulk_commit();
                bulk_wait_read<0>();
                bar_arrive(bar_cs);
            } else if (warp == 7 && n + 1 < nchunks) {
                if (elect_one() && ok) load_t(n + 1);  // dW is there: T has been read
            }
            __syncwarp();
            // ---- dS
            if (ok) ok = bar_wait(bar_x, xph, spin);
            xph ^= 1;
            fence_after();
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float y[16];
                tmem_ld16(tl + COL_Y + 16 * half, y);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    S[8 * half + i] = fma2(pk(gC, gC), S[8 * half + i], pk(y[2 * i], y[2 * i + 1]));
            }
            fence_before();
            bar_arrive(bar_yr);
            if (!ok) misc[1] = 1;  // and its waits pass from here on, in this thread and soon in all
        }
        if (warp == 5 && lane == 0) bulk_wait_all();
        if (ok && p.ds0 && in_bounds(p.status, sat, 32, nstate)) {
            float4 *dst = reinterpret_cast<float4 *>(p.ds0 + sat);
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i] = make_float4(lo(S[2 * i]), hi(S[2 * i]), lo(S[2 * i + 1]), hi(S[2 * i + 1]));
        }
    }
    if (!ok) misc[1] = 1;
    leave();
}

// ----------------------------------------------------------------------- gradients of a chunk
// One block of eight warps per (chunk, value head), two per SM.  Warp (q, half) holds rows
// 16 q .. 16 q + 15 and columns 32 half .. of every 64 x 64 result, thread (row, hl) columns 8 hl ..
// 8 hl + 7 of both 16-wide blocks there: whether a block lies left of, on or right of the diagonal is
// the same for the whole warp.  Two rounds of products:
//   dO U^T, dW U^T, K K^T, Q K^T                     -> A1, A2, x
//   diag(scale gamma) dO S_prev^T + A1 K, dW S_prev^T, (A2 + A2^T) K + A1^T Q, U dS^T -> the gradients
// A1 and A2 enter the second round rounded to bf16.  For dg, where the terms of A1 and of A2 can
// cancel (keys near one another), what the rounding left is added back as its row and column sums.
//
// The blocks stay and take chunks in turn.  Thirteen tiles: Q, K and dW twice (the next chunk's load
// while this one's are still read), V, dO (then diag(scale gamma) dO in its place), U, S_prev, dS, A1,
// A2.  The loads of the next chunk start as soon as the second round of products is done.  dQ, dK and
// dV of a whole chunk leave as tiles (from where A1, A2 and dW were): a row of a thread's own is 16
// bytes, and stores of those were the kernel's largest use of the shared-memory pipe.
//
// Measured: B8 T4096 H32 332 us for 1.6 GB (448 with a block a chunk, direct stores and no load ahead);
// B8 T1024 H32 91 us, DRAM 46 %, issue 42 %, shared-memory pipe 39 %: two chunks an SM, each waiting
// for its own loads, products and barriers in turn.
constexpr int kGThreads = 256;
constexpr int GO_Q = 0, GO_K = 2 * kTile, GO_DW = 4 * kTile;  // + kTile * (item % 2)
constexpr int GO_V = 6 * kTile, GO_DO = 7 * kTile, GO_U = 8 * kTile, GO_S = 9 * kTile, GO_DS = 10 * kTile;
constexpr int GO_A1 = 11 * kTile, GO_A2 = 12 * kTile, GO_DEC = 13 * kTile;
constexpr int GO_ARR = GO_DEC + static_cast<int>(sizeof(Decays));
constexpr int GO_RED = GO_ARR + static_cast<int>(sizeof(ChunkArrays));  // [4 sums][2 halves][64], [8] warps' sums, [4]
constexpr int GO_COL = GO_RED + 4 * 2 * 256 + 64;   // [4 block rows][64] column sums
constexpr int GO_DIAG = GO_COL + 4 * 256;           // [64] diagonal of A1
constexpr int GO_BAR = GO_DIAG + 256;
constexpr int kGSmemBytes = GO_BAR + 32 + 1024;
static_assert(2 * (kGSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM do not fit");
constexpr uint32_t GC_DOU = 0, GC_DWU = 64, GC_QK = 128, GC_KK = 192;           // first round
constexpr uint32_t GC_DQ = 0, GC_DK = 64, GC_DWS = 128, GC_UDS = 192;           // second

struct GradParams {
    int64_t B, T, Hk, H, nseq;
    const int32_t *offsets;
    const __nv_bfloat16 *g, *beta;
    float scale;
    const unsigned char *states, *us, *ds, *dw;  // [chunks][H] tiles
    int64_t nchunks;
    __nv_bfloat16 *dq, *dk, *dv, *dg, *dbeta;
    float *dq_h, *dk_h;  // [B,T,H,64] shares of the value heads, or null
    int *status;
    uint32_t spin_limit;
    int inject_timeout;
};

// A thread's 16 columns, as pairs: [4 b + i] of block b (b = 0, 1).
struct Row {
    P2 x[8];
};
struct Raw {
    uint32_t r[16];
};
__device__ __forceinline__ void tmem_ld_blocks(uint32_t taddr, Raw &v)  // no wait
{
#pragma unroll
    for (int b = 0; b < 2; ++b)
        asm volatile("tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8], 8;"
                     : "=r"(v.r[8 * b]), "=r"(v.r[8 * b + 1]), "=r"(v.r[8 * b + 2]), "=r"(v.r[8 * b + 3]),
                       "=r"(v.r[8 * b + 4]), "=r"(v.r[8 * b + 5]), "=r"(v.r[8 * b + 6]), "=r"(v.r[8 * b + 7])
                     : "r"(taddr + 16 * b));
}
__device__ __forceinline__ Row row_of(Raw &v)  // after the wait
{
    Row y;
#pragma unroll
    for (int i = 0; i < 16; ++i) after_wait(v.r[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i) y.x[i] = pk(__uint_as_float(v.r[2 * i]), __uint_as_float(v.r[2 * i + 1]));
    return y;
}
__device__ __forceinline__ void unpack_row(const uint4 (&y)[2], Row &v)
{
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        v.x[4 * b] = unpack2(y[b].x);
        v.x[4 * b + 1] = unpack2(y[b].y);
        v.x[4 * b + 2] = unpack2(y[b].z);
        v.x[4 * b + 3] = unpack2(y[b].w);
    }
}
__device__ __forceinline__ uint4 pack_block(const Row &v, int b)
{
    return make_uint4(pack2(v.x[4 * b]), pack2(v.x[4 * b + 1]), pack2(v.x[4 * b + 2]), pack2(v.x[4 * b + 3]));
}
__device__ __forceinline__ float sum2(P2 x) { return lo(x) + hi(x); }
__device__ __forceinline__ float dot(const Row &a, const Row &b)
{
    P2 s = mul2(a.x[0], b.x[0]), r = mul2(a.x[1], b.x[1]);
#pragma unroll
    for (int i = 2; i < 8; i += 2) {
        s = fma2(a.x[i], b.x[i], s);
        r = fma2(a.x[i + 1], b.x[i + 1], r);
    }
    return sum2(add2(s, r));
}
// 8 columns (4 pairs) summed over the 16 rows of a half-warp: the total of column (lane >> 1) & 7
__device__ __forceinline__ float column_sum(const P2 (&d)[4], int lane)
{
    const bool b8 = lane & 8, b4 = lane & 4, b2 = lane & 2;
    P2 y[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) y[i] = add2(b8 ? d[2 + i] : d[i], shfl_xor2(b8 ? d[i] : d[2 + i], 8));
    const P2 z = add2(b4 ? y[1] : y[0], shfl_xor2(b4 ? y[0] : y[1], 4));
    float s = (b2 ? hi(z) : lo(z)) + __shfl_xor_sync(0xffffffffu, b2 ? lo(z) : hi(z), 2);
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    return s;
}
__device__ __forceinline__ void st_blocks(__nv_bfloat16 *p, const Row &v)
{
    *reinterpret_cast<uint4 *>(p) = pack_block(v, 0);
    *reinterpret_cast<uint4 *>(p + 16) = pack_block(v, 1);
}
__device__ __forceinline__ void st_blocks(float *p, const Row &v)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4 *>(p + 16 * (i >> 1) + 4 * (i & 1)) =
            make_float4(lo(v.x[2 * i]), hi(v.x[2 * i]), lo(v.x[2 * i + 1]), hi(v.x[2 * i + 1]));
}

// One (chunk, value head).
struct Item {
    int64_t h, hk, t0;
    int tv;          // tokens of the chunk, 0: there is no such chunk
    int row_b, row_t;  // tensor-map coordinates of the first token
};
__device__ __forceinline__ Item item_at(const GradParams &p, uint32_t n)
{
    const uint32_t heads = static_cast<uint32_t>(p.H), id = n / heads, h = n % heads;
    int64_t seq, first, len;
    const int c = chunk_of(p.offsets, p.nseq, p.T, id, &seq, &first, &len);
    Item x;
    x.h = h;
    x.hk = h / (heads / static_cast<uint32_t>(p.Hk));
    x.t0 = first + static_cast<int64_t>(c) * kC;
    const int64_t left = len - (x.t0 - first);
    x.tv = c < 0 ? 0 : static_cast<int>(left < kC ? left : kC);
    x.row_b = p.offsets ? 0 : static_cast<int>(seq);
    x.row_t = static_cast<int>(p.offsets ? x.t0 : x.t0 - first);
    return x;
}

__global__ void __launch_bounds__(kGThreads, 2)
delta_bwd_grad_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_do,
                      const __grid_constant__ CUtensorMap map_dq, const __grid_constant__ CUtensorMap map_dk,
                      const __grid_constant__ CUtensorMap map_dv, const GradParams p)
{
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int64_t ntok = p.B * p.T;
    const uint32_t total = static_cast<uint32_t>(p.nchunks * p.H);
    const uint32_t bar0 = smem_u32(sm + GO_BAR), bar1 = bar0 + 8, bar2 = bar0 + 16;  // tiles there; rounds done
    volatile uint32_t *tm = reinterpret_cast<volatile uint32_t *>(sm + GO_BAR + 24);
    Decays &dec = *reinterpret_cast<Decays *>(sm + GO_DEC);
    ChunkArrays &arr = *reinterpret_cast<ChunkArrays *>(sm + GO_ARR);
    float *red = reinterpret_cast<float *>(sm + GO_RED), *diag = reinterpret_cast<float *>(sm + GO_DIAG);
    float *cols = reinterpret_cast<float *>(sm + GO_COL);

    // the block's next item that is a chunk (total: none left)
    auto next_item = [&](uint32_t n, Item *x) -> uint32_t {
        for (; n < total; n += gridDim.x) {
            *x = item_at(p, n);
            if (x->tv > 0) break;
        }
        return n < total ? n : total;
    };
    auto load = [&](uint32_t n, const Item &x, int buf) {  // one thread
        const uint32_t id = n / static_cast<uint32_t>(p.H);
        const int64_t tile = static_cast<int64_t>(n) * kTile;  // n = id * H + h
        if (!tma_coord_ok(p.status, 0, 2, kN, x.row_t, p.T) || !in_bounds(p.status, id, 1, p.nchunks)) return;
        const int h = static_cast<int>(x.h), hk = static_cast<int>(x.hk);
        bar_expect_tx(bar0, 8 * kTile);
        bulk_load(smem_u32(sm + GO_U), p.us + tile, kTile, bar0);
        bulk_load(smem_u32(sm + GO_DW + kTile * buf), p.dw + tile, kTile, bar0);
        tma_load_4d(smem_u32(sm + GO_DO), &map_do, 0, h, x.row_t, x.row_b, bar0);
        tma_load_4d(smem_u32(sm + GO_Q + kTile * buf), &map_q, 0, hk, x.row_t, x.row_b, bar0);
        tma_load_4d(smem_u32(sm + GO_K + kTile * buf), &map_k, 0, hk, x.row_t, x.row_b, bar0);
        tma_load_4d(smem_u32(sm + GO_V), &map_v, 0, h, x.row_t, x.row_b, bar0);
        bulk_load(smem_u32(sm + GO_S), p.states + tile, kTile, bar0);
        bulk_load(smem_u32(sm + GO_DS), p.ds + tile, kTile, bar0);
    };
    const int st = tid - 32;  // warps 1 and 2: the token whose decay this thread prepares
    uint16_t g_next = 0, b_next = 0;
    auto fetch = [&](const Item &x) {
        g_next = b_next = 0;
        if (st < 0 || st >= 64 || st >= x.tv || !in_bounds(p.status, x.t0 + st, 1, ntok)) return;
        const int64_t at = (x.t0 + st) * p.H + x.h;
        g_next = reinterpret_cast<const uint16_t *>(p.g)[at];
        b_next = reinterpret_cast<const uint16_t *>(p.beta)[at];
    };
    Item cur, nxt;
    uint32_t n = next_item(blockIdx.x, &cur);
    if (n >= total) return;
    if (warp == 0) {
        if (lane == 0) {
            for (int i = 0; i < 3; ++i) bar_init(bar0 + 8 * i, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            load(n, cur, 0);
        }
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(const_cast<uint32_t *>(tm))),
                     "r"(256u));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fetch(cur);
    fence_before();
    __syncthreads();
    fence_after();
    const int q = warp & 3, half = warp >> 2, row = 16 * q + (lane & 15), col = 32 * half + 8 * (lane >> 4);
    const uint32_t sw[2] = {swz(row, 2 * col), swz(row, 2 * col + 32)};  // this thread's places in a tile
    const uint32_t tbase = tm[0], tl = tbase + (static_cast<uint32_t>(32 * q) << 16) + 32 * half;
    auto tile_row = [&](int tile, Row &x) {
        const uint4 y[2] = {*reinterpret_cast<const uint4 *>(sm + tile + sw[0]), *reinterpret_cast<const uint4 *>(sm + tile + sw[1])};
        unpack_row(y, x);
    };
    auto put_row = [&](int tile, const Row &x) {
        *reinterpret_cast<uint4 *>(sm + tile + sw[0]) = pack_block(x, 0);
        *reinterpret_cast<uint4 *>(sm + tile + sw[1]) = pack_block(x, 1);
    };

    auto leave = [&](bool out) {  // out: a wait of this thread's ran out
        if (warp == 7 && elect_one()) bulk_wait_all();
        fence_before();
        const int bad = __syncthreads_or(out);
        fence_after();
        if (bad && tid == 0) {
            record_status(p.status, kStatusTimeout);
            for (int i = 0; i < 3; ++i)  // what is in flight
                for (uint32_t ph = 0; ph < 2; ++ph) bar_wait(bar0 + 8 * i, ph, 200);
        }
        __syncthreads();
        if (warp == 0)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(256u));
    };
    if (p.inject_timeout) {  // there are no products yet whose end bar1 could tell
        leave(tid == 0 && !bar_wait(bar1, 0, p.spin_limit));
        return;
    }
    int ok = 1;
    for (int it = 0; n < total; ++it, cur = nxt) {
        const int buf = it & 1, ph = it & 1, tQ = GO_Q + kTile * buf, tK = GO_K + kTile * buf, tW = GO_DW + kTile * buf;
        const uint32_t aQ = smem_u32(sm + tQ), aK = smem_u32(sm + tK), aW = smem_u32(sm + tW), aO = smem_u32(sm + GO_DO);
        const uint32_t aU = smem_u32(sm + GO_U), aS = smem_u32(sm + GO_S), aD = smem_u32(sm + GO_DS);
        const uint32_t a1 = smem_u32(sm + GO_A1), a2 = smem_u32(sm + GO_A2);
        const int64_t token = cur.t0 + row, at = (token * p.H + cur.h) * kN + col;
        const bool whole = cur.tv == kC, valid = row < cur.tv && in_bounds(p.status, token, 1, ntok);
        ok = bar_wait(bar0, ph, p.spin_limit);
        if (!whole) {
            zero_rows(sm + tQ, cur.tv, tid, kGThreads);
            zero_rows(sm + tK, cur.tv, tid, kGThreads);
            zero_rows(sm + GO_V, cur.tv, tid, kGThreads);
            zero_rows(sm + GO_DO, cur.tv, tid, kGThreads);
            fence_async_smem();
        }
        if (__syncthreads_or(!ok)) {
            ok = 0;
            break;
        }
        if (warp == 0) {
            const uint64_t dO = desc_k(aO), dU = desc_k(aU), dW = desc_k(aW), dK = desc_k(aK), dQ = desc_k(aQ);
            if (elect_one()) {
                mma_tile<kStepK, kStepK, false>(tbase + GC_DOU, dO, dU, idesc(64, 0, 0));
                mma_tile<kStepK, kStepK, false>(tbase + GC_DWU, dW, dU, idesc(64, 0, 0));
                mma_tile<kStepK, kStepK, false>(tbase + GC_QK, dQ, dK, idesc(64, 0, 0));
                mma_tile<kStepK, kStepK, false>(tbase + GC_KK, dK, dK, idesc(64, 0, 0));
                mma_commit(bar1);
            }
            __syncwarp();
        } else if (warp < 3) {
            scan_decays<1>(dec, arr, st, widen(g_next), widen(b_next));
        }
        const uint32_t n2 = next_item(n + gridDim.x, &nxt);
        if (n2 < total) fetch(nxt);
        // ---- the row's dW.V; <dS, S_prev>
        float dots, dwv;
        {
            Row x, y;
            tile_row(tW, x);
            tile_row(GO_V, y);
            dwv = dot(x, y);
            tile_row(GO_S, x);
            tile_row(GO_DS, y);
            dots = dot(x, y);
        }
        __syncthreads();
        const float beta = arr.beta[row], gam = arr.gamma[row], tail = arr.tail[row];
        Row gm;  // Gamma, 1 on the diagonal
        const float n0 = dec.pn[row], f0 = dec.pf[row];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int blk = 2 * half + b;
            if (blk < q) {
                float mn = 0.f, mf = 0.f;
#pragma unroll
                for (int m = 1; m < 3; ++m)
                    if (m > blk && m < q) mn += dec.bs[m], mf += dec.bs[4 + m];
                const float rf = ex2_approx((n0 + mn) + (f0 + mf));
#pragma unroll
                for (int i = 0; i < 4; ++i) gm.x[4 * b + i] = mul2(ld_p2(dec.cf + col + 16 * b + 2 * i), pk(rf, rf));
            } else if (blk == q) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int cc = col + 16 * b + 2 * i;
                    const P2 cn = ld_p2(dec.pn + cc), cff = ld_p2(dec.pf + cc);
                    gm.x[4 * b + i] = pk(cc <= row ? ex2_approx((n0 - lo(cn)) + (f0 - lo(cff))) : 0.f,
                                         cc + 1 <= row ? ex2_approx((n0 - hi(cn)) + (f0 - hi(cff))) : 0.f);
                }
            }
        }
        {
            Row x;  // the first round's reading of dO is over once its results are there: see below
            ok = bar_wait(bar1, ph, p.spin_limit);
            fence_after();
            const float sg = p.scale * gam;
            tile_row(GO_DO, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) x.x[i] = mul2(x.x[i], pk(sg, sg));
            put_row(GO_DO, x);
        }
        // ---- A1, A2, sum Gamma (k k) (dW.U), and what rounding A1 and A2 leaves
        float xt = 0.f, rowd = 0.f;
        {
            Raw ro, rw, rq, rk;
            tmem_ld_blocks(tl + GC_DOU, ro);
            tmem_ld_blocks(tl + GC_DWU, rw);
            tmem_ld_blocks(tl + GC_QK, rq);
            tmem_ld_blocks(tl + GC_KK, rk);
            tmem_wait_ld();
            const Row o = row_of(ro), wu = row_of(rw), qk = row_of(rq), kk = row_of(rk);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int blk = 2 * half + b;
                uint32_t h1[4] = {}, h2[4] = {};
                if (blk <= q) {
                    P2 left[4], xs = pk(0.f, 0.f), rows = xs;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int k = 4 * b + i, cc = col + 16 * b + 2 * i;
                        P2 v1 = mul2(mul2(gm.x[k], pk(p.scale, p.scale)), o.x[k]), g = gm.x[k];
                        if (blk == q) {  // A1's diagonal is added to dQ and dK at the end
                            if (cc == row) diag[row] = lo(v1);
                            if (cc + 1 == row) diag[row] = hi(v1);
                            v1 = pk(cc < row ? lo(v1) : 0.f, cc + 1 < row ? hi(v1) : 0.f);
                            g = pk(cc < row ? lo(g) : 0.f, cc + 1 < row ? hi(g) : 0.f);
                        }
                        const P2 gw = mul2(g, wu.x[k]);
                        xs = fma2(gw, kk.x[k], xs);
                        const P2 v2 = mul2(gw, pk(-beta, -beta));
                        h1[i] = pack2(v1);
                        h2[i] = pack2(v2);
                        // x, taken twice, has A2's row sum unrounded already: its remainder counts the
                        // other way there
                        const P2 m1 = pk(-1.f, -1.f);
                        const P2 d1 = mul2(fma2(unpack2(h1[i]), m1, v1), qk.x[k]);
                        const P2 d2 = mul2(fma2(unpack2(h2[i]), m1, v2), kk.x[k]);
                        left[i] = add2(d1, d2);
                        rows = add2(rows, fma2(d2, m1, d1));
                    }
                    xt += sum2(xs);
                    rowd += sum2(rows);
                    const float s = column_sum(left, lane);
                    if ((lane & 1) == 0) cols[64 * q + col + 16 * b + ((lane >> 1) & 7)] = s;
                }
                *reinterpret_cast<uint4 *>(sm + GO_A1 + sw[b]) = make_uint4(h1[0], h1[1], h1[2], h1[3]);
                *reinterpret_cast<uint4 *>(sm + GO_A2 + sw[b]) = make_uint4(h2[0], h2[1], h2[2], h2[3]);
            }
        }
        fence_async_smem();
        fence_before();
        if (__syncthreads_or(!ok)) {
            ok = 0;
            break;
        }
        fence_after();
        if (warp == 0) {
            const uint64_t dO = desc_k(aO), dS = desc_k(aS), dA1 = desc_k(a1), dA1t = desc_mn(a1), dA2 = desc_k(a2), dA2t = desc_mn(a2);
            const uint64_t dKn = desc_mn(aK), dQn = desc_mn(aQ), dU = desc_k(aU), dD = desc_k(aD), dW = desc_k(aW);
            if (elect_one()) {
                mma_tile<kStepK, kStepK, false>(tbase + GC_DQ, dO, dS, idesc(64, 0, 0));
                mma_tile<kStepK, kStepMn, true>(tbase + GC_DQ, dA1, dKn, idesc(64, 0, 1));
                mma_tile<kStepK, kStepK, false>(tbase + GC_DWS, dW, dS, idesc(64, 0, 0));
                mma_tile<kStepK, kStepK, false>(tbase + GC_UDS, dU, dD, idesc(64, 0, 0));
                mma_tile<kStepK, kStepMn, false>(tbase + GC_DK, dA2, dKn, idesc(64, 0, 1));
                mma_tile<kStepMn, kStepMn, true>(tbase + GC_DK, dA2t, dKn, idesc(64, 1, 1));
                mma_tile<kStepMn, kStepMn, true>(tbase + GC_DK, dA1t, dQn, idesc(64, 1, 1));
                mma_commit(bar2);
            }
            __syncwarp();
        }
        Row qr, kr;
        tile_row(tQ, qr);
        tile_row(tK, kr);
        ok = bar_wait(bar2, ph, p.spin_limit);
        fence_after();
        if (n2 < total && warp == 7 && elect_one()) {  // the tiles are free (this thread stored the last chunk's)
            bulk_wait_read<0>();
            load(n2, nxt, buf ^ 1);
        }
        __syncwarp();
        // ---- dQ, dK, dV
        float e, r2;
        {
            const float a = diag[row], bg = -beta * gam;
            const P2 aa = pk(a, a);
            Raw rx, ry, rz;
            tmem_ld_blocks(tl + GC_DQ, rx);
            tmem_wait_ld();
            Row x = row_of(rx);
            e = dot(x, qr) + rowd;
#pragma unroll
            for (int i = 0; i < 8; ++i) x.x[i] = fma2(aa, kr.x[i], x.x[i]);
            if (p.dq_h) {
                if (valid) st_blocks(p.dq_h + at, x);
            } else if (whole) {
                put_row(GO_A1, x);
            } else if (valid) {
                st_blocks(p.dq + at, x);
            }
            tmem_ld_blocks(tl + GC_DK, rx);
            tmem_ld_blocks(tl + GC_DWS, ry);
            tmem_ld_blocks(tl + GC_UDS, rz);
            tmem_wait_ld();
            x = row_of(rx);
            const Row y = row_of(ry);
            Row z = row_of(rz);
            xt = fmaf(gam, dot(kr, y), xt);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x.x[i] = fma2(pk(bg, bg), y.x[i], x.x[i]);
                z.x[i] = mul2(z.x[i], pk(tail, tail));
            }
            e -= dot(kr, x);
            r2 = dot(kr, z);
#pragma unroll
            for (int i = 0; i < 8; ++i) x.x[i] = add2(x.x[i], fma2(aa, qr.x[i], z.x[i]));
            if (p.dk_h) {
                if (valid) st_blocks(p.dk_h + at, x);
            } else if (whole) {
                put_row(GO_A2, x);
            } else if (valid) {
                st_blocks(p.dk + at, x);
            }
            tile_row(tW, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) x.x[i] = mul2(x.x[i], pk(beta, beta));
            if (whole) put_row(tW, x);
            else if (valid) st_blocks(p.dv + at, x);
        }
        fence_async_smem();
        // ---- sums over a row's four threads, and over the chunk
        dwv += __shfl_xor_sync(0xffffffffu, dwv, 16);
        xt += __shfl_xor_sync(0xffffffffu, xt, 16);
        e += __shfl_xor_sync(0xffffffffu, e, 16);
        r2 += __shfl_xor_sync(0xffffffffu, r2, 16);
#pragma unroll
        for (int d = 1; d < 32; d *= 2) dots += __shfl_xor_sync(0xffffffffu, dots, d);
        if (lane < 16) {
            red[half * 64 + row] = dwv;
            red[128 + half * 64 + row] = xt;
            red[256 + half * 64 + row] = e;
            red[384 + half * 64 + row] = r2;
        }
        if (lane == 0) red[512 + warp] = dots;
        fence_before();
        if (__syncthreads_or(!ok)) {
            ok = 0;
            break;
        }
        fence_after();
        if (warp == 7) {
            if (elect_one()) {
                if (whole && tma_coord_ok(p.status, 0, 2, kN, cur.row_t + kC - 1, p.T)) {
                    const int h = static_cast<int>(cur.h), hk = static_cast<int>(cur.hk);
                    if (!p.dq_h) {
                        tma_store_4d(&map_dq, 0, hk, cur.row_t, cur.row_b, a1);
                        tma_store_4d(&map_dk, 0, hk, cur.row_t, cur.row_b, a2);
                    }
                    tma_store_4d(&map_dv, 0, h, cur.row_t, cur.row_b, aW);
                }
                bulk_commit();
                bulk_wait_read<0>();  // A1 and A2 are written again before this thread's next wait
            }
            __syncwarp();
        } else if (warp < 2) {
            const int t = tid;
            const float x = red[128 + t] + red[192 + t], own = red[384 + t] + red[448 + t];
            float s = red[256 + t] + red[320 + t] - 2.f * arr.beta[t] * x, before = own;
            for (int i = t >> 4; i < 4; ++i) s -= cols[64 * i + t];  // rows from the column's own block on
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {  // from the token to its warp's last; from the first to the token
                const float y = __shfl_down_sync(0xffffffffu, s, d), z = __shfl_up_sync(0xffffffffu, before, d);
                if (lane + d < 32) s += y;
                if (lane >= d) before += z;
            }
            if (lane == 0) red[520 + warp] = s;
            if (lane == 31) red[522 + warp] = before;
            before = __shfl_up_sync(0xffffffffu, before, 1);  // without the token itself
            if (lane == 0) before = 0.f;
            group_sync<2, 64>();
            if (warp == 0) s += red[521];
            else before += red[522];
            float dot_all = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) dot_all += red[512 + w];
            if (t < cur.tv && in_bounds(p.status, cur.t0 + t, 1, ntok)) {
                p.dg[(cur.t0 + t) * p.H + cur.h] = __float2bfloat16_rn(s + (before + arr.gamma[kC - 1] * dot_all));
                p.dbeta[(cur.t0 + t) * p.H + cur.h] = __float2bfloat16_rn(red[t] + red[64 + t] - x);
            }
        }
        n = n2;
    }
    leave(!ok);
}

// Byte layout of the workspace: T, four tiles for every chunk and value head, the value heads'
// shares of dq and dk.
struct Layout {
    size_t t, states, us, ds, dw, shares, total;
};
Layout layout(const DeltaArgs &a)
{
    const size_t tiles = static_cast<size_t>(delta_chunks(a) * a.H) * kTile;
    Layout l;
    l.t = 0;
    l.states = (delta_t_bytes(a) + 1023) / 1024 * 1024;
    l.us = l.states + tiles;
    l.ds = l.us + tiles;
    l.dw = l.ds + tiles;
    l.shares = l.dw + tiles;
    l.total = l.shares + (a.H == a.Hk ? 0 : static_cast<size_t>(2 * a.B * a.T * a.H * kN) * sizeof(float));
    return l;
}

}  // namespace

size_t delta_backward_tc_workspace_bytes(const DeltaArgs &a) { return layout(a).total; }

cudaError_t delta_backward_tc_launch(const DeltaBwdArgs &a, cudaStream_t s)
{
    const DeltaArgs &f = a.f;
    if (f.nseq * f.H == 0) return cudaSuccess;
    const int64_t chunks = delta_chunks(f);
    if (chunks * f.H > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const Layout l = layout(f);
    unsigned char *ws = static_cast<unsigned char *>(a.workspace);
    CUtensorMap mq, mk, mv, mo, mdq, mdk, mdv;
    if (!make_map(&mq, f.q, f.B, f.T, f.Hk) || !make_map(&mk, f.k, f.B, f.T, f.Hk) || !make_map(&mv, f.v, f.B, f.T, f.H) ||
        !make_map(&mo, a.dout, f.B, f.T, f.H) || !make_map(&mdq, a.dq, f.B, f.T, f.Hk) ||
        !make_map(&mdk, a.dk, f.B, f.T, f.Hk) || !make_map(&mdv, a.dv, f.B, f.T, f.H))
        return cudaErrorInvalidValue;
    cudaError_t e = delta_prep_launch(f, ws + l.t, s);
    if (e != cudaSuccess) return e;
    e = delta_states_launch(f, ws + l.t, ws + l.states, ws + l.us, s);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(delta_bwd_state_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kLoneSmemBytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(delta_bwd_grad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kGSmemBytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(delta_bwd_state_kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(delta_bwd_grad_kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e != cudaSuccess) return e;
    const __nv_bfloat16 *g = static_cast<const __nv_bfloat16 *>(f.g), *beta = static_cast<const __nv_bfloat16 *>(f.beta);
    const StateParams sp{f.B, f.T, f.Hk, f.H, f.nseq, f.offsets, g, beta, ws + l.t, chunks, f.scale, a.dsT, a.ds0,
                         ws + l.ds, ws + l.dw, f.status, g_chunked_inject_timeout ? 100u : 100000u,
                         g_chunked_inject_timeout};
    // The two walks read T and the inputs and nothing of each other: this one may start while the
    // first still runs (a programmatic launch; T's kernel was complete before the first began).  It
    // ends only after the first has, so that the next kernel, launched as usual, follows both.
    // With fewer sequences than the GPU holds they run side by side (5 sequences of up to 1023
    // tokens, 16 heads: 154 -> 121 us a call).
    cudaLaunchAttribute beside[1];
    beside[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    beside[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(f.nseq * f.H));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = 2 * f.nseq * f.H <= kLoneCtas ? kLoneSmemBytes : kSmemBytes;
    cfg.stream = s;
    cfg.attrs = beside;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, delta_bwd_state_kernel, mq, mk, mo, sp);
    if (e != cudaSuccess) return e;
    const bool shared = f.H != f.Hk;
    float *dq_h = shared ? reinterpret_cast<float *>(ws + l.shares) : nullptr;
    float *dk_h = shared ? dq_h + f.B * f.T * f.H * kN : nullptr;
    const GradParams gp{f.B, f.T, f.Hk, f.H, f.nseq, f.offsets, g, beta, f.scale,
                        ws + l.states, ws + l.us, ws + l.ds, ws + l.dw, chunks,
                        static_cast<__nv_bfloat16 *>(a.dq), static_cast<__nv_bfloat16 *>(a.dk),
                        static_cast<__nv_bfloat16 *>(a.dv), static_cast<__nv_bfloat16 *>(a.dg),
                        static_cast<__nv_bfloat16 *>(a.dbeta), dq_h, dk_h, f.status,
                        g_chunked_inject_timeout ? 100u : 100000u, g_chunked_inject_timeout};
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        sms <= 0)
        sms = 148;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(chunks * f.H, 2LL * sms));
    delta_bwd_grad_kernel<<<grid, kGThreads, kGSmemBytes, s>>>(mq, mk, mv, mo, mdq, mdk, mdv, gp);
    e = cudaGetLastError();
    if (e == cudaSuccess && shared) e = delta_sum_heads_launch(a, dq_h, dk_h, s);
    return e;
}

}  // namespace wkv
