// delta_chunked.cu -- the gated delta rule in 64-token chunks on B200 tensor cores (tcgen05 +
// TMA + TMEM), bf16 inputs.
//
// One CTA owns one (sequence, value head) and walks it chunk by chunk with the state S (64 x 64
// fp32) in registers.  delta_tc.cuh has the chunk's algebra; T of every chunk was formed before, in
// delta_prep.cu.  (Forming T here too, in the same warps, was slower: T's code and the chain's
// together do not stay in the instruction caches, and each ran at half its speed.)  Two CTAs
// share an SM.  Per chunk:
//   chain group (warps 4-7)   S -> K S -> W -> T W = U -> K^T diag(tail) U -> S: three products,
//                             each waiting for the last.  One warp issues them, another the copies
//                             of later chunks, both while the group waits for a product anyway;
//   output group (warps 0-3)  Q K^T and P a chunk ahead, scale diag(gamma) Q S + P U, the output.
//
// Accuracy.  The state is an fp32 result, so every operand between S and the next S is two bf16
// terms, hi and lo (K and V are exact): S, W, T and diag(tail) U, three products where both
// sides are split.  What that leaves is 2^-16 of each operand.  The output is rounded to bf16,
// and there P, U and the S of Q S are single bf16 (with 32 columns a CTA, below, only P is).
//
// A product of N = 64 takes 50 cycles of the tensor core whatever M is, one of N = 128 takes 64
// (measured): so the two terms of an operand lie side by side as one B of 128 columns, and their
// accumulators are added when they are read.
//
// Shared memory (13 tiles of 8 KB): K, Q and T (hi, lo) of two chunks, V of one (it is read early
// in the chain), P, and three chain tiles A, B, C in a row that take S hi/lo (A, B), W hi/lo
// (B, C), diag(tail) U hi/lo (A, B) and U (C) in turn.  Tensor memory (256 columns): the chain's
// accumulators (128) and, for two chunks, one that takes Q K^T and then the output.
//
// With few (sequence, head) pairs two CTAs take 32 of the 64 value columns each (NV): the columns of S
// are independent given K, and half of them is half of the conversions.  Both terms of an operand
// then lie in one tile, side by side, and Q S and P U take both too.
//
// The backward pass's first walk is the same kernel (STATES): without queries and outputs, it
// leaves the bf16 state before every chunk and U, as images of their tiles.
//
// Measured.  Bound by the latency of the chain: one CTA alone on its SM takes 4230 cycles a chunk,
// some 700 for each of the three products (256 to 450 of them the tensor core's) and the rest the
// conversions between registers, shared and tensor memory; two CTAs on an SM take 6230 for a chunk
// of each.  B8 T4096 H32: 210 us (STATES 185) after 84 to 91 for T; B8 T1024 H32: 64 us, tensor pipe
// 32 % active, DRAM 36 %, issue 33 %.  With 32 columns a CTA some 3900 cycles a chunk.  Slower: loads
// issued by the output group (331 us a call against 306), a vote of the group after every wait, a
// warp that only issues.
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
constexpr int OFF_DEC = 13 * kTile;                               // Decays
constexpr int OFF_ARR = OFF_DEC + static_cast<int>(sizeof(Decays));  // ChunkArrays, [chunk % 3]
constexpr int OFF_BAR = OFF_ARR + 3 * static_cast<int>(sizeof(ChunkArrays));
constexpr int OFF_MISC = OFF_BAR + 22 * 8;
constexpr int kSmemBytes = OFF_MISC + 32 + 1024;  // + alignment slack
static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM do not fit");
constexpr uint32_t COL_X = 0, COL_O = 128, kTmemCols = 256;

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
    unsigned char *states, *us;  // STATES: [chunks][H] tiles of 8 KB
    int *status;
    uint32_t spin_limit;
    int inject_timeout;
};

// The columns vcol .. vcol + NV - 1 of (sequence, head) number n.  STATES: the backward pass's walk.
template <bool STATES, int NV>
__device__ __forceinline__ void walk(const CUtensorMap *map_q, const CUtensorMap *map_k, const CUtensorMap *map_v,
                                     const Params &p, int64_t n, int vcol)
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
    const uint32_t bar_a = smem_u32(&bars[7]);    // Q K^T done
    const uint32_t bar_x = smem_u32(&bars[8]);    // K S, U, K^T U done (three phases a chunk)
    const uint32_t bar_qs = smem_u32(&bars[9]);   // Q S done
    const uint32_t bar_o = smem_u32(&bars[10]);   // P U done
    const uint32_t bar_sw = smem_u32(&bars[13]);  // S, U written
    const uint32_t bar_uw = smem_u32(&bars[16]);
    const uint32_t bar_never = smem_u32(&bars[17]);
    // decays written: + 8 * (chunk % 3), since the output group may pass two more chunks here before the
    // chain waits for this one
    const uint32_t bar_s0 = smem_u32(&bars[18]);
    const uint32_t bar_drain = smem_u32(&bars[21]);

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform, see elect_one
    const int64_t seq = n / p.H, h = n % p.H, hk = h / (p.H / p.Hk);
    int64_t first_, len_;
    sequence_span(p.offsets, seq, p.T, &first_, &len_);
    const int first = static_cast<int>(first_), len = static_cast<int>(len_);  // fewer than 2^31 tokens in all
    const int64_t slot = sequence_slot(p.slots, seq, p.nslots, tid == 0 ? p.status : nullptr);
    const int nchunks = (len + kC - 1) / kC;
    const int64_t chunk0 = first_chunk(p.offsets != nullptr, seq, first, p.T);
    // tensor-map coordinates of the sequence's first token
    const int row_b = p.offsets ? 0 : static_cast<int>(seq), row_t = p.offsets ? first : 0;
    const uint32_t spin = p.spin_limit;
    const int64_t ntok = p.B * p.T;

    if (tid == 0) {
        for (int i = 0; i < 22; ++i)
            bar_init(smem_u32(&bars[i]), i == 21 ? 3 : i > 17 ? 64 : 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        misc[1] = 0;
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(const_cast<uint32_t *>(misc))),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    // P is lower triangular: the blocks above the diagonal are zeroed once
    for (int i = tid; i < kTile / 16; i += kThreads)
        *reinterpret_cast<uint4 *>(sm + OFF_P + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
    fence_async_smem();
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tbase = misc[0];
    // The backward pass's other walk needs nothing of this one and may start beside it.
    if (STATES) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    auto load_tile = [&](const CUtensorMap *map, uint32_t off, int64_t head, int c, uint32_t bar) {
        if (!tma_coord_ok(p.status, 0, 2, kN, row_t + static_cast<int64_t>(c) * kC, p.T)) return;
        bar_expect_tx(bar, kTile);
        tma_load_4d(smem_u32(sm + off), map, 0, static_cast<int>(head), row_t + c * kC, row_b, bar);
    };
    auto load_t = [&](int c) {  // one thread
        if (!in_bounds(p.status, chunk0 + c, 1, p.nchunks)) return;
        const uint32_t bar = bar_t0 + 8 * (c & 1);
        bar_expect_tx(bar, kTBytes);
        bulk_load(smem_u32(sm + OFF_T + kTBytes * (c & 1)), p.t + ((chunk0 + c) * p.H + h) * kTBytes, kTBytes, bar);
    };
    if (warp == 7) {
        for (int c = 0; c < 2 && c < nchunks; ++c) {
            if (elect_one()) {
                load_tile(map_k, OFF_K + kTile * c, hk, c, bar_k0 + 8 * c);
                if (!STATES) load_tile(map_q, OFF_Q + kTile * c, hk, c, bar_q0 + 8 * c);
                if (c < 1) load_tile(map_v, OFF_V, h, c, bar_v);
            }
            __syncwarp();
        }
        if (!STATES) asm volatile("griddepcontrol.wait;" ::: "memory");  // T's kernel is done
        for (int c = 0; c < 2 && c < nchunks; ++c) {
            if (elect_one()) load_t(c);
            __syncwarp();
        }
    }
    int abort = 0;
    if (p.inject_timeout && tid == 0) abort = !bar_wait(bar_never, 0, p.spin_limit);
    abort = __syncthreads_or(abort);
    if (abort) misc[1] = 1;

    if (warp < 4) {
        // ---------------------------------------------------------------- output group
        const int w = warp;
        Decays &dec = *reinterpret_cast<Decays *>(sm + OFF_DEC);
        ChunkArrays *arrays = reinterpret_cast<ChunkArrays *>(sm + OFF_ARR);
        // Warps 2 and 3 prepare the decays; the tokens' g and beta are loaded a chunk ahead and
        // widened only when their chunk comes, so that nothing waits for the load before.
        const int st = tid - 64;
        uint16_t g_next = 0, b_next = 0;
        auto fetch = [&](int c) {
            const int t = c * kC + st;
            g_next = b_next = 0;
            if (t >= len || !in_bounds(p.status, first + t, 1, ntok)) return;
            const int64_t at = static_cast<int64_t>(first + t) * p.H + h;
            g_next = reinterpret_cast<const uint16_t *>(p.g)[at];
            b_next = reinterpret_cast<const uint16_t *>(p.beta)[at];
        };
        auto scan = [&](int c) {
            const float gv = widen(g_next), bv = widen(b_next);
            if (c + 1 < nchunks) fetch(c + 1);
            scan_decays<3>(dec, arrays[c % 3], st, gv, bv);
            bar_arrive(bar_s0 + 8 * (c % 3));
        };
        // Q K^T of chunk c (warp 0).  Rows past the sequence's end hold another's tokens; they stay in
        // rows of P that are not stored and in columns that the mask takes out.
        auto products = [&](int c) -> int {
            const uint32_t aK = smem_u32(sm + OFF_K + kTile * (c & 1)), aQ = smem_u32(sm + OFF_Q + kTile * (c & 1));
            const bool there = bar_wait(bar_k0 + 8 * (c & 1), (c >> 1) & 1, spin) &&
                               bar_wait(bar_q0 + 8 * (c & 1), (c >> 1) & 1, spin);
            if (!__all_sync(0xffffffffu, there)) return 0;
            fence_after();
            const uint64_t dk = desc_k(aK), dq = desc_k(aQ);
            if (elect_one()) {
                mma_tile<kStepK, kStepK, false>(tbase + COL_O + 64 * (c & 1), dq, dk, idesc(64, 0, 0));
                mma_commit(bar_a);
            }
            __syncwarp();
            return 1;
        };
        const uint32_t co = tbase + (static_cast<uint32_t>(32 * w) << 16) + COL_O;  // + 64 * (chunk % 2)
        const int row = 16 * w + (lane & 15), col = vcol + NV / 2 * (lane >> 4);  // its output row, first column
        auto store_o = [&](int c) {  // output rows of chunk c
            P2 x[NV / 4];
            if constexpr (NV == 64) tmem_ld_row(co + 64 * (c & 1), x);
            else tmem_ld_sum16<16, 32>(co + 64 * (c & 1), x);
            const int tok = c * kC + row;
            if (tok < len && in_bounds(p.status, first + tok, 1, ntok)) {
                uint4 *dst = reinterpret_cast<uint4 *>(p.o + (static_cast<int64_t>(first + tok) * p.H + h) * kN + col);
#pragma unroll
                for (int i = 0; i < NV / 16; ++i)
                    dst[i] = make_uint4(pack2(x[4 * i]), pack2(x[4 * i + 1]), pack2(x[4 * i + 2]), pack2(x[4 * i + 3]));
            }
        };
        int ok = 1;
        uint32_t ph[4][4], pl[4][4];  // P of the next chunk to store; pl: unused
        if (!abort && nchunks > 0) {
            if (w >= 2) {
                fetch(0);
                scan(0);
            }
            if (!STATES) {
                if (w == 0) ok = products(0);
                group_sync<1, 128>();
                if (ok) ok = bar_wait(bar_a, 0, spin);
                fence_after();
                form_p<false>(dec, w, lane, co, p.scale, ph, pl);
                fence_before();
            }
        }
        for (int c = 0; c < nchunks && !abort; ++c) {
            if (misc[1]) ok = 0;
            group_sync<1, 128>();  // Q K^T and the decays have been read
            if (STATES) {  // nothing but the next chunk's decays
                if (ok && c > 0) ok = bar_wait(bar_o, (c - 1) & 1, spin);
                if (!ok) misc[1] = 1;
                if (w >= 2 && c + 1 < nchunks) scan(c + 1);
                continue;
            }
            const uint32_t dst = tbase + COL_O + 64 * (c & 1);
            if (w == 1) {  // Q S, once S is written
                if (ok) ok = bar_wait(bar_sw, c & 1, spin);
                fence_after();
                __syncwarp();
                const uint64_t dQ = desc_k(smem_u32(sm + OFF_Q + kTile * (c & 1))), dS = desc_mn(smem_u32(sm + OFF_A));
                if (elect_one()) {
                    mma_tile<kStepK, kStepMn, false>(dst, dQ, dS, idesc(64, 0, 1));
                    mma_commit(bar_qs);
                }
                __syncwarp();
            }
            if (w >= 2 && c + 1 < nchunks) scan(c + 1);
            if (c > 0) {
                if (ok) ok = bar_wait(bar_o, (c - 1) & 1, spin);  // P has been read, the output is there
                fence_after();
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j <= w) st_block(sm + OFF_P, w, j, lane, ph[j]);
            fence_async_smem();
            if (c > 0) store_o(c - 1);
            // scale diag(gamma) Q S, in place
            if (ok) ok = bar_wait(bar_qs, c & 1, spin);
            fence_after();
            {
                float v[32];
                tmem_ld32(co + 64 * (c & 1), v);
                const float sg = p.scale * arrays[c % 3].gamma[row];
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] *= sg;
                tmem_st32(co + 64 * (c & 1), v);
            }
            fence_before();
            group_sync<1, 128>();
            if (c + 1 < nchunks) {
                if (w == 0 && !products(c + 1)) ok = 0;
                if (ok) ok = bar_wait(bar_a, (c + 1) & 1, spin);
                fence_after();
                form_p<false>(dec, w, lane, co + 64 * ((c + 1) & 1), p.scale, ph, pl);
                fence_before();
            }
            if (w == 1) {  // + P U
                if (ok) ok = bar_wait(bar_uw, c & 1, spin);
                fence_after();
                __syncwarp();
                const uint64_t dP = desc_k(smem_u32(sm + OFF_P)), dU = desc_mn(smem_u32(sm + OFF_CC));
                if (elect_one()) {
                    mma_tile<kStepK, kStepMn, true>(dst, dP, dU, idesc(64, 0, 1));
                    mma_commit(bar_o);
                }
                __syncwarp();
            }
            if (!ok) misc[1] = 1;
        }
        if (!STATES && !abort && nchunks > 0) {
            if (ok) ok = bar_wait(bar_o, (nchunks - 1) & 1, spin);
            fence_after();
            if (ok) store_o(nchunks - 1);
        }
        if (!ok) misc[1] = 1;
    } else {
        // ------------------------------------------------------------------ chain group
        const int q = warp & 3;
        const uint32_t tl = tbase + (static_cast<uint32_t>(32 * q) << 16);
        constexpr int kHalves = NV / 32;  // a thread's columns, 16 at a time
        const int row = 16 * q + (lane & 15), col = NV / 2 * (lane >> 4);  // its row, first of 16 kHalves columns
        unsigned char *tA = sm + OFF_A, *tB = sm + OFF_B, *tC = sm + OFF_CC;
        unsigned char *tA2 = NV == 64 ? tB : tA, *tB2 = NV == 64 ? tC : tB;  // of the low terms
        const int64_t nstate = p.nslots * p.H * kN * kN;
        const int64_t sat = ((slot * p.H + h) * kN + row) * kN + vcol + col;
        P2 S[8 * kHalves];
        if (p.s0 && slot >= 0 && in_bounds(p.status, sat, NV / 2, nstate)) {
            const float4 *src = reinterpret_cast<const float4 *>(p.s0 + sat);
#pragma unroll
            for (int i = 0; i < 4 * kHalves; ++i) {
                const float4 x = src[i];
                S[2 * i] = pk(x.x, x.y);
                S[2 * i + 1] = pk(x.z, x.w);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8 * kHalves; ++i) S[i] = pk(0.f, 0.f);
        }
        // this thread's columns of a tile: i-th 16 bytes, also of the low terms and of V
        const uint32_t at0 = swz(row, 2 * col), av0 = swz(row, 2 * (vcol + col));
        auto at = [&](int i) { return at0 ^ static_cast<uint32_t>(16 * i); };
        auto at_lo = [&](int i) { return at(i) ^ (NV == 32 ? 64u : 0u); };
        auto at_v = [&](int i) { return av0 ^ static_cast<uint32_t>(16 * i); };
        // 16 of them as two bf16 terms, in two tiles or, of 32 columns, side by side in one
        auto store_split = [&](const P2 *x, int half, unsigned char *th, unsigned char *tlo) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t a[4], b[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) split2(x[4 * i + e], &a[e], &b[e]);
                *reinterpret_cast<uint4 *>(th + at(2 * half + i)) = make_uint4(a[0], a[1], a[2], a[3]);
                *reinterpret_cast<uint4 *>(tlo + at_lo(2 * half + i)) = make_uint4(b[0], b[1], b[2], b[3]);
            }
        };
        const uint64_t dA = desc_mn(smem_u32(tA)), dB = desc_mn(smem_u32(tB));
        constexpr uint32_t kId = idesc(64, 0, 1), kId2 = idesc(2 * NV, 0, 1), kIdT2 = idesc(2 * NV, 1, 1);
        // group barrier: what was written is ready for the products issued next.  After a wait that ran
        // out every thread walks on, without waiting and without loading, so that the barriers hold.
        auto meet = [&]() {
            fence_async_smem();
            fence_before();
            group_sync<2, 128>();
            fence_after();
        };
        uint32_t xph = 0;  // phase of bar_x
        int ok = !abort;
        for (int c = 0; c < nchunks && !abort; ++c) {
            const uint32_t aK = smem_u32(sm + OFF_K + kTile * (c & 1));
            const int64_t tile = ((chunk0 + c) * p.H + h) * kTile;
            // ---- S hi, lo; K S
            if (misc[1]) ok = 0;
#pragma unroll
            for (int half = 0; half < kHalves; ++half) store_split(S + 8 * half, half, tA, tA2);
            if (c * kC + kC > len) {  // the last chunk's rows past the end
                if (ok) ok = bar_wait(bar_k0 + 8 * (c & 1), (c >> 1) & 1, spin);
                zero_rows(sm + OFF_K + kTile * (c & 1), len - c * kC, tid - 128, 128);
            }
            meet();
            if (warp == 4) {
                const uint64_t dK = desc_k(aK);
                if (ok) ok = bar_wait_spin(bar_k0 + 8 * (c & 1), (c >> 1) & 1, spin * 64u);
                __syncwarp();
                if (elect_one()) {
                    mma_tile<kStepK, kStepMn, false>(tbase + COL_X, dK, dA, kId2);
                    mma_commit(bar_x);
                }
            } else if (STATES && warp == 5 && lane == 0) {
                if (in_bounds(p.status, chunk0 + c, 1, p.nchunks)) bulk_store(p.states + tile, smem_u32(tA), kTile);
                bulk_commit();
                bulk_wait_read<0>();
                bar_arrive(bar_qs);
            } else if (warp == 7 && c > 0 && c + 1 < nchunks) {  // S is there: the chunk before is done with its tiles
                if (elect_one() && ok) {
                    load_tile(map_k, OFF_K + kTile * ((c + 1) & 1), hk, c + 1, bar_k0 + 8 * ((c + 1) & 1));
                    if (!STATES) load_tile(map_q, OFF_Q + kTile * ((c + 1) & 1), hk, c + 1, bar_q0 + 8 * ((c + 1) & 1));
                }
            }
            __syncwarp();
            // ---- W = beta (v - gamma K S)
            if (ok) ok = bar_wait(bar_s0 + 8 * (c % 3), (c / 3) & 1, spin);
            const ChunkArrays &arr = reinterpret_cast<const ChunkArrays *>(sm + OFF_ARR)[c % 3];
            const float gam = arr.gamma[row], tail = arr.tail[row], bet = arr.beta[row], gC = arr.gamma[kC - 1];
            const P2 b2 = pk(bet, bet), bg = pk(-bet * gam, -bet * gam), t2 = pk(tail, tail), g2 = pk(gC, gC);
            if (ok) ok = bar_wait(bar_v, c & 1, spin);
            if (ok && c > 0) ok = bar_wait(bar_o, (c - 1) & 1, spin);  // P U has read U
            if (ok) ok = bar_wait(bar_t0 + 8 * (c & 1), (c >> 1) & 1, spin);
            if (ok) ok = bar_wait(bar_x, xph, spin);
            xph ^= 1;
            fence_after();
            // only now may Q S be issued: beside K S it would hold that up
            if (!STATES && warp == 5 && lane == 0) bar_arrive(bar_sw);
            __syncwarp();
            const bool token = c * kC + row < len;  // else another sequence's, or nothing
#pragma unroll
            for (int half = 0; half < kHalves; ++half) {
                P2 x[8];
                tmem_ld_sum16<NV / 2, NV>(tl + COL_X + 16 * half, x);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint4 vv = make_uint4(0u, 0u, 0u, 0u);
                    if (token) vv = *reinterpret_cast<const uint4 *>(sm + OFF_V + at_v(2 * half + i));
                    const uint32_t vw[4] = {vv.x, vv.y, vv.z, vv.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[4 * i + e] = fma2(bg, x[4 * i + e], mul2(b2, unpack2(vw[e])));
                }
                store_split(x, half, tB, tB2);
            }
            meet();
            if (warp == 4) {  // ---- U = T W
                const uint32_t aT = smem_u32(sm + OFF_T + 2 * kTile * (c & 1));
                const uint64_t dTh = desc_t(aT), dTl = desc_t(aT + kTile);
                if (elect_one()) {
                    mma_tile<kStepTK, kStepMn, false>(tbase + COL_X, dTh, dB, kId2);
                    mma_tile<kStepTK, kStepMn, true>(tbase + COL_X, dTl, dB, kId);
                    mma_commit(bar_x);
                }
                __syncwarp();
            } else if (warp == 7 && c + 1 < nchunks) {
                if (elect_one() && ok) load_tile(map_v, OFF_V, h, c + 1, bar_v);
                __syncwarp();
            }
            // ---- U, and diag(tail) U hi, lo
            if (ok) ok = bar_wait(bar_qs, c & 1, spin);  // Q S has read S
            if (ok) ok = bar_wait(bar_x, xph, spin);
            xph ^= 1;
            fence_after();
#pragma unroll
            for (int half = 0; half < kHalves; ++half) {
                P2 x[8];
                tmem_ld_sum16<NV / 2, NV>(tl + COL_X + 16 * half, x);
                if (NV == 32) store_split(x, half, tC, tC);
#pragma unroll
                for (int i = 0; i < 2 && NV == 64; ++i)
                    *reinterpret_cast<uint4 *>(tC + at(2 * half + i)) =
                        make_uint4(pack2(x[4 * i]), pack2(x[4 * i + 1]), pack2(x[4 * i + 2]), pack2(x[4 * i + 3]));
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = mul2(x[i], t2);
                store_split(x, half, tA, tA2);
            }
            meet();
            if (warp == 4) {  // ---- K^T diag(tail) U
                const uint64_t dKt = desc_mn(aK);
                if (elect_one()) {
                    mma_tile<kStepMn, kStepMn, false>(tbase + COL_X, dKt, dA, kIdT2);
                    mma_commit(bar_x);
                }
                __syncwarp();
            } else if (STATES && warp == 5 && lane == 0) {
                if (in_bounds(p.status, chunk0 + c, 1, p.nchunks)) bulk_store(p.us + tile, smem_u32(tC), kTile);
                bulk_commit();
                bulk_wait_read<0>();
                bar_arrive(bar_o);
            } else if (warp == 7 && c + 2 < nchunks) {
                if (elect_one() && ok) load_t(c + 2);
            }
            __syncwarp();
            // ---- S
            if (ok) ok = bar_wait(bar_x, xph, spin);
            xph ^= 1;
            fence_after();
            if (!STATES && warp == 5 && lane == 0) bar_arrive(bar_uw);  // P U, likewise
            __syncwarp();
#pragma unroll
            for (int half = 0; half < kHalves; ++half) {
                P2 x[8];
                tmem_ld_sum16<NV / 2, NV>(tl + COL_X + 16 * half, x);
#pragma unroll
                for (int i = 0; i < 8; ++i) S[8 * half + i] = fma2(g2, S[8 * half + i], x[i]);
            }
            if (!ok) misc[1] = 1;  // and its waits pass from here on, in this thread and soon in all
        }
        if (STATES && warp == 5 && lane == 0) bulk_wait_all();
        if (abort) ok = 0;
        if (!ok) misc[1] = 1;
        if (ok && p.sT && slot >= 0 && in_bounds(p.status, sat, NV / 2, nstate)) {
            float4 *dst = reinterpret_cast<float4 *>(p.sT + sat);
#pragma unroll
            for (int i = 0; i < 4 * kHalves; ++i) dst[i] = make_float4(lo(S[2 * i]), hi(S[2 * i]), lo(S[2 * i + 1]), hi(S[2 * i + 1]));
        }
    }

    // ---- drain after an abort, then release tensor memory
    fence_before();
    abort = __syncthreads_or(abort | misc[1]);
    fence_after();
    if (abort) {
        record_status(p.status, kStatusTimeout);
        if ((warp == 0 || warp == 1 || warp == 4) && elect_one()) mma_commit(bar_drain);  // the issuers
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

// Most (sequence, head) pairs that take two CTAs each, of 32 value columns: less to convert between
// two products, as long as each CTA has an SM.  64 columns against 32, us: B1 T4096 H8 157 / 136, H64
// 192 / 179; B1 T2048 H74 101 / 97; B2 T1024 H50 58 / 64.
constexpr int64_t kNarrowPairs = 74;
// Most pairs of a packed call that decides by its lengths: the pairs walking at a time are on average
// the tokens over the longest sequence, times the heads, and that is what has to be few.  13
// sequences of 0 to 2048 tokens, 6665 in all, H16: 106 us with 64 columns, 97 with 32.
constexpr int64_t kPackedPairs = 1024;

// Whether a packed call's pairs take two CTAs each.  All threads of the block; every block finds the same.
__device__ __forceinline__ bool few_at_a_time(const Params &p)
{
    __shared__ unsigned warp_max[kThreads / 32], warp_sum[kThreads / 32];
    unsigned most = 0, sum = 0;
    for (int64_t i = threadIdx.x; i < p.nseq; i += kThreads) {
        int64_t first, len;
        sequence_span(p.offsets, i, p.T, &first, &len);
        most = max(most, static_cast<unsigned>(len));
        sum += static_cast<unsigned>(len);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    sum = __reduce_add_sync(0xffffffffu, sum);
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = most, warp_sum[threadIdx.x >> 5] = sum;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) {
        most = w ? max(most, warp_max[w]) : warp_max[w];
        sum = w ? sum + warp_sum[w] : warp_sum[w];
    }
    return static_cast<int64_t>(sum) * p.H <= kNarrowPairs * static_cast<int64_t>(most);
}

// NV: value columns of a CTA, 64 or, in two CTAs, 32; 0: as few_at_a_time says.
template <bool STATES, int NV>
__global__ void __launch_bounds__(kThreads, 2)
delta_chunked_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const Params p)
{
    if constexpr (NV > 0) {
        walk<STATES, NV>(&map_q, &map_k, &map_v, p, blockIdx.x / (kN / NV), NV * static_cast<int>(blockIdx.x % (kN / NV)));
    } else {
        const int64_t n = blockIdx.x / 2;
        const int part = blockIdx.x % 2;
        if (few_at_a_time(p)) walk<STATES, 32>(&map_q, &map_k, &map_v, p, n, 32 * part);
        else if (part == 0) walk<STATES, 64>(&map_q, &map_k, &map_v, p, n, 0);
    }
}

template <bool STATES, int NV>
cudaError_t launch(const DeltaArgs &a, const void *t, void *states, void *us, cudaStream_t s)
{
    if (a.nseq * a.H == 0) return cudaSuccess;
    CUtensorMap mq, mk, mv;
    if (!make_map(&mq, STATES ? a.k : a.q, a.B, a.T, a.Hk) || !make_map(&mk, a.k, a.B, a.T, a.Hk) ||
        !make_map(&mv, a.v, a.B, a.T, a.H))
        return cudaErrorInvalidValue;
    auto kern = delta_chunked_kernel<STATES, NV>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kLoneSmemBytes);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e != cudaSuccess) return e;
    const Params p{a.B, a.T, a.Hk, a.H, a.nseq, a.nslots, a.offsets, a.slots, static_cast<const __nv_bfloat16 *>(a.g),
                   static_cast<const __nv_bfloat16 *>(a.beta), static_cast<const unsigned char *>(t), delta_chunks(a),
                   a.scale, a.s0, static_cast<__nv_bfloat16 *>(a.o), a.sT, static_cast<unsigned char *>(states),
                   static_cast<unsigned char *>(us), a.status, g_chunked_inject_timeout ? 100u : 100000u,
                   g_chunked_inject_timeout};
    // The forward walk may start (barriers, tensor memory, the first tiles) while T's kernel still runs.
    cudaLaunchAttribute early[1];
    early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    const int64_t ctas = a.nseq * a.H * (NV == 64 ? 1 : 2);
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (STATES ? 2 : 1) * ctas <= kLoneCtas ? kLoneSmemBytes : kSmemBytes;
    cfg.stream = s;
    cfg.attrs = early;
    cfg.numAttrs = STATES ? 0 : 1;
    return cudaLaunchKernelEx(&cfg, kern, mq, mk, mv, p);
}
}  // namespace

cudaError_t delta_chunked_launch(const DeltaArgs &a, const void *t, cudaStream_t s)
{
    const int64_t pairs = a.nseq * a.H;
    if (pairs <= kNarrowPairs) return launch<false, 32>(a, t, nullptr, nullptr, s);
    if (a.offsets && pairs <= kPackedPairs) return launch<false, 0>(a, t, nullptr, nullptr, s);
    return launch<false, 64>(a, t, nullptr, nullptr, s);
}

cudaError_t delta_states_launch(const DeltaArgs &a, const void *t, void *states, void *us, cudaStream_t s)
{
    return launch<true, 64>(a, t, states, us, s);
}

}  // namespace wkv
