// state_pool.cu -- copying, forking, freeing and compacting slots of a pool of states.
//
// A pool is [layers, nslots, slot_bytes].  Both kernels work on byte ranges: a task is one range
// of W bytes of one layer, taken for all the slots of the call together.  What happens to one
// byte range never depends on another, so a block needs no agreement with other blocks:
//   copy     every source's range is loaded into shared memory before any destination's is
//            written, so the call acts as if all sources were read first (swaps, cycles and
//            shifts included), with no scratch in global memory.  A source named by several
//            pairs (a fork) is loaded once.  Of several pairs with one destination the last counts.
//   compact  the j-th live slot moves to slot j.  A destination lies at or before its source,
//            so a batch of moves, loaded whole before it is stored, never overwrites a source
//            of a later batch, and the next batch may load while this one is stored.
//
// Both are bound by the bytes: data goes global -> shared -> global by bulk copies and never
// passes through registers.  One warp moves the data (each lane issues the copies of its own
// pairs) through two stages, so one task loads while the other is stored; blocks stay
// resident and take tasks in turn.  Measured: 64 forks of 8 states and 2 freed slots over 12 layers of
// 32 heads 90 us, 5.2 TB/s (nine bytes in ten are written); a pool of 256 states of 64 heads, half of
// them live, compacted in 50 us, 5.3 TB/s.
//
// A copy is at its best with few sources.  A stage holds one range of each, so the ranges shrink to
// 400 bytes at 256 sources and 16 at 4096, and every block compares the pairs with one another before
// its first byte.  Permutations over 12 layers: 256 states of 32 heads 1.66 ms (1.9 TB/s), 1024 of 4
// heads 3.7 ms (0.44), 4096 of one head 23 ms (0.07).
#include "tc_common.cuh"

#include <algorithm>

namespace wkv {
namespace {
using namespace tc;

constexpr int kThreads = 256;
constexpr int kCopySmem = 224 * 1024;      // the copy kernel's block owns an SM
constexpr int kZeroBytes = 8 * 1024;       // zeros for freed slots, and the largest copy range
constexpr int kCompactStage = 32 * 1024;   // two stages, three blocks per SM

// Bytes of a task's range: at most `most`, a multiple of 16, so that `blocks` blocks have the same number
// of tasks as nearly as it can be, but no less than 512 where `most` allows (shorter bulk copies waste
// their issue).  A pool of no layers or of empty slots has no tasks, and any range serves.
__host__ __device__ int64_t pick_range(int64_t layers, int64_t slot_bytes, int64_t most, int64_t blocks)
{
    if (most < 16) most = 16;
    if (layers == 0 || slot_bytes == 0) return most / 16 * 16;
    const int64_t least = most < 512 ? most : 512, per = (slot_bytes + most - 1) / most;
    const int64_t rounds = (layers * per + blocks - 1) / blocks, even = rounds * blocks / layers;
    const int64_t range = even > per ? (slot_bytes + even - 1) / even : most;
    return ((range > least ? range : least) + 15) / 16 * 16 < most ? ((range > least ? range : least) + 15) / 16 * 16
                                                                    : most / 16 * 16;
}

struct CopyParams {
    StateCopyArgs a;
    int stage;              // bytes of one of the two stages
    uint32_t wait_limit;
    int inject_timeout;
};

// Whether the warp's wait for its it-th stage was met.  If it ran out, the copies in flight (the next
// stage's too, with `next`) have been waited for as well, with the same limit.
template <typename P> __device__ __forceinline__ bool arrived(const P &p, const uint64_t *bars, int64_t it, bool next)
{
    const uint32_t bar = smem_u32(&bars[it & 1]), phase = static_cast<uint32_t>((it >> 1) & 1);
    const bool ok = p.inject_timeout ? bar_wait(smem_u32(&bars[2]), 0, p.wait_limit) : bar_wait(bar, phase, p.wait_limit);
    if (__all_sync(0xffffffffu, ok)) return true;
    if ((threadIdx.x & 31) == 0) record_status(p.a.status, kStatusTimeout);
    bar_wait(bar, phase, p.wait_limit);
    if (next) bar_wait(smem_u32(&bars[(it + 1) & 1]), static_cast<uint32_t>(((it + 1) >> 1) & 1), p.wait_limit);
    return false;
}

// Shared memory: the two stages, zeros, then per pair its source and destination, the pair that
// loads its source (itself, an earlier one, -1: zeros, -2: the pair does nothing) and, for a
// loading pair, its place in the stage.
__global__ void __launch_bounds__(kThreads)
state_copy_kernel(const CopyParams p)
{
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
    unsigned char *zeros = sm + 2 * p.stage;
    __shared__ uint64_t bars[3];  // the stages loaded; the third is never signalled
    __shared__ int nload;
    const int n = static_cast<int>(p.a.n), tid = threadIdx.x;
    int *src = reinterpret_cast<int *>(zeros + kZeroBytes), *dst = src + n, *from = dst + n, *pos = from + n;
    const int nslots = static_cast<int>(p.a.nslots);

    for (int i = tid; i < n; i += kThreads) {
        int s = p.a.src[i], d = p.a.dst[i];
        if (s >= nslots || d >= nslots) {  // outside the pool: the pair is left out
            record_status(p.a.status, kStatusArg);
            d = -1;
        }
        src[i] = s < 0 ? -1 : s;
        dst[i] = d < 0 ? -1 : d;
    }
    for (int i = tid; i < kZeroBytes / 16; i += kThreads) reinterpret_cast<uint4 *>(zeros)[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) {
        nload = 0;
        for (int i = 0; i < 3; ++i) bar_init(smem_u32(&bars[i]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    // a pair whose destination a later pair names again does nothing, nor does one that names
    // its own slot; a pair's source is loaded by the first pair that still has it
    for (int i = tid; i < n; i += kThreads) {
        const int d = dst[i];
        int dead = d < 0 || d == src[i];
        for (int j = i + 1; j < n && !dead; ++j) dead = dst[j] == d;
        from[i] = dead ? -2 : -1;
    }
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
        const int s = src[i];
        if (from[i] == -2 || s < 0) continue;
        int j = 0;
        while (j < i && !(src[j] == s && from[j] != -2)) ++j;
        from[i] = j;  // never -2 or -1, so a concurrent reader's test above is unchanged
    }
    __syncthreads();
    fence_async_smem();  // the zeros are read by bulk stores
    // stage positions in pair order: position of pair i's own load = loading pairs before it
    if (tid < 32) {
        int count = 0;
        for (int i0 = 0; i0 < n; i0 += 32) {
            const int i = i0 + tid;
            const bool loads = i < n && from[i] == i;
            const unsigned m = __ballot_sync(0xffffffffu, loads);
            if (loads) pos[i] = count + __popc(m & ((1u << tid) - 1));
            count += __popc(m);
        }
        if (tid == 0) nload = count;
    }
    __syncthreads();
    if (tid >= 32) return;
    const int lane = tid;
    // bytes of one task's range: the stage holds one of every source, however many pairs share them
    const int64_t range = pick_range(p.a.layers, p.a.slot_bytes, min(kZeroBytes, p.stage / max(nload, 1) / 16 * 16), gridDim.x);
    const int64_t per_layer = (p.a.slot_bytes + range - 1) / range, tasks = p.a.layers * per_layer;
    const int64_t layer_bytes = p.a.nslots * p.a.slot_bytes;
    const int64_t pool_bytes = p.a.layers * layer_bytes;
    auto load = [&](int64_t task, int st) {
        const int64_t layer = task / per_layer, off = task % per_layer * range;
        const uint32_t w = static_cast<uint32_t>(min(range, p.a.slot_bytes - off));
        const uint32_t bar = smem_u32(&bars[st]);
        if (lane == 0) bar_expect_tx(bar, w * nload);
        __syncwarp();
        for (int i = lane; i < n; i += 32)
            if (from[i] == i) {
                const int64_t at = layer * layer_bytes + src[i] * p.a.slot_bytes + off;
                if (in_bounds(p.a.status, at, w, pool_bytes) &&
                    in_bounds(p.a.status, pos[i] * range, w, p.stage))
                    bulk_load(smem_u32(sm + st * p.stage + pos[i] * range), p.a.pool + at, w, bar);
            }
    };
    int64_t it = 0;
    if (blockIdx.x < tasks) load(blockIdx.x, 0);
    for (int64_t task = blockIdx.x; task < tasks; task += gridDim.x, ++it) {
        const int st = static_cast<int>(it & 1);
        if (task + gridDim.x < tasks) {
            bulk_wait_read<0>();  // this lane's stores of the task before have read the other stage
            __syncwarp();
            load(task + gridDim.x, st ^ 1);
        }
        if (!arrived(p, bars, it, task + gridDim.x < tasks)) break;
        const int64_t layer = task / per_layer, off = task % per_layer * range;
        const uint32_t w = static_cast<uint32_t>(min(range, p.a.slot_bytes - off));
        for (int i = lane; i < n; i += 32) {
            const int f = from[i];
            if (f == -2) continue;
            const int64_t at = layer * layer_bytes + dst[i] * p.a.slot_bytes + off;
            if (in_bounds(p.a.status, at, w, pool_bytes))
                bulk_store(p.a.pool + at, smem_u32(f < 0 ? zeros : sm + st * p.stage + pos[f] * range), w);
        }
        bulk_commit();
    }
    bulk_wait_all();
}

struct CompactParams {
    StateCompactArgs a;
    int64_t range, per_layer;
    int batch;              // moves per stage
    uint32_t wait_limit;
    int inject_timeout;
};

__global__ void __launch_bounds__(kThreads)
state_compact_kernel(const CompactParams p)
{
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
    uint16_t *list = reinterpret_cast<uint16_t *>(sm + 2 * kCompactStage);  // live slots in order
    __shared__ uint64_t bars[3];  // as above
    __shared__ int warp_sum[kThreads / 32], s_first;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nslots = static_cast<int>(p.a.nslots);
    if (tid == 0) {
        s_first = nslots;
        for (int i = 0; i < 3; ++i) bar_init(smem_u32(&bars[i]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    int count = 0;
    for (int i0 = 0; i0 < nslots; i0 += kThreads) {  // places of the live slots, 256 at a time
        const int i = i0 + tid;
        const bool live = i < nslots && p.a.live[i] != 0;
        const unsigned m = __ballot_sync(0xffffffffu, live);
        if (lane == 0) warp_sum[warp] = __popc(m);
        __syncthreads();
        int at = count + __popc(m & ((1u << lane) - 1));
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) at += warp_sum[w];
            count += warp_sum[w];
        }
        if (live) {
            list[at] = static_cast<uint16_t>(i);
            if (at != i) atomicMin(&s_first, at);
        }
        if (blockIdx.x == 0 && i < nslots) p.a.new_index[i] = live ? at : -1;
        __syncthreads();
    }
    if (blockIdx.x == 0 && tid == 0) *p.a.count = count;
    if (warp != 0) return;
    const int first = s_first;  // moves are live places first .. count - 1
    if (first >= count) return;
    const int nb = (count - first + p.batch - 1) / p.batch;  // batches per range
    const int64_t tasks = p.a.layers * p.per_layer;
    const int64_t mine = tasks > blockIdx.x ? (tasks - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
    const int64_t total = mine * nb;
    const int64_t layer_bytes = p.a.nslots * p.a.slot_bytes, pool_bytes = p.a.layers * layer_bytes;
    auto where = [&](int64_t it, int64_t *base, uint32_t *w, int *m0, int *m1) {
        const int64_t task = blockIdx.x + it / nb * gridDim.x;
        const int64_t off = task % p.per_layer * p.range;
        *base = task / p.per_layer * layer_bytes + off;
        *w = static_cast<uint32_t>(min(p.range, p.a.slot_bytes - off));
        *m0 = first + static_cast<int>(it % nb) * p.batch;
        *m1 = min(*m0 + p.batch, count);
    };
    auto load = [&](int64_t it) {
        int64_t base;
        uint32_t w;
        int m0, m1;
        where(it, &base, &w, &m0, &m1);
        const int st = static_cast<int>(it & 1);
        const uint32_t bar = smem_u32(&bars[st]);
        if (lane == 0) bar_expect_tx(bar, w * (m1 - m0));
        __syncwarp();
        for (int m = m0 + lane; m < m1; m += 32) {
            const int64_t at = base + list[m] * p.a.slot_bytes;
            if (in_bounds(p.a.status, at, w, pool_bytes) && in_bounds(p.a.status, (m - m0) * p.range, w, kCompactStage))
                bulk_load(smem_u32(sm + st * kCompactStage + (m - m0) * p.range), p.a.pool + at, w, bar);
        }
    };
    if (total > 0) load(0);
    for (int64_t it = 0; it < total; ++it) {
        const int st = static_cast<int>(it & 1);
        if (it + 1 < total) {
            bulk_wait_read<0>();  // the other stage's stores have read it
            __syncwarp();
            load(it + 1);
        }
        if (!arrived(p, bars, it, it + 1 < total)) break;
        int64_t base;
        uint32_t w;
        int m0, m1;
        where(it, &base, &w, &m0, &m1);
        for (int m = m0 + lane; m < m1; m += 32) {
            const int64_t at = base + m * p.a.slot_bytes;
            if (in_bounds(p.a.status, at, w, pool_bytes))
                bulk_store(p.a.pool + at, smem_u32(sm + st * kCompactStage + (m - m0) * p.range), w);
        }
        bulk_commit();
    }
    bulk_wait_all();
}

uint32_t wait_limit() { return g_chunked_inject_timeout ? 100u : 100000u; }

int64_t sms()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
        return 148;
    return n;
}

}  // namespace

cudaError_t state_copy_launch(const StateCopyArgs &a, cudaStream_t s)
{
    const int64_t stage = (kCopySmem - 128 - kZeroBytes - 16 * a.n) / 2 / 128 * 128;
    const cudaError_t e = cudaFuncSetAttribute(state_copy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kCopySmem);
    if (e != cudaSuccess) return e;
    const unsigned grid = static_cast<unsigned>(std::min(a.layers * ((a.slot_bytes + 511) / 512), sms()));
    state_copy_kernel<<<grid, kThreads, kCopySmem, s>>>(CopyParams{a, static_cast<int>(stage), wait_limit(), g_chunked_inject_timeout});
    return cudaGetLastError();
}

cudaError_t state_compact_launch(const StateCompactArgs &a, cudaStream_t s)
{
    const int64_t blocks = 3 * sms();
    const int64_t range = pick_range(a.layers, a.slot_bytes, 4096, blocks);
    const int64_t per_layer = (a.slot_bytes + range - 1) / range;
    const int smem = 2 * kCompactStage + static_cast<int>(a.nslots) * 2 + 128;
    const cudaError_t e = cudaFuncSetAttribute(state_compact_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               2 * kCompactStage + static_cast<int>(kMaxCompactSlots) * 2 + 128);
    if (e != cudaSuccess) return e;
    const unsigned grid = static_cast<unsigned>(std::min(std::max<int64_t>(a.layers * per_layer, 1), blocks));
    state_compact_kernel<<<grid, kThreads, smem, s>>>(CompactParams{a, range, per_layer, static_cast<int>(kCompactStage / range),
                                                                  wait_limit(), g_chunked_inject_timeout});
    return cudaGetLastError();
}

}  // namespace wkv
