// pa_build_step: a serving step's block tables, lengths, positions and slots
// built on the GPU from the requests' lengths.
//
// The host allocator's bookkeeping ([book] chapter 4, §4.4.1 block table and
// §4.4.3 slot mapping; "01 · PagedAttention 与 KV cache 块管理" §4.3: freed
// blocks return to the head of the free list) written as prefix sums: with
// b(x) = ceil(x / block_size), row s with L cached and q new tokens takes
// b(L + q) - b(L) blocks, a finished row gives b(L) back, and
//
//   stack  V = free_list[0 .. n), then each finished row's blocks, last first
//   pop i  = V[n + R - 1 - i]          (R blocks given back)
//   row s takes pops P_s .. P_(s+1) - 1 (P: exclusive prefix of the rows' needs)
//   token t of row s: position L + t - cu_s, slot = table[pos / B] * B + pos % B
//
// so every table entry, position and slot follows from the prefixes alone,
// without an order between threads.
//
// The work is a few bytes per row and 8 per token: the launch and a chain of
// dependent loads (lengths -> prefix -> free list -> slot) bound it, not
// bandwidth. One cluster does it in one launch: every CTA scans all rows
// itself (at most 4096 x 8 bytes, from L2), then takes its share of the new
// table entries and tokens; the one barrier, between the last read of the
// lengths and their in-place update, is the cluster's own. Measured (GB300,
// replayed from a graph): 5.3 us for 256 rows of one token, 12.3 us for 4096
// mixed rows and 31000 tokens, 10.3 us for 16 prompts of 160000 tokens; one
// CTA took 5.4, 65 and 118.
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "../../include/pa.h"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

__device__ int g_step_error;  // PA_DEVERR_* bits of pa_build_step

namespace {

constexpr int kStepThreads = 1024;
constexpr int kStepMaxSeqs = 4096;  // the prefixes live in shared memory
constexpr int kStepCluster = 16;  // CTAs, the largest cluster
constexpr int kStepRows = kStepMaxSeqs / kStepThreads;  // consecutive rows of a thread
constexpr int kStepMany = 4;  // tokens of a thread in a round, when there are more than threads

__device__ __forceinline__ void step_raise(int bit) { atomicOr(&g_step_error, bit); }

struct StepParams {
    int32_t *block_tables;
    const int32_t *seq_lens;
    const int32_t *query_lens;
    int32_t *free_list;
    const int32_t *num_free;
    int32_t *seq_lens_out;
    int32_t *num_free_out;
    int32_t *cu_seqlens_q;
    int32_t *positions;     // may be null
    int32_t *slot_mapping;
    int32_t *num_admitted;
    int max_blocks_per_seq, num_seqs, token_capacity, num_blocks, block_size;
    uint32_t div_mul, div_shift;  // x / block_size = umulhi(x, div_mul) >> div_shift for x < 2^31
};

// Sums that stop at 2^31 - 1 instead of wrapping: associative, so they scan.
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, 0x7fffffffu); }

// For each of K values x: the last row r of [lo, n) with prefix[r] <= x
// (prefix[lo] <= x). The K searches run side by side: a step's shared-memory
// loads are in flight together.
template <int K>
__device__ __forceinline__ void rows_of(const uint32_t *prefix, int lo, int n, const uint32_t (&x)[K], int (&row)[K])
{
#pragma unroll
    for (int k = 0; k < K; ++k)
        row[k] = lo;
    for (int half = n - lo > 1 ? 1 << (31 - __clz(n - lo - 1)) : 0; half > 0; half >>= 1) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int at = row[k] + half;
            if (at < n && prefix[at] <= x[k])
                row[k] = at;
        }
    }
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__host__ __device__ inline int step_padded(int num_seqs) { return (num_seqs / kStepRows + 1) * kStepRows; }

// K: tokens a thread handles in a round.
template <int K>
__global__ void __launch_bounds__(kStepThreads) build_step_kernel(const StepParams p)
{
    extern __shared__ __align__(16) uint32_t step_smem[];
    const int S = p.num_seqs, B = p.block_size;
    auto blocks_below = [&](uint32_t x) { return __umulhi(x, p.div_mul) >> p.div_shift; };  // x / B
    auto ceil_blocks = [&](uint32_t x) { return blocks_below(x + (uint32_t)B - 1u); };
    // Per row, and one behind the last; sized for whole threads' rows.
    const int padded = step_padded(S);
    uint32_t *cu = step_smem;          // first token
    uint32_t *pop = cu + padded;       // first pop
    uint32_t *gone = pop + padded;     // first given-back block
    int *len = reinterpret_cast<int *>(gone + padded);  // cached tokens
    __shared__ uint32_t sums[3][kStepThreads / 32];
    __shared__ int s_rows;
    __shared__ uint32_t s_tokens, s_pops;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long long max_len = (long long)p.max_blocks_per_seq * B;
    if (tid == 0) {
        s_rows = 0;
        s_tokens = s_pops = 0u;
    }

    // 1. Each thread's kStepRows rows: tokens wanted, blocks needed, blocks
    // given back. Rows past the batch want nothing.
    struct Sums {
        uint32_t t, n, b;
    };
    const int s0 = tid * kStepRows;
    int L[kStepRows], q[kStepRows];
    int n_free = *p.num_free;
#pragma unroll
    for (int j = 0; j < kStepRows; ++j) {
        L[j] = s0 + j < S ? p.seq_lens[s0 + j] : 0;
        q[j] = s0 + j < S ? p.query_lens[s0 + j] : 0;
    }
    Sums row[kStepRows], sum = {0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < kStepRows; ++j) {
        row[j] = Sums{0u, 0u, 0u};
        if (L[j] < 0 || L[j] > max_len || (q[j] > 0 && L[j] + (long long)q[j] > max_len)) {
            if (cluster_rank() == 0)
                step_raise(PA_DEVERR_SEQ_LEN);  // an inconsistent row gets nothing and gives nothing
        } else if (q[j] > 0) {
            row[j].t = (uint32_t)q[j];
            row[j].n = ceil_blocks((uint32_t)L[j] + (uint32_t)q[j]) - ceil_blocks((uint32_t)L[j]);
        } else if (q[j] < 0) {
            row[j].b = ceil_blocks((uint32_t)L[j]);
        }
        sum = Sums{sat_add(sum.t, row[j].t), sat_add(sum.n, row[j].n), sat_add(sum.b, row[j].b)};
    }
    // Inclusive scan of a triple over the warp.
    auto warp_scan = [&](Sums v) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t t = __shfl_up_sync(kFull, v.t, o), n = __shfl_up_sync(kFull, v.n, o),
                           b = __shfl_up_sync(kFull, v.b, o);
            if (lane >= o)
                v = Sums{sat_add(v.t, t), sat_add(v.n, n), sat_add(v.b, b)};
        }
        return v;
    };
    // The lane before's value, 0 for lane 0: inclusive to exclusive.
    auto before = [&](Sums v) {
        v = Sums{__shfl_up_sync(kFull, v.t, 1), __shfl_up_sync(kFull, v.n, 1), __shfl_up_sync(kFull, v.b, 1)};
        return lane ? v : Sums{0u, 0u, 0u};
    };
    const Sums mine = warp_scan(sum);
    if (lane == 31) {
        sums[0][warp] = mine.t;
        sums[1][warp] = mine.n;
        sums[2][warp] = mine.b;
    }
    cluster_arrive();  // this thread has read the lengths and the free count
    __syncthreads();
    static_assert(kStepThreads == 1024, "one warp scans the 32 warps' sums");
    const Sums all = warp_scan(Sums{sums[0][lane], sums[1][lane], sums[2][lane]});
    const uint32_t b_all = __shfl_sync(kFull, all.b, 31);
    const Sums ahead = before(mine), warps = before(all);
    Sums off = Sums{__shfl_sync(kFull, warps.t, warp), __shfl_sync(kFull, warps.n, warp), __shfl_sync(kFull, warps.b, warp)};
    off = Sums{sat_add(off.t, ahead.t), sat_add(off.n, ahead.n), sat_add(off.b, ahead.b)};
    if (n_free < 0 || n_free > p.num_blocks || (long long)n_free + b_all > p.num_blocks) {
        // More free blocks than the pool has: keep what fits.
        if (tid == 0 && cluster_rank() == 0)
            step_raise(PA_DEVERR_BLOCK_ID);
        n_free = max(0, min(n_free, p.num_blocks));
    }
    const uint32_t back_all = min(b_all, (uint32_t)(p.num_blocks - n_free));
    const uint32_t avail = (uint32_t)n_free + back_all;  // blocks on the stack

    // 2. Rows are served in order while their blocks and tokens fit; the
    // others take none. A row's prefixes go to shared memory.
    {
        int fit = 0;
        uint32_t t_last = 0u, n_last = 0u;
        Sums at[kStepRows];
#pragma unroll
        for (int j = 0; j < kStepRows; ++j) {
            at[j] = off;
            off = Sums{sat_add(off.t, row[j].t), sat_add(off.n, row[j].n), sat_add(off.b, row[j].b)};
            if (s0 + j < S && off.n <= avail && off.t <= (uint32_t)p.token_capacity) {
                ++fit;
                t_last = off.t;
                n_last = off.n;
            }
        }
        if (s0 < padded) {
            static_assert(kStepRows == 4, "a thread's rows are one 16-byte store");
            *reinterpret_cast<uint4 *>(cu + s0) = make_uint4(at[0].t, at[1].t, at[2].t, at[3].t);
            *reinterpret_cast<uint4 *>(pop + s0) = make_uint4(at[0].n, at[1].n, at[2].n, at[3].n);
            *reinterpret_cast<uint4 *>(gone + s0) = make_uint4(at[0].b, at[1].b, at[2].b, at[3].b);
            *reinterpret_cast<int4 *>(len + s0) = make_int4(L[0], L[1], L[2], L[3]);
        }
        if (tid == kStepThreads - 1 && S == kStepMaxSeqs)
            gone[S] = off.b;
        fit = __reduce_add_sync(kFull, fit);
        t_last = __reduce_max_sync(kFull, t_last);
        n_last = __reduce_max_sync(kFull, n_last);
        if (lane == 0 && fit) {
            atomicAdd(&s_rows, fit);
            atomicMax(&s_tokens, t_last);
            atomicMax(&s_pops, n_last);
        }
    }
    __syncthreads();
    const int rows = s_rows;                    // rows served: 0 .. rows - 1
    const uint32_t tokens = s_tokens, pops = s_pops;
    for (int s = rows + tid; s <= S; s += kStepThreads) {
        cu[s] = tokens;
        pop[s] = pops;
    }
    __syncthreads();

    // Pop i of the stack (its id is checked on use).
    auto popped = [&](uint32_t i) -> int {
        const uint32_t at = avail - 1u - i;
        if (at < (uint32_t)n_free)
            return p.free_list[at];
        const uint32_t k[1] = {at - (uint32_t)n_free};
        int s[1];
        rows_of<1>(gone, 0, S, k, s);
        return p.block_tables[(long long)s[0] * p.max_blocks_per_seq + (gone[s[0] + 1] - 1u - k[0])];
    };

    // 3. New table entries.
    const uint32_t step = gridDim.x * kStepThreads, me = cluster_rank() * kStepThreads + tid;
    for (uint32_t i = me; i < pops; i += step) {
        const uint32_t x[1] = {i};
        int s[1];
        rows_of<1>(pop, 0, rows, x, s);
        const int id = popped(i);
        if ((unsigned)id >= (unsigned)p.num_blocks)
            step_raise(PA_DEVERR_BLOCK_ID);
        p.block_tables[(long long)s[0] * p.max_blocks_per_seq + ceil_blocks((uint32_t)len[s[0]]) + (i - pop[s[0]])] = id;
    }
    // 4. Positions and slots, -1 behind the last token: a warp takes chunks of
    // 32 K tokens and looks for their rows between its first and last token's.
    for (uint32_t c0 = (me & ~31u) * K; c0 < (uint32_t)p.token_capacity; c0 += K * step) {
        uint32_t t[K];
        int s[K], pos[K], id[K];
#pragma unroll
        for (int k = 0; k < K; ++k)
            t[k] = c0 + 32u * k + lane;
        if (c0 < tokens) {
            const uint32_t ends[2] = {c0, min(c0 + 32u * K, tokens) - 1u};
            int bound[2];
            rows_of<2>(cu, 0, rows, ends, bound);
            rows_of<K>(cu, bound[0], bound[1] + 1, t, s);
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            pos[k] = 0;
            id[k] = -1;
            if (t[k] < tokens) {
                const uint32_t L = (uint32_t)len[s[k]], x = L + (t[k] - cu[s[k]]);
                const uint32_t held = ceil_blocks(L), j = blocks_below(x);
                pos[k] = (int)x;
                id[k] = j < held ? p.block_tables[(long long)s[k] * p.max_blocks_per_seq + j] : popped(pop[s[k]] + (j - held));
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (t[k] < (uint32_t)p.token_capacity) {
                int slot = -1;
                if ((unsigned)id[k] < (unsigned)p.num_blocks)
                    slot = id[k] * B + (pos[k] - (int)blocks_below((uint32_t)pos[k]) * B);
                else if (t[k] < tokens)
                    step_raise(PA_DEVERR_BLOCK_ID);
                if (p.positions)
                    p.positions[t[k]] = pos[k];
                p.slot_mapping[t[k]] = slot;
            }
    }
    // 5. Given-back blocks that no row took stay on the free list.
    const uint32_t left = avail - pops;
    for (uint32_t i = (uint32_t)n_free + me; i < left; i += step) {
        const int id = popped(avail - 1u - i);
        if ((unsigned)id >= (unsigned)p.num_blocks)
            step_raise(PA_DEVERR_BLOCK_ID);
        p.free_list[i] = id;
    }

    // 6. Lengths, offsets, counts: after every CTA has read the old ones.
    cluster_wait();
    for (int s = me; s < S; s += (int)step) {
        const uint32_t took = cu[s + 1] - cu[s];
        const bool retired = gone[s + 1] != gone[s];
        p.seq_lens_out[s] = retired ? 0 : len[s] + (int)took;
    }
    for (int s = me; s <= S; s += (int)step)
        p.cu_seqlens_q[s] = (int32_t)cu[s];
    if (me == 0) {
        *p.num_free_out = (int32_t)left;
        *p.num_admitted = rows;
    }
}

size_t step_smem_bytes(int num_seqs) { return (size_t)step_padded(num_seqs) * 4 * sizeof(uint32_t); }

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

}  // namespace

int step_take_device_error(int *bits)
{
    int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_step_error, sizeof(int));
    if (e == cudaSuccess)
        e = cudaMemcpyToSymbol(g_step_error, &zero, sizeof(int));
    *bits = e == cudaSuccess ? v : 0;
    return (int)e;
}

}  // namespace pa

using namespace pa;

extern "C" int pa_build_step(int32_t *block_tables, int max_blocks_per_seq, const int32_t *seq_lens,
                             const int32_t *query_lens, int num_seqs, int32_t *free_list, const int32_t *num_free,
                             int32_t *seq_lens_out, int32_t *num_free_out, int32_t *cu_seqlens_q, int32_t *positions,
                             int32_t *slot_mapping, int token_capacity, int32_t *num_admitted, int num_blocks,
                             int block_size, pa_stream_t stream)
{
    const char *who = "pa_build_step";
    if (num_seqs < 0 || num_seqs > kStepMaxSeqs)
        return set_error(PA_ERR_INVALID_ARG, "%s: num_seqs %d outside [0, %d]", who, num_seqs, kStepMaxSeqs);
    if (block_size < 16 || block_size % 16 != 0)
        return set_error(PA_ERR_INVALID_ARG, "%s: block_size %d must be a positive multiple of 16", who, block_size);
    if (num_blocks <= 0 || max_blocks_per_seq <= 0 || token_capacity < 0 || token_capacity > (1 << 30))
        return set_error(PA_ERR_INVALID_ARG, "%s: bad sizes", who);
    if ((long long)max_blocks_per_seq * block_size > (1LL << 30))
        return set_error(PA_ERR_INVALID_ARG, "%s: max_blocks_per_seq * block_size too large", who);
    if ((long long)num_blocks * block_size > 0x7fffffffLL)
        return set_error(PA_ERR_INVALID_ARG, "%s: num_blocks * block_size does not fit an int32 slot", who);
    if (!free_list || !num_free || !num_free_out || !cu_seqlens_q || !num_admitted || (token_capacity > 0 && !slot_mapping) ||
        (num_seqs > 0 && (!block_tables || !seq_lens || !query_lens || !seq_lens_out)))
        return set_error(PA_ERR_INVALID_ARG, "%s: null pointer argument", who);
    if (!aligned4(block_tables) || !aligned4(seq_lens) || !aligned4(query_lens) || !aligned4(free_list) ||
        !aligned4(num_free) || !aligned4(seq_lens_out) || !aligned4(num_free_out) || !aligned4(cu_seqlens_q) ||
        !aligned4(positions) || !aligned4(slot_mapping) || !aligned4(num_admitted))
        return set_error(PA_ERR_INVALID_ARG, "%s: misaligned pointer (4 B)", who);

    StepParams prm{block_tables, seq_lens,  query_lens,   free_list,    num_free,           seq_lens_out, num_free_out,
                   cu_seqlens_q, positions, slot_mapping, num_admitted, max_blocks_per_seq, num_seqs,     token_capacity,
                   num_blocks,   block_size,  0u,           0u};
    // x / B for x < 2^31 as a 32-bit high product and a shift: with k the
    // least 2^k >= B, m = ceil(2^(31 + k) / B) < 2^32 overestimates 1 / B by
    // less than 2^-31 / B in all, too little to reach the next whole number.
    int k = 0;
    while ((1LL << k) < block_size)
        ++k;
    prm.div_mul = (uint32_t)(((1ull << (31 + k)) + (unsigned)block_size - 1) / (unsigned)block_size);
    prm.div_shift = (uint32_t)(k - 1);
    // A token per thread, or with more tokens than threads kStepMany at a time
    // (measured: 4.9 against 6.1 us at 256 tokens, 13.9 against 9.8 at 262144).
    const void *fns[2] = {reinterpret_cast<const void *>(&build_step_kernel<1>),
                          reinterpret_cast<const void *>(&build_step_kernel<kStepMany>)};
    const void *fn = fns[token_capacity > kStepCluster * kStepThreads ? 1 : 0];
    // The largest batch's shared memory is allowed once per device, so that a
    // call being captured into a CUDA graph makes no attribute call.
    static std::mutex mu;
    static bool raised[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return set_error(PA_ERR_CUDA, "%s: cudaGetDevice: %s", who, cudaGetErrorString(e));
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev >= 64 || !raised[dev]) {
            for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
                e = cudaFuncSetAttribute(fns[i], cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)step_smem_bytes(kStepMaxSeqs));
                if (e == cudaSuccess)
                    e = cudaFuncSetAttribute(fns[i], cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            }
            if (e != cudaSuccess)
                return set_error(PA_ERR_CUDA, "%s: cudaFuncSetAttribute: %s", who, cudaGetErrorString(e));
            if (dev < 64)
                raised[dev] = true;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kStepCluster);  // one cluster
    cfg.blockDim = dim3(kStepThreads);
    cfg.dynamicSmemBytes = step_smem_bytes(num_seqs);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kStepCluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *args[] = {&prm};
    e = cudaLaunchKernelExC(&cfg, fn, args);
    if (e != cudaSuccess)
        return set_error(PA_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
    return PA_OK;
}
