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
// lengths and their in-place update, is the cluster's own.
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
constexpr int kStepCluster = 1;

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
};

// Sums that stop at 2^31 - 1 instead of wrapping: associative, so they scan.
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, 0x7fffffffu); }

// Last row r of [0, n) with prefix[r] <= x (prefix[0] = 0 <= x).
__device__ __forceinline__ int row_of(const uint32_t *prefix, int n, uint32_t x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__global__ void __launch_bounds__(kStepThreads) build_step_kernel(const StepParams p)
{
    extern __shared__ uint32_t step_smem[];
    const int S = p.num_seqs, B = p.block_size;
    uint32_t *cu = step_smem;           // [S + 1] first token of each row
    uint32_t *pop = cu + S + 1;         // [S + 1] first pop of each row
    uint32_t *gone = pop + S + 1;       // [S + 1] first given-back block of each row
    int *len = reinterpret_cast<int *>(gone + S + 1);  // [S] cached tokens
    __shared__ uint32_t sums[3][kStepThreads / 32];
    __shared__ int s_rows;
    __shared__ uint32_t s_tokens, s_pops;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long long max_len = (long long)p.max_blocks_per_seq * B;
    if (tid == 0) {
        s_rows = 0;
        s_tokens = s_pops = 0u;
    }

    // 1. Each thread's rows [s0, s1): tokens wanted, blocks needed, blocks
    // given back, and their exclusive prefixes over the batch.
    const int per = (S + kStepThreads - 1) / kStepThreads;
    const int s0 = min(S, tid * per), s1 = min(S, s0 + per);
    auto row = [&](int s, int L, int q, uint32_t &want, uint32_t &need, uint32_t &back, bool flag) {
        want = need = back = 0u;
        if (L < 0 || L > max_len || (q > 0 && L + (long long)q > max_len)) {
            if (flag)
                step_raise(PA_DEVERR_SEQ_LEN);  // an inconsistent row gets nothing and gives nothing
            return;
        }
        const uint32_t held = ((uint32_t)L + B - 1) / B;
        if (q > 0) {
            want = (uint32_t)q;
            need = ((uint32_t)L + (uint32_t)q + B - 1) / B - held;
        } else if (q < 0) {
            back = held;
        }
    };
    uint32_t t_sum = 0u, n_sum = 0u, b_sum = 0u;
    for (int s = s0; s < s1; ++s) {
        const int L = p.seq_lens[s], q = p.query_lens[s];
        uint32_t want, need, back;
        row(s, L, q, want, need, back, cluster_rank() == 0);
        len[s] = L;
        cu[s] = want;
        pop[s] = need;
        gone[s] = back;
        t_sum = sat_add(t_sum, want);
        n_sum = sat_add(n_sum, need);
        b_sum = sat_add(b_sum, back);
    }
    uint32_t t_inc = t_sum, n_inc = n_sum, b_inc = b_sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t a = __shfl_up_sync(kFull, t_inc, o), b = __shfl_up_sync(kFull, n_inc, o),
                       c = __shfl_up_sync(kFull, b_inc, o);
        if (lane >= o) {
            t_inc = sat_add(t_inc, a);
            n_inc = sat_add(n_inc, b);
            b_inc = sat_add(b_inc, c);
        }
    }
    if (lane == 31) {
        sums[0][warp] = t_inc;
        sums[1][warp] = n_inc;
        sums[2][warp] = b_inc;
    }
    // Exclusive within the warp.
    t_inc = __shfl_up_sync(kFull, t_inc, 1);
    n_inc = __shfl_up_sync(kFull, n_inc, 1);
    b_inc = __shfl_up_sync(kFull, b_inc, 1);
    if (lane == 0)
        t_inc = n_inc = b_inc = 0u;
    int n_free = *p.num_free;
    cluster_arrive();  // this thread has read the lengths and the free count
    __syncthreads();
    uint32_t t_off = 0u, n_off = 0u, b_off = 0u, b_all = 0u;
    for (int w = 0; w < kStepThreads / 32; ++w) {
        if (w < warp) {
            t_off = sat_add(t_off, sums[0][w]);
            n_off = sat_add(n_off, sums[1][w]);
            b_off = sat_add(b_off, sums[2][w]);
        }
        b_all = sat_add(b_all, sums[2][w]);
    }
    if (n_free < 0 || n_free > p.num_blocks || (long long)n_free + b_all > p.num_blocks) {
        // More free blocks than the pool has: keep what fits.
        if (tid == 0 && cluster_rank() == 0)
            step_raise(PA_DEVERR_BLOCK_ID);
        n_free = max(0, min(n_free, p.num_blocks));
    }
    const uint32_t back_all = min(b_all, (uint32_t)(p.num_blocks - n_free));
    const uint32_t avail = (uint32_t)n_free + back_all;  // blocks on the stack

    // 2. Rows are served in order while their blocks and tokens fit.
    {
        uint32_t t = sat_add(t_off, t_inc), n = sat_add(n_off, n_inc), b = sat_add(b_off, b_inc);
        int rows = 0;
        uint32_t t_last = 0u, n_last = 0u;
        for (int s = s0; s < s1; ++s) {
            const uint32_t want = cu[s], need = pop[s], back = gone[s];
            cu[s] = t;
            pop[s] = n;
            gone[s] = b;
            t = sat_add(t, want);
            n = sat_add(n, need);
            b = sat_add(b, back);
            if (n <= avail && t <= (uint32_t)p.token_capacity) {
                ++rows;
                t_last = t;
                n_last = n;
            }
        }
        if (rows) {
            atomicAdd(&s_rows, rows);
            atomicMax(&s_tokens, t_last);
            atomicMax(&s_pops, n_last);
        }
    }
    __syncthreads();
    const int rows = s_rows;                    // rows served: 0 .. rows - 1
    const uint32_t tokens = s_tokens, pops = s_pops;
    for (int s = rows + tid; s <= S; s += kStepThreads) {  // the others take none
        cu[s] = tokens;
        pop[s] = pops;
    }
    if (tid == 0)
        gone[S] = b_all;
    __syncthreads();

    // Pop i of the stack (checked on use).
    auto popped = [&](uint32_t i) -> int {
        const uint32_t at = avail - 1u - i;
        if (at < (uint32_t)n_free)
            return p.free_list[at];
        const uint32_t k = at - (uint32_t)n_free;
        const int s = row_of(gone, S, k);
        return p.block_tables[(long long)s * p.max_blocks_per_seq + (gone[s + 1] - 1u - k)];
    };

    // 3. New table entries.
    const int step = (int)gridDim.x * kStepThreads, me = (int)cluster_rank() * kStepThreads + tid;
    for (uint32_t i = me; i < pops; i += step) {
        const int s = row_of(pop, S, i);
        const uint32_t held = ((uint32_t)len[s] + B - 1) / B;
        const int id = popped(i);
        if ((unsigned)id >= (unsigned)p.num_blocks)
            step_raise(PA_DEVERR_BLOCK_ID);
        p.block_tables[(long long)s * p.max_blocks_per_seq + held + (i - pop[s])] = id;
    }
    // 4. Positions and slots, -1 behind the last token.
    for (int t = me; t < p.token_capacity; t += step) {
        int pos = 0, slot = -1;
        if ((uint32_t)t < tokens) {
            const int s = row_of(cu, S, (uint32_t)t);
            pos = len[s] + (int)((uint32_t)t - cu[s]);
            const uint32_t held = ((uint32_t)len[s] + B - 1) / B, j = (uint32_t)pos / B;
            const int id = j < held ? p.block_tables[(long long)s * p.max_blocks_per_seq + j] : popped(pop[s] + (j - held));
            if ((unsigned)id < (unsigned)p.num_blocks)
                slot = id * B + (pos - (int)j * B);
            else
                step_raise(PA_DEVERR_BLOCK_ID);
        }
        if (p.positions)
            p.positions[t] = pos;
        p.slot_mapping[t] = slot;
    }
    // 5. Given-back blocks that no row took stay on the free list.
    const uint32_t left = avail - pops;
    for (uint32_t i = (uint32_t)n_free + me; i < left; i += step)
        p.free_list[i] = popped(avail - 1u - i);

    // 6. Lengths, offsets, counts: after every CTA has read the old ones.
    cluster_wait();
    for (int s = me; s < S; s += step) {
        const uint32_t took = cu[s + 1] - cu[s];
        const bool retired = gone[s + 1] != gone[s];
        p.seq_lens_out[s] = retired ? 0 : len[s] + (int)took;
    }
    for (int s = me; s <= S; s += step)
        p.cu_seqlens_q[s] = (int32_t)cu[s];
    if (me == 0) {
        *p.num_free_out = (int32_t)left;
        *p.num_admitted = rows;
    }
}

size_t step_smem_bytes(int num_seqs) { return ((size_t)num_seqs * 4 + 3) * sizeof(uint32_t); }

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
                   num_blocks,   block_size};
    const void *fn = reinterpret_cast<const void *>(&build_step_kernel);
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
            e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)step_smem_bytes(kStepMaxSeqs));
            if (e != cudaSuccess)
                return set_error(PA_ERR_CUDA, "%s: cudaFuncSetAttribute: %s", who, cudaGetErrorString(e));
            if (dev < 64)
                raised[dev] = true;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kStepCluster);
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
