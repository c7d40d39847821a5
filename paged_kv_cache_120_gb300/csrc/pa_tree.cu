// The speculative step's small operators: a drafted tree's positions and
// masks (pa_build_tree), which of its tokens the target accepts
// (pa_verify_draft), and the accepted tokens' K and V moved into place with
// lengths and blocks brought in line (pa_commit_draft). Attention of the
// tree's tokens is in pa_tree_attention.cu and pa_kernels.cu.
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cstdint>
#include <mutex>

#include "../../include/pa.h"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

__device__ int g_tree_error;  // PA_DEVERR_* bits of this file's kernels

namespace {

constexpr int kMaxSeqs = 4096;
constexpr int kMaxNodes = PA_MAX_TREE_NODES;

__device__ __forceinline__ void tree_raise(int bit) { atomicOr(&g_tree_error, bit); }

// ------------------------------------------------------------- pa_build_tree

// One CTA per sequence. With up(i) a node's parent and M(i) the set {i}, each
// round does M(i) |= M(up(i)) and up(i) = up(up(i)): after r rounds M(i) holds
// the first 2^r nodes on i's way up, so that a single file of n nodes takes
// log2 n rounds instead of n steps. The sets are updated in place: a row that
// another thread has already widened holds ancestors of i all the same. Depths
// add up along the same jumps. A launch and some rounds in shared memory bound
// it, not bandwidth.
__global__ void __launch_bounds__(1024)
    build_tree_kernel(const int32_t *__restrict__ parents, const int32_t *__restrict__ cu_q, const int32_t *__restrict__ seq_lens,
                      int total_q, int words, int32_t *__restrict__ positions, uint32_t *__restrict__ masks)
{
    extern __shared__ uint32_t tree_smem[];
    __shared__ int up[2][kMaxNodes], depth[2][kMaxNodes];
    const int s = blockIdx.x, tid = threadIdx.x, threads = blockDim.x;
    const int q0 = cu_q[s], L = seq_lens[s];
    const long long n64 = (long long)cu_q[s + 1] - q0;
    if (n64 < 0 || n64 > min(kMaxNodes, 32 * words) || q0 < 0 || q0 > total_q - n64 || L < n64) {
        if (tid == 0)
            tree_raise(PA_DEVERR_SEQ_LEN);
        return;
    }
    const int n = (int)n64;
    for (int i = tid; i < n; i += threads) {
        const int a = parents[q0 + i];
        const bool has = a >= 0 && a < i;
        if (!has && a != -1)
            tree_raise(PA_DEVERR_TREE);
        up[0][i] = has ? a : -1;
        depth[0][i] = has ? 1 : 0;
    }
    uint32_t *set = tree_smem;  // [n][words]
    for (int k = tid; k < n * words; k += threads) {
        const int i = k / words, w = k - i * words;
        set[k] = w == i >> 5 ? 1u << (i & 31) : 0u;
    }
    __syncthreads();
    int cur = 0;
    for (int reach = 1; reach < n; reach *= 2) {
        int more = 0;
        for (int k = tid; k < n * words; k += threads) {
            const int i = k / words, w = k - i * words, a = up[cur][i];
            if (a >= 0 && w <= a >> 5)  // ancestors come before their descendants
                set[k] |= set[a * words + w];
        }
        for (int i = tid; i < n; i += threads) {
            const int a = up[cur][i];
            const int b = a >= 0 ? up[cur][a] : -1;
            up[cur ^ 1][i] = b;
            depth[cur ^ 1][i] = depth[cur][i] + (a >= 0 ? depth[cur][a] : 0);
            more |= b >= 0;
        }
        cur ^= 1;
        if (!__syncthreads_or(more))
            break;
    }
    for (int k = tid; k < n * words; k += threads)
        masks[(long long)q0 * words + k] = set[k];
    if (positions)
        for (int i = tid; i < n; i += threads)
            positions[q0 + i] = L - n + depth[cur][i];
}

// ----------------------------------------------------------- pa_verify_draft

// A sum held as an unevaluated pair hi + lo of fp32 numbers (about 46 bits):
// where a draw falls next to a border, 24 bits are too few, and fp64 adds are
// a thirtieth of the fp32 rate here.
struct Sum {
    float hi, lo;
};

// s + (x + e): Knuth's two-sum of the leading parts, the rest into lo.
__device__ __forceinline__ void add(Sum &s, float x, float e)
{
    const float t = s.hi + x, b = t - s.hi;
    s.lo += ((s.hi - (t - b)) + (x - b)) + e;
    s.hi = t;
}

__device__ __forceinline__ double value(const Sum &s) { return (double)s.hi + (double)s.lo; }

// max(p - a q, 0) as a pair, a = ah + al >= 0: the product's and the
// difference's rounding errors are kept. Anything not above 0 (NaN too) is 0.
__device__ __forceinline__ Sum weight(float p, float q, float ah, float al)
{
    const float m = __fmul_rn(ah, q), me = fmaf(ah, q, -m);  // kept apart: no fused p - ah q
    const float d = p - m, b = d - p;
    const float e = ((p - (d - b)) + (-m - b)) - (me + al * q);
    const float hi = d + e;
    if (!(hi > 0.f))
        return Sum{0.f, 0.f};
    return Sum{hi, isinf(hi) ? 0.f : e - (hi - d)};
}

template <typename T>
__device__ __forceinline__ float to_float(T x)
{
    if constexpr (sizeof(T) == 4)
        return x;
    else
        return static_cast<float>(x);
}

// 16 bytes as fp32 values.
template <typename T>
__device__ __forceinline__ void widen(const uint4 &v, float *x)
{
    if constexpr (sizeof(T) == 4) {
        x[0] = __uint_as_float(v.x);
        x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z);
        x[3] = __uint_as_float(v.w);
    } else {
        constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = unpack2<BF16>(w[k]);
            x[2 * k] = f.x;
            x[2 * k + 1] = f.y;
        }
    }
}

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// A 64-bit word of shared memory of CTA `rank` of this cluster, at the address that `p` has here.
__device__ __forceinline__ unsigned long long load_from(const void *p, uint32_t rank)
{
    uint32_t a;
    unsigned long long v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
    return v;
}

struct VerifyParams {
    int32_t *num_accepted, *path, *tokens_out;
    const int32_t *tokens, *parents, *cu_q;
    const void *target, *draft;
    const float *uniforms;
    long long target_stride, draft_stride;
    int total_q, vocab;
};

enum : int { kGreedy = 0, kSample = 1, kDraft = 2 };
constexpr int kVerifyThreads = 256, kVerifyWarps = kVerifyThreads / 32, kMaxCluster = 16;

// A cluster of CTAs takes a sequence down its tree; a row of the target (and
// of the drafter) is read by all of them, a contiguous part per warp, so that
// parts follow one another in the order of the vocabulary.
//
//   greedy: the row's first largest entry y; on to the first child holding y.
//   sample: y drawn from the row; on to the first child holding y (the same
//           law as accepting each child with its probability in what is left).
//   draft:  children were drawn from the drafter's row q. Child x is accepted
//           if u q(x) Z < r(x); r = p, Z = 1 at first, and after each refusal
//           what is left of the target, r = max(r - Z q, 0), Z = sum r. In
//           terms of the row itself r = max(p - A q, 0), A the sum of the Z so
//           far, so that a refusal costs one pass and no row is ever stored.
//           The last refusal is followed by a draw from r.
//   a draw: the first entry whose running sum passes u times the row's sum:
//           sums per warp, exchanged over the cluster, name the warp that
//           holds it, which goes through its part again.
//
// The chain from row to row bounds it (one row has to be read before the next
// is known), then the rows' bytes. Every sum is taken in one order, whatever
// the timing.
template <typename T, int MODE>
__global__ void __launch_bounds__(kVerifyThreads) verify_draft_kernel(const VerifyParams p, int cluster)
{
    constexpr int VEC = 16 / sizeof(T);
    __shared__ int s_parent[kMaxNodes], s_token[kMaxNodes];
    __shared__ float s_p[MODE == kDraft ? kMaxNodes : 1], s_q[MODE == kDraft ? kMaxNodes : 1];
    // Exchanged with the other CTAs; two turns, so that a slot is written
    // again only after a barrier behind its last read.
    __shared__ unsigned long long s_out[2], s_token_out[2];
    __shared__ double s_warp[2][kVerifyWarps];
    __shared__ unsigned long long s_best[kVerifyWarps];
    __shared__ double s_cta[2][kMaxCluster];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int s = blockIdx.x / cluster, rank = (int)cluster_rank();
    const T *target = static_cast<const T *>(p.target), *draft = static_cast<const T *>(p.draft);
    const int q0 = p.cu_q[s], V = p.vocab;
    const long long n64 = (long long)p.cu_q[s + 1] - q0;
    const bool bad = n64 < 0 || n64 > kMaxNodes || q0 < 0 || q0 > p.total_q - n64;
    if (bad || n64 == 0) {  // the whole cluster leaves here
        if (rank == 0 && tid == 0) {
            if (bad)
                tree_raise(PA_DEVERR_SEQ_LEN);
            p.num_accepted[s] = 0;
        }
        return;
    }
    const int n = (int)n64;
    for (int i = tid; i < n; i += kVerifyThreads) {
        const int a = p.parents[q0 + i], x = p.tokens[q0 + i];
        const bool has = a >= 0 && a < i;
        if (!has && a != -1 && rank == 0)
            tree_raise(PA_DEVERR_TREE);
        s_parent[i] = has ? a : -1;
        s_token[i] = x;
        if constexpr (MODE == kDraft) {
            // The two numbers that decide on this node as a first child.
            const bool in = has && (unsigned)x < (unsigned)V;
            s_p[i] = in ? to_float(target[(q0 + a) * p.target_stride + x]) : 0.f;
            s_q[i] = in ? to_float(draft[(q0 + a) * p.draft_stride + x]) : 0.f;
        }
        if (rank == 0) {
            p.path[q0 + i] = -1;
            p.tokens_out[q0 + i] = -1;
        }
    }
    __syncthreads();

    // First child of `node` behind node `after`; n if none. Every warp for itself.
    auto child_of = [&](int node, int after) {
        for (int i0 = after + 1; i0 < n; i0 += 32) {
            const unsigned hit = __ballot_sync(kFull, i0 + lane < n && s_parent[i0 + lane] == node);
            if (hit)
                return i0 + __ffs(hit) - 1;
        }
        return n;
    };

    // This warp's part of a row: 16-byte vectors [v0, v1) counted from the
    // aligned address at or below the row's first element, `mis` elements
    // before it.
    const int part = rank * kVerifyWarps + warp, parts = cluster * kVerifyWarps;
    struct Row {
        const T *p, *q;
        int mis, v0, v1;
        bool q_vec;  // the drafter's row lies like the target's
    };
    auto row_at = [&](int node) {
        Row r;
        r.p = target + (q0 + node) * p.target_stride;
        r.q = MODE == kDraft ? draft + (q0 + node) * p.draft_stride : nullptr;
        r.mis = (int)((reinterpret_cast<uintptr_t>(r.p) & 15) / sizeof(T));
        r.q_vec = MODE == kDraft && ((reinterpret_cast<uintptr_t>(r.p) ^ reinterpret_cast<uintptr_t>(r.q)) & 15) == 0;
        const long long vecs = ((long long)V + r.mis + VEC - 1) / VEC;
        r.v0 = (int)(vecs * part / parts);
        r.v1 = (int)(vecs * (part + 1) / parts);
        return r;
    };
    // The VEC elements of vector v of a row, 0 outside it.
    auto load = [&](const T *row, int mis, int v, bool vec, float *x) {
        const int i0 = v * VEC - mis;
        if (vec && i0 >= 0 && i0 + VEC <= V) {
            widen<T>(__ldg(reinterpret_cast<const uint4 *>(row + i0)), x);
        } else {
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                x[k] = i0 + k >= 0 && i0 + k < V ? to_float(row[i0 + k]) : 0.f;
        }
    };
    // Vector v's weights.
    auto weights = [&](const Row &r, int v, float ah, float al, Sum *w) {
        float x[VEC], y[VEC];
        load(r.p, r.mis, v, true, x);
        if (MODE == kDraft && ah != 0.f) {
            load(r.q, r.mis, v, r.q_vec, y);
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                w[k] = weight(x[k], y[k], ah, al);
        } else {
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                w[k] = Sum{x[k] > 0.f ? x[k] : 0.f, 0.f};
        }
    };
    auto warp_sum = [&](Sum t) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            add(t, __shfl_xor_sync(kFull, t.hi, o), __shfl_xor_sync(kFull, t.lo, o));
        return value(Sum{__shfl_sync(kFull, t.hi, 0), __shfl_sync(kFull, t.lo, 0)});
    };
    int turn = 0;
    // Every CTA's word, gathered: s_cta[turn][c] and the sum of all, in the
    // order of the parts. Leaves the warps' own sums in s_warp[turn].
    auto total_of = [&](const Row &r, double a) {
        const float ah = (float)a, al = (float)(a - (double)ah);
        Sum t = {0.f, 0.f};
#pragma unroll 4
        for (int v = r.v0 + lane; v < r.v1; v += 32) {
            Sum w[VEC];
            weights(r, v, ah, al, w);
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                add(t, w[k].hi, w[k].lo);
        }
        const double mine = warp_sum(t);
        turn ^= 1;
        if (lane == 0)
            s_warp[turn][warp] = mine;
        __syncthreads();
        if (tid == 0) {
            double c = 0.0;
            for (int w = 0; w < kVerifyWarps; ++w)
                c += s_warp[turn][w];
            s_out[turn] = (unsigned long long)__double_as_longlong(c);
        }
        cluster_barrier();
        if (tid < cluster)
            s_cta[turn][tid] = __longlong_as_double((long long)load_from(&s_out[turn], tid));
        __syncthreads();
        double z = 0.0;
        for (int c = 0; c < cluster; ++c)
            z += s_cta[turn][c];
        return z;
    };
    // A token drawn from max(p - a q, 0), whose sum z total_of has just left
    // behind. Every CTA gets it.
    auto draw = [&](const Row &r, double a, double z, float u) {
        const double t = (double)u * z;
        // The last CTA and warp with a positive sum takes what rounding leaves over.
        double before = 0.0;
        int owner = -1, last = -1;
        for (int c = 0; c < cluster; ++c) {
            const double x = s_cta[turn][c];
            if (x > 0.0) {
                last = c;
                if (owner < 0 && before + x > t)
                    owner = c;
            }
            if (owner < 0)
                before += x;
        }
        const bool over = owner < 0;
        if (over)
            owner = last;
        if (owner == rank) {
            if (over)
                before = -DBL_MAX;
            int w_owner = -1, w_last = -1;
            double w_before = before;
            for (int w = 0; w < kVerifyWarps; ++w) {
                const double x = s_warp[turn][w];
                if (x > 0.0) {
                    w_last = w;
                    if (w_owner < 0 && w_before + x > t)
                        w_owner = w;
                }
                if (w_owner < 0)
                    w_before += x;
            }
            if (w_owner < 0) {  // rounding: the last part's last positive entry
                w_owner = w_last;
                w_before = -DBL_MAX;
            }
            if (warp == w_owner) {
                const float ah = (float)a, al = (float)(a - (double)ah);
                double run = w_before;
                int found = -1, positive = -1;
                for (int v0 = r.v0; v0 < r.v1 && found < 0; v0 += 32) {
                    const int v = v0 + lane;
                    Sum w[VEC], mine = {0.f, 0.f};
                    if (v < r.v1)
                        weights(r, v, ah, al, w);
#pragma unroll
                    for (int k = 0; k < VEC; ++k) {
                        if (v >= r.v1)
                            w[k] = Sum{0.f, 0.f};
                        add(mine, w[k].hi, w[k].lo);
                    }
                    Sum incl = mine;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const float h = __shfl_up_sync(kFull, incl.hi, o), l = __shfl_up_sync(kFull, incl.lo, o);
                        if (lane >= o)
                            add(incl, h, l);
                    }
                    const float eh = __shfl_up_sync(kFull, incl.hi, 1), el = __shfl_up_sync(kFull, incl.lo, 1);
                    Sum at = lane ? Sum{eh, el} : Sum{0.f, 0.f};
                    int here = -1;
#pragma unroll
                    for (int k = 0; k < VEC; ++k) {
                        if (w[k].hi > 0.f) {
                            add(at, w[k].hi, w[k].lo);
                            positive = v * VEC + k - r.mis;
                            if (here < 0 && run + value(at) > t)
                                here = positive;
                        }
                    }
                    const unsigned hit = __ballot_sync(kFull, here >= 0);
                    if (hit)
                        found = __shfl_sync(kFull, here, __ffs(hit) - 1);
                    run += value(Sum{__shfl_sync(kFull, incl.hi, 31), __shfl_sync(kFull, incl.lo, 31)});
                }
                positive = __reduce_max_sync(kFull, positive);
                if (lane == 0)
                    s_token_out[turn] = (unsigned long long)(found >= 0 ? found : max(positive, 0));
            }
        }
        cluster_barrier();
        return (int)load_from(&s_token_out[turn], owner < 0 ? 0 : owner);
    };
    // The row's first largest entry, NaN passed over.
    auto largest = [&](const Row &r) {
        float best = -INFINITY;
        int at = 0x7fffffff;
#pragma unroll 4
        for (int v = r.v0 + lane; v < r.v1; v += 32) {
            float x[VEC];
            load(r.p, r.mis, v, true, x);
            const int i0 = v * VEC - r.mis;
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                if (i0 + k >= 0 && i0 + k < V && x[k] > best) {
                    best = x[k];
                    at = i0 + k;
                }
        }
        // Ordered as whole numbers: the larger value first, then the lower index.
        const uint32_t b = __float_as_uint(best + 0.f);
        const uint32_t up = b & 0x80000000u ? ~b : b | 0x80000000u;
        unsigned long long key = (unsigned long long)up << 32 | (0x7fffffffu - (unsigned)at);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            key = max(key, __shfl_xor_sync(kFull, key, o));
        turn ^= 1;
        if (lane == 0)
            s_best[warp] = key;
        __syncthreads();
        if (tid == 0) {
            for (int w = 0; w < kVerifyWarps; ++w)
                key = max(key, s_best[w]);
            s_out[turn] = key;
        }
        cluster_barrier();
        key = 0ull;
        for (int c = 0; c < cluster; ++c)
            key = max(key, load_from(&s_out[turn], c));
        const int i = (int)(0x7fffffffu - (uint32_t)key);
        return i < V ? i : 0;
    };

    int node = 0;
    for (int k = 0; k < n; ++k) {  // each step goes to a later node
        int next = n, token = 0;
        double a = 0.0, z = 1.0;  // draft: see above
        const Row r = row_at(node);
        if constexpr (MODE == kDraft) {
            for (int kid = child_of(node, node); kid < n;) {
                double rx = s_p[kid];
                const double qx = s_q[kid];
                if (a > 0.0)
                    rx = fmax(rx - a * qx, 0.0);
                if ((double)p.uniforms[2 * (q0 + kid)] * qx * z < rx) {
                    next = kid;
                    break;
                }
                a += z;
                kid = child_of(node, kid);
                if (kid < n)
                    z = total_of(r, a);
            }
        }
        if (next == n) {
            if constexpr (MODE == kGreedy) {
                token = largest(r);
            } else {
                z = total_of(r, a);
                if (!(z > 0.0 && z <= DBL_MAX) && a > 0.0) {
                    a = 0.0;  // nothing is left of the row: the target's own
                    z = total_of(r, a);
                }
                if (z > 0.0 && z <= DBL_MAX)
                    token = draw(r, a, z, p.uniforms[2 * (q0 + node) + 1]);
                else if (rank == 0 && tid == 0)
                    tree_raise(PA_DEVERR_TREE);
            }
            if constexpr (MODE != kDraft) {
                next = child_of(node, node);
                while (next < n && s_token[next] != token)
                    next = child_of(node, next);
            }
        }
        if (rank == 0 && tid == 0) {
            p.path[q0 + k] = node;
            p.tokens_out[q0 + k] = next < n ? s_token[next] : token;
            if (next == n)
                p.num_accepted[s] = k + 1;
        }
        if (next == n)
            break;
        node = next;
    }
    cluster_barrier();  // nobody leaves while its shared memory may be read
}

// ----------------------------------------------------------- pa_commit_draft

constexpr int kMaxLayers = 512;
struct CommitLayers {
    uint4 *p[kMaxLayers];
};

struct CommitParams {
    const int32_t *block_tables, *cu_q, *seq_lens, *num_accepted, *path;
    int32_t *seq_lens_out, *free_list;
    const int32_t *num_free;
    int32_t *num_free_out;
    int max_blocks_per_seq, num_seqs, total_q, num_layers, num_blocks, block_size;
    int row_vecs;         // 16-byte vectors of a token's K (or V) row
    long long half_vecs;  // of a pool's K half
};

// A sequence's node count (0: idle) and accepted nodes; false if they or its length are inconsistent.
__device__ __forceinline__ bool commit_row(const CommitParams &p, int s, int &q0, int &n, int &k, int &L)
{
    q0 = p.cu_q[s];
    const long long n64 = (long long)p.cu_q[s + 1] - q0;
    L = p.seq_lens[s];
    k = p.num_accepted[s];
    n = (int)n64;
    return n64 >= 0 && n64 <= kMaxNodes && q0 >= 0 && q0 <= p.total_q - n64 && L >= n64 &&
           L <= (long long)p.max_blocks_per_seq * p.block_size && (n == 0 || (k >= 0 && k <= n));
}

constexpr int kMoveThreads = 256, kMoveBatch = 8;

// Moves: a thread takes one 16-byte column of one layer's K or V rows and all
// of a sequence's accepted tokens, in ascending order, kMoveBatch of them read
// before the first is written. Token path[j] >= j goes to place j, so a write
// never reaches a row that a later batch still reads, and no other thread
// touches the column: no copy in between, no barrier. HBM bounds it.
__global__ void __launch_bounds__(kMoveThreads) commit_move_kernel(const __grid_constant__ CommitLayers layers, const CommitParams p)
{
    __shared__ long long s_from[kMaxNodes], s_to[kMaxNodes];
    grid_launch_dependents();  // the bookkeeping runs beside the moves
    const int tid = threadIdx.x;
    const int s = blockIdx.y;
    int q0, n, k, L;
    if (!commit_row(p, s, q0, n, k, L)) {
        if (blockIdx.x == 0 && tid == 0)
            tree_raise(PA_DEVERR_SEQ_LEN);
        return;
    }
    if (n == 0)
        return;
    int wrong = 0;
    for (int j = tid; j < k; j += kMoveThreads) {
        const int at = p.path[q0 + j];
        if (at < j || at >= n || (j > 0 && p.path[q0 + j - 1] >= at))
            wrong = 1;
        s_to[j] = -1;
        if (at > j && at < n) {
            const int from = L - n + at, to = L - n + j;
            const int32_t *table = p.block_tables + (long long)s * p.max_blocks_per_seq;
            const int fb = table[from / p.block_size], tb = table[to / p.block_size];
            if ((unsigned)fb >= (unsigned)p.num_blocks || (unsigned)tb >= (unsigned)p.num_blocks) {
                if (blockIdx.x == 0)
                    tree_raise(PA_DEVERR_BLOCK_ID);
            } else {
                s_from[j] = ((long long)fb * p.block_size + from % p.block_size) * p.row_vecs;
                s_to[j] = ((long long)tb * p.block_size + to % p.block_size) * p.row_vecs;
            }
        }
    }
    if (__syncthreads_or(wrong)) {
        if (blockIdx.x == 0 && tid == 0)
            tree_raise(PA_DEVERR_TREE);
        return;
    }
    const long long columns = 2LL * p.num_layers * p.row_vecs;
    const long long c = (long long)blockIdx.x * kMoveThreads + tid;
    if (c >= columns)
        return;
    const int lk = (int)(c / p.row_vecs), v = (int)(c - (long long)lk * p.row_vecs);
    uint4 *col = layers.p[lk >> 1] + (lk & 1) * p.half_vecs + v;
    for (int j0 = 0; j0 < k; j0 += kMoveBatch) {
        uint4 x[kMoveBatch];
#pragma unroll
        for (int b = 0; b < kMoveBatch; ++b)
            if (j0 + b < k && s_to[j0 + b] >= 0)
                x[b] = col[s_from[j0 + b]];
#pragma unroll
        for (int b = 0; b < kMoveBatch; ++b)
            if (j0 + b < k && s_to[j0 + b] >= 0)
                col[s_to[j0 + b]] = x[b];
    }
}

constexpr int kBookThreads = 1024, kBookRows = kMaxSeqs / kBookThreads;

// Bookkeeping, one CTA beside the moves: new lengths, and the blocks behind
// them back onto the free list, row after row, a row's last block first (an
// exclusive prefix of the rows' surplus blocks gives each its place). Reads
// what the moves read and writes only when they are done: lengths and count
// may be updated in place.
__global__ void __launch_bounds__(kBookThreads) commit_book_kernel(const CommitParams p)
{
    __shared__ int sums[kBookThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int after[kBookRows], held[kBookRows], gone[kBookRows], sum = 0;
    const int n_in = p.free_list ? *p.num_free : 0;
#pragma unroll
    for (int r = 0; r < kBookRows; ++r) {
        const int s = tid * kBookRows + r;
        after[r] = held[r] = gone[r] = 0;
        if (s >= p.num_seqs)
            continue;
        int q0, n, k, L;
        bool ok = commit_row(p, s, q0, n, k, L);
        if (ok && n > 0) {
            int prev = -1;
            for (int j = 0; j < k; ++j) {
                const int at = p.path[q0 + j];
                ok = ok && at > prev && at < n;
                prev = at;
            }
        }
        after[r] = L;
        if (ok && n > 0) {  // flagged by the moves if not
            after[r] = L - n + k;
            held[r] = (L + p.block_size - 1) / p.block_size;
            gone[r] = p.free_list ? held[r] - (after[r] + p.block_size - 1) / p.block_size : 0;
        }
        sum += gone[r];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kFull, incl, o);
        if (lane >= o)
            incl += v;
    }
    if (lane == 31)
        sums[warp] = incl;
    __syncthreads();
    int off = 0, all = 0;
    for (int w = 0; w < kBookThreads / 32; ++w) {
        off += w < warp ? sums[w] : 0;
        all += sums[w];
    }
    int at = off + incl - sum;
    grid_dependency_wait();  // the moves have read the lengths and the count
    const int base = max(0, min(n_in, p.num_blocks));
    if (tid == 0 && p.free_list) {
        if (n_in != base || all > p.num_blocks - base)
            tree_raise(PA_DEVERR_BLOCK_ID);
        *p.num_free_out = base + min(all, p.num_blocks - base);
    }
#pragma unroll
    for (int r = 0; r < kBookRows; ++r) {
        const int s = tid * kBookRows + r;
        if (s >= p.num_seqs)
            continue;
        p.seq_lens_out[s] = after[r];
        for (int i = 0; i < gone[r]; ++i, ++at) {
            const int id = p.block_tables[(long long)s * p.max_blocks_per_seq + held[r] - 1 - i];
            if ((unsigned)id >= (unsigned)p.num_blocks)
                tree_raise(PA_DEVERR_BLOCK_ID);
            if (at < p.num_blocks - base)
                p.free_list[base + at] = id;
        }
    }
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace

int tree_take_device_error(int *bits)
{
    int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_tree_error, sizeof(int));
    if (e == cudaSuccess)
        e = cudaMemcpyToSymbol(g_tree_error, &zero, sizeof(int));
    *bits = e == cudaSuccess ? v : 0;
    return (int)e;
}

}  // namespace pa

using namespace pa;

namespace {

// Attributes of the verify kernels and of pa_build_tree's, set once per
// device, so that a call being captured into a CUDA graph makes no such call;
// the SM count with them.
template <typename T>
const void *verify_fn(int mode)
{
    switch (mode) {
    case kGreedy:
        return reinterpret_cast<const void *>(&verify_draft_kernel<T, kGreedy>);
    case kSample:
        return reinterpret_cast<const void *>(&verify_draft_kernel<T, kSample>);
    default:
        return reinterpret_cast<const void *>(&verify_draft_kernel<T, kDraft>);
    }
}

const void *verify_kernel(int dtype, int mode)
{
    return dtype == PA_F32 ? verify_fn<float>(mode) : dtype == PA_BF16 ? verify_fn<__nv_bfloat16>(mode) : verify_fn<__half>(mode);
}

int tree_setup(const char *who, int *sms_out)
{
    static std::mutex mu;
    static int sm_count[64] = {};
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return set_error(PA_ERR_CUDA, "%s: cudaGetDevice: %s", who, cudaGetErrorString(e));
    std::lock_guard<std::mutex> lock(mu);
    sms = dev < 64 ? sm_count[dev] : 0;
    if (sms == 0) {
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        for (int dtype : {PA_F16, PA_BF16, PA_F32})
            for (int mode = kGreedy; mode <= kDraft && e == cudaSuccess; ++mode)
                e = cudaFuncSetAttribute(verify_kernel(dtype, mode), cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(reinterpret_cast<const void *>(&build_tree_kernel),
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxNodes / 32 * kMaxNodes * 4);
        if (e != cudaSuccess)
            return set_error(PA_ERR_CUDA, "%s: kernel attributes: %s", who, cudaGetErrorString(e));
        if (dev < 64)
            sm_count[dev] = sms;
    }
    *sms_out = sms;
    return PA_OK;
}

}  // namespace

extern "C" int pa_build_tree(const int32_t *parents, const int32_t *cu_seqlens_q, const int32_t *seq_lens, int num_seqs,
                             int total_q, int32_t *positions, int32_t *tree_masks, int mask_words, pa_stream_t stream)
{
    const char *who = "pa_build_tree";
    if (num_seqs < 0 || num_seqs > kMaxSeqs || total_q < 0)
        return set_error(PA_ERR_INVALID_ARG, "%s: num_seqs %d outside [0, %d] or total_q %d", who, num_seqs, kMaxSeqs, total_q);
    if (mask_words < 1 || mask_words > kMaxNodes / 32)
        return set_error(PA_ERR_INVALID_ARG, "%s: mask_words %d outside [1, %d]", who, mask_words, kMaxNodes / 32);
    if (num_seqs == 0 || total_q == 0)
        return PA_OK;
    if (!parents || !cu_seqlens_q || !seq_lens || !tree_masks)
        return set_error(PA_ERR_INVALID_ARG, "%s: null pointer argument", who);
    if (!aligned(parents, 4) || !aligned(cu_seqlens_q, 4) || !aligned(seq_lens, 4) || !aligned(positions, 4) || !aligned(tree_masks, 4))
        return set_error(PA_ERR_INVALID_ARG, "%s: misaligned pointer (4 B)", who);
    int sms = 0;
    const int rc = tree_setup(who, &sms);
    if (rc != PA_OK)
        return rc;
    // A thread per word of the largest tree's masks, up to a full CTA.
    const int threads = std::max(64, std::min(1024, 32 * mask_words * mask_words));
    build_tree_kernel<<<num_seqs, threads, (size_t)32 * mask_words * mask_words * 4, reinterpret_cast<cudaStream_t>(stream)>>>(
        parents, cu_seqlens_q, seq_lens, total_q, mask_words, positions, reinterpret_cast<uint32_t *>(tree_masks));
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return set_error(PA_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
    return PA_OK;
}

extern "C" int pa_verify_draft(int32_t *num_accepted, int32_t *path, int32_t *tokens_out, const int32_t *tokens,
                               const int32_t *parents, const int32_t *cu_seqlens_q, int num_seqs, int total_q,
                               const void *target, int64_t target_stride, const void *draft, int64_t draft_stride,
                               int vocab_size, int dtype, const float *uniforms, pa_stream_t stream)
{
    const char *who = "pa_verify_draft";
    if (dtype != PA_F16 && dtype != PA_BF16 && dtype != PA_F32)
        return set_error(PA_ERR_UNSUPPORTED, "%s: dtype %d (want PA_F16, PA_BF16 or PA_F32)", who, dtype);
    if (num_seqs < 0 || num_seqs > kMaxSeqs || total_q < 0)
        return set_error(PA_ERR_INVALID_ARG, "%s: num_seqs %d outside [0, %d] or total_q %d", who, num_seqs, kMaxSeqs, total_q);
    if (vocab_size < 1 || vocab_size > (1 << 30) || target_stride < vocab_size || (draft && draft_stride < vocab_size))
        return set_error(PA_ERR_INVALID_ARG, "%s: vocab_size %d outside [1, 2^30], or a row stride below it", who, vocab_size);
    if (draft && !uniforms)
        return set_error(PA_ERR_INVALID_ARG, "%s: draft rows without random numbers (greedy verification takes none)", who);
    if (num_seqs == 0)
        return PA_OK;
    if (!num_accepted || !cu_seqlens_q || (total_q > 0 && (!path || !tokens_out || !tokens || !parents || !target)))
        return set_error(PA_ERR_INVALID_ARG, "%s: null pointer argument", who);
    const size_t elem = dtype == PA_F32 ? 4 : 2;
    if (!aligned(num_accepted, 4) || !aligned(path, 4) || !aligned(tokens_out, 4) || !aligned(tokens, 4) || !aligned(parents, 4) ||
        !aligned(cu_seqlens_q, 4) || !aligned(uniforms, 4) || !aligned(target, elem) || !aligned(draft, elem))
        return set_error(PA_ERR_INVALID_ARG, "%s: misaligned pointer (4 B, rows their element's size)", who);
    int sms = 0;
    const int rc = tree_setup(who, &sms);
    if (rc != PA_OK)
        return rc;
    // CTAs a sequence: as many as about two an SM allow, of 2048 entries at least.
    int cluster = 1;
    while (cluster < kMaxCluster && (long long)num_seqs * cluster * 2 <= 2 * sms && vocab_size >= 2048 * cluster * 2)
        cluster *= 2;
    VerifyParams prm{num_accepted, path, tokens_out, tokens, parents, cu_seqlens_q, target, draft,
                     uniforms, target_stride, draft_stride, total_q, vocab_size};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_seqs * cluster);
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *args[] = {&prm, &cluster};
    const cudaError_t e = cudaLaunchKernelExC(&cfg, verify_kernel(dtype, !uniforms ? kGreedy : draft ? kDraft : kSample), args);
    if (e != cudaSuccess)
        return set_error(PA_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
    return PA_OK;
}

extern "C" int pa_commit_draft(void *const *kv_caches, int num_layers, const int32_t *block_tables, int max_blocks_per_seq,
                               const int32_t *cu_seqlens_q, const int32_t *seq_lens, const int32_t *num_accepted,
                               const int32_t *path, int num_seqs, int total_q, int32_t *seq_lens_out, int32_t *free_list,
                               const int32_t *num_free, int32_t *num_free_out, int num_blocks, int block_size,
                               int num_kv_heads, int head_size, int dtype, pa_stream_t stream)
{
    const char *who = "pa_commit_draft";
    if (dtype != PA_F16 && dtype != PA_BF16 && dtype != PA_FP8_E4M3)
        return set_error(PA_ERR_UNSUPPORTED, "%s: dtype %d", who, dtype);
    if (num_seqs < 0 || num_seqs > kMaxSeqs || total_q < 0 || num_layers < 1 || num_layers > kMaxLayers || num_blocks <= 0 ||
        max_blocks_per_seq <= 0 || block_size < 16 || block_size % 16 != 0 || num_kv_heads <= 0 || head_size <= 0)
        return set_error(PA_ERR_INVALID_ARG, "%s: bad sizes (num_seqs <= %d, 1 <= num_layers <= %d, block_size a multiple of 16)",
                         who, kMaxSeqs, kMaxLayers);
    if ((long long)max_blocks_per_seq * block_size > (1LL << 30))
        return set_error(PA_ERR_INVALID_ARG, "%s: max_blocks_per_seq * block_size too large", who);
    const long long row_bytes = (long long)num_kv_heads * head_size * (dtype == PA_FP8_E4M3 ? 1 : 2);
    if (row_bytes % 16 != 0 || row_bytes > (1LL << 31))
        return set_error(PA_ERR_INVALID_ARG, "%s: a token's row (num_kv_heads * head_size elements) must be a multiple of 16 bytes, at most 2^31", who);
    if (num_seqs == 0)
        return PA_OK;
    if (!kv_caches || !block_tables || !cu_seqlens_q || !seq_lens || !num_accepted || (total_q > 0 && !path) || !seq_lens_out ||
        (free_list && (!num_free || !num_free_out)))
        return set_error(PA_ERR_INVALID_ARG, "%s: null pointer argument", who);
    if (!aligned(block_tables, 4) || !aligned(cu_seqlens_q, 4) || !aligned(seq_lens, 4) || !aligned(num_accepted, 4) ||
        !aligned(path, 4) || !aligned(seq_lens_out, 4) || !aligned(free_list, 4) || !aligned(num_free, 4) || !aligned(num_free_out, 4))
        return set_error(PA_ERR_INVALID_ARG, "%s: misaligned pointer (4 B)", who);
    CommitLayers layers;
    for (int l = 0; l < num_layers; ++l) {
        if (!kv_caches[l] || !aligned(kv_caches[l], 16))
            return set_error(PA_ERR_INVALID_ARG, "%s: layer %d pool null or misaligned", who, l);
        layers.p[l] = static_cast<uint4 *>(kv_caches[l]);
    }
    for (int l = num_layers; l < kMaxLayers; ++l)
        layers.p[l] = nullptr;
    CommitParams prm;
    prm.block_tables = block_tables;
    prm.cu_q = cu_seqlens_q;
    prm.seq_lens = seq_lens;
    prm.num_accepted = num_accepted;
    prm.path = path;
    prm.seq_lens_out = seq_lens_out;
    prm.free_list = free_list;
    prm.num_free = num_free;
    prm.num_free_out = num_free_out;
    prm.max_blocks_per_seq = max_blocks_per_seq;
    prm.num_seqs = num_seqs;
    prm.total_q = total_q;
    prm.num_layers = num_layers;
    prm.num_blocks = num_blocks;
    prm.block_size = block_size;
    prm.row_vecs = (int)(row_bytes / 16);
    prm.half_vecs = (long long)num_blocks * block_size * prm.row_vecs;
    const long long columns = 2LL * num_layers * prm.row_vecs;
    const dim3 grid((unsigned)((columns + kMoveThreads - 1) / kMoveThreads), num_seqs);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    commit_move_kernel<<<grid, kMoveThreads, 0, st>>>(layers, prm);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return set_error(PA_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kBookThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *args[] = {&prm};
    e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void *>(&commit_book_kernel), args);
    if (e != cudaSuccess)
        return set_error(PA_ERR_CUDA, "%s: bookkeeping launch: %s", who, cudaGetErrorString(e));
    return PA_OK;
}
