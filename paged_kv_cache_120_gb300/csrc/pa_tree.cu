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

// A CTA takes kGroupWords words of a sequence's masks, blocks of 32 nodes in
// turn. Within a block a warp finds each node's topmost ancestor there, the ones
// on the way and their number, by jumping (5 rounds of shuffles); that ancestor's
// parent lies in an earlier block, so that a node's row is that parent's row and
// the block's own word. Block after block, the rows before them complete: n / 32
// steps of one shared load a word, whatever the depth. A launch bounds the small
// cases, the steps the large ones. 16 sequences of up to 1000 nodes in single
// file: 60.9 us jumping over the whole tree (log2 n rounds over all words), 15.9
// with all words in one CTA, 7.2 so.
constexpr int kGroupWords = 8;
__global__ void __launch_bounds__(32 * kGroupWords)
    build_tree_kernel(const int32_t *__restrict__ parents, const int32_t *__restrict__ cu_q, const int32_t *__restrict__ seq_lens,
                      int total_q, int words, int lane_words, int32_t *__restrict__ positions, uint32_t *__restrict__ masks)
{
    extern __shared__ uint32_t tree_smem[];  // [n][lane_words]
    __shared__ int s_above[kMaxNodes], s_depth[kMaxNodes];
    __shared__ uint32_t s_own[kMaxNodes];
    const int s = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool first = blockIdx.y == 0;  // the group that flags and writes positions
    const int q0 = cu_q[s], L = seq_lens[s];
    const long long n64 = (long long)cu_q[s + 1] - q0;
    if (n64 < 0 || n64 > min(kMaxNodes, 32 * words) || q0 < 0 || q0 > total_q - n64 || L < n64) {
        if (first && tid == 0)
            tree_raise(PA_DEVERR_SEQ_LEN);
        return;
    }
    const int n = (int)n64, blocks = (n + 31) / 32;
    for (int b = warp; b < blocks; b += blockDim.x / 32) {
        const int i = 32 * b + lane;
        int a = i < n ? parents[q0 + i] : -1;
        if (a < -1 || a >= i) {
            if (first && i < n)
                tree_raise(PA_DEVERR_TREE);
            a = -1;
        }
        int top = a >= 32 * b ? a - 32 * b : lane;  // of the block; itself: no ancestor there
        int steps = a >= 32 * b ? 1 : 0;
        uint32_t own = 1u << lane;
#pragma unroll
        for (int r = 0; r < 5; ++r) {
            own |= __shfl_sync(kFull, own, top);
            steps += __shfl_sync(kFull, steps, top);
            top = __shfl_sync(kFull, top, top);
        }
        s_above[i] = __shfl_sync(kFull, a, top);
        s_depth[i] = steps;
        s_own[i] = own;
    }
    __syncthreads();
    // Thread: word w of one node of the block; neighbours share a row.
    const int w0 = blockIdx.y * kGroupWords, w = w0 + (tid & (lane_words - 1));
    for (int b = w0; b < blocks; ++b) {
        const int i = 32 * b + tid / lane_words;
        if (i < n) {
            const int above = s_above[i];
            // A row has no bits in words behind its own block's.
            uint32_t set = w == b ? s_own[i] : 0u;
            if (w < b && above >> 5 >= w)
                set = tree_smem[above * lane_words + w - w0];
            tree_smem[i * lane_words + w - w0] = set;
            if (w == 0 && above >= 0)
                s_depth[i] += s_depth[above] + 1;
        }
        __syncthreads();
    }
    if (w < words)
        for (int i = tid / lane_words; i < n; i += 32)
            masks[(long long)(q0 + i) * words + w] = i >> 5 >= w0 ? tree_smem[i * lane_words + w - w0] : 0u;
    if (first && positions)
        for (int i = tid; i < n; i += blockDim.x)
            positions[q0 + i] = L - n + s_depth[i];
}

// ----------------------------------------------------------- pa_verify_draft

// A sum held as an unevaluated pair hi + lo of fp32 numbers (about 46 bits):
// where a draw falls next to a border, 24 bits are too few, and fp64 runs at a
// sixty-fourth of the fp32 rate here (16 adds by every thread took 1 us).
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

__device__ __forceinline__ bool above(const Sum &a, const Sum &b) { return (a.hi - b.hi) + (a.lo - b.lo) > 0.f; }

// x (y.hi + y.lo)
__device__ __forceinline__ Sum times(float x, const Sum &y)
{
    const float h = __fmul_rn(x, y.hi);
    return Sum{h, fmaf(x, y.lo, fmaf(x, y.hi, -h))};
}

__device__ __forceinline__ Sum shfl(const Sum &s, int from)
{
    return Sum{__shfl_sync(kFull, s.hi, from), __shfl_sync(kFull, s.lo, from)};
}

// Inclusive sums over the lanes, STEP apart: lane i gets those of i, i - STEP, ...
template <int STEP>
__device__ __forceinline__ Sum running(Sum s)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = STEP; o < 32; o <<= 1) {
        const float h = __shfl_up_sync(kFull, s.hi, o), l = __shfl_up_sync(kFull, s.lo, o);
        if (lane >= o)
            add(s, h, l);
    }
    return s;
}

// max(p - a q, 0) as a pair, a >= 0, q >= 0 (the callers make entries that are not
// above 0, NaN among them, 0: they would add to what is left): the product's and the difference's
// rounding errors are kept ((p - d) - m is the latter's where p >= m, and only
// there it counts). Anything not above 0 (NaN too) is 0.
__device__ __forceinline__ Sum weight(float p, float q, const Sum &a)
{
    const float m = __fmul_rn(a.hi, q), me = fmaf(a.hi, q, -m);  // kept apart: no fused p - a q
    const float d = p - m, e = ((p - d) - m) - fmaf(a.lo, q, me);
    return d + e > 0.f ? Sum{d, e} : Sum{0.f, 0.f};
}

// Two sums side by side, and the same of two entries each (packed fp32, an
// instruction for two: by single ones the arithmetic took as long as the rows).
struct Sum2 {
    uint64_t hi, lo;
};

__device__ __forceinline__ void add(Sum2 &s, const Sum2 &w)
{
    const uint64_t t = add2(s.hi, w.hi), b = sub2(t, s.hi);
    s.lo = add2(s.lo, add2(add2(sub2(s.hi, sub2(t, b)), sub2(w.hi, b)), w.lo));
    s.hi = t;
}

__device__ __forceinline__ Sum2 weight(uint64_t p, uint64_t q, const Sum2 &a, uint64_t minus_a)
{
    const uint64_t nm = mul2(minus_a, q);
    const uint64_t d = add2(p, nm), e = sub2(add2(sub2(p, d), nm), fma2(a.lo, q, fma2(a.hi, q, nm)));
    float d0, d1, e0, e1;
    unpk2(d, d0, d1);
    unpk2(e, e0, e1);
    const bool in0 = d0 + e0 > 0.f, in1 = d1 + e1 > 0.f;
    return Sum2{pk2(in0 ? d0 : 0.f, in1 ? d1 : 0.f), pk2(in0 ? e0 : 0.f, in1 ? e1 : 0.f)};
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

// The address that `p` of this CTA's shared memory has in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t address_in(const void *p, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}

__device__ __forceinline__ unsigned long long load_from(const void *p, uint32_t rank)
{
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(address_in(p, rank)) : "memory");
    return v;
}

__device__ __forceinline__ void store_to(void *p, uint32_t rank, int v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(address_in(p, rank)), "r"(v) : "memory");
}

__device__ __forceinline__ unsigned long long bits_of(const Sum &s)
{
    return (unsigned long long)__float_as_uint(s.hi) << 32 | __float_as_uint(s.lo);
}

__device__ __forceinline__ Sum sum_of(unsigned long long b)
{
    return Sum{__uint_as_float((uint32_t)(b >> 32)), __uint_as_float((uint32_t)b)};
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
constexpr int kVerifyThreads = 256, kVerifyWarps = kVerifyThreads / 32, kMaxCluster = 8;
constexpr int kEntries = 64;
constexpr int kTiles = 8, kStep = 32 / kTiles;  // 512-byte tiles of a row that a warp loads at once; lanes that hold one's sum
// CTAs an SM: the drafter's rows beside the target's take 128 registers a thread.
__host__ __device__ constexpr int verify_ctas(int mode) { return mode == kDraft ? 2 : 3; }

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
//   a draw: the first entry whose running sum passes u times the row's sum.
//           The warps' sums, exchanged over the cluster, name the warp that
//           holds it; its tiles' sums (kept in registers where a part is one
//           chunk of kTiles) the tile, then the lane, which looks again at its
//           16 bytes.
//
// The chain from row to row bounds it (one row has to be read before the next
// is known: load, exchange, load again, exchange), then the rows' bytes. Every
// sum is taken in one order, whatever the timing.
template <typename T, int MODE>
__global__ void __launch_bounds__(kVerifyThreads, verify_ctas(MODE)) verify_draft_kernel(const VerifyParams p, int cluster)
{
    constexpr int VEC = 16 / sizeof(T);
    constexpr bool DRAFT = MODE == kDraft;
    __shared__ int s_parent[kMaxNodes], s_token[kMaxNodes];
    __shared__ float s_p[DRAFT ? kMaxNodes : 1], s_q[DRAFT ? kMaxNodes : 1], s_u[DRAFT ? kMaxNodes : 1];
    // The warps' words, and the CTA's, exchanged with the others; two turns, so
    // that a slot is written again only after a barrier behind its last read.
    __shared__ unsigned long long s_warp[2][kVerifyWarps], s_cta[2];
    __shared__ int s_drawn[2];
    __shared__ float2 s_tile[kVerifyWarps][kEntries];  // the sums of a warp's tiles, or of groups of them

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
        if constexpr (DRAFT) {
            // The numbers that decide on this node.
            const bool in = has && (unsigned)x < (unsigned)V;
            s_p[i] = in ? to_float(target[(q0 + a) * p.target_stride + x]) : 0.f;
            s_q[i] = in ? fmaxf(to_float(draft[(q0 + a) * p.draft_stride + x]), 0.f) : 0.f;
            s_u[i] = p.uniforms[2 * (q0 + i)];
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
        r.q = DRAFT ? draft + (q0 + node) * p.draft_stride : nullptr;
        r.mis = (int)((reinterpret_cast<uintptr_t>(r.p) & 15) / sizeof(T));
        r.q_vec = DRAFT && ((reinterpret_cast<uintptr_t>(r.p) ^ reinterpret_cast<uintptr_t>(r.q)) & 15) == 0;
        const long long vecs = ((long long)V + r.mis + VEC - 1) / VEC;
        r.v0 = (int)(vecs * part / parts);
        r.v1 = (int)(vecs * (part + 1) / parts);
        return r;
    };
    // Vector v of a row, zeros outside it.
    auto load = [&](const T *row, int mis, int v, bool vec) {
        const int i0 = v * VEC - mis;
        if (vec && i0 >= 0 && i0 + VEC <= V)
            return __ldg(reinterpret_cast<const uint4 *>(row + i0));
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int k = 0; k < VEC; ++k)
            if (i0 + k >= 0 && i0 + k < V) {
                if constexpr (sizeof(T) == 4)
                    w[k] = __float_as_uint(row[i0 + k]);
                else
                    w[k / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(row)[i0 + k] << (16 * (k & 1));
            }
        return make_uint4(w[0], w[1], w[2], w[3]);
    };
    auto weights = [&](const uint4 &vp, const uint4 &vq, const Sum &a, Sum *w) {
        float x[VEC], y[VEC];
        widen<T>(vp, x);
        if (DRAFT && a.hi != 0.f) {
            widen<T>(vq, y);
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                w[k] = weight(x[k], fmaxf(y[k], 0.f), a);
        } else {
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                w[k] = Sum{x[k] > 0.f ? x[k] : 0.f, 0.f};
        }
    };
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    // Tile lane / kStep's sum over the lanes, of the kTiles tiles from vector v on.
    auto chunk = [&](const Row &r, int v, const Sum &a) {
        Sum tile[kTiles];  // this lane's sums of its vectors
        uint4 x[kTiles], y[DRAFT ? kTiles : 1];
        const bool with_q = DRAFT && a.hi != 0.f;
        // Inside the row, as most chunks are, nothing has to be looked at.
        if (v + 32 * kTiles <= r.v1 && v > 0 && (v + 32 * kTiles) * VEC - r.mis <= V && (!with_q || r.q_vec)) {
            const uint4 *xp = reinterpret_cast<const uint4 *>(r.p - r.mis) + v + lane;
            const uint4 *yp = DRAFT ? reinterpret_cast<const uint4 *>(r.q - r.mis) + v + lane : nullptr;
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
                x[t] = __ldg(xp + 32 * t);
            if constexpr (DRAFT) {
                if (with_q) {
#pragma unroll
                    for (int t = 0; t < kTiles; ++t)
                        y[t] = __ldg(yp + 32 * t);
                }
            }
        } else {
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                const int at = v + 32 * t + lane;
                x[t] = at < r.v1 ? load(r.p, r.mis, at, true) : none;
                if constexpr (DRAFT)
                    y[t] = at < r.v1 && with_q ? load(r.q, r.mis, at, r.q_vec) : none;
            }
        }
        // Tiles t and t + kTiles / 2 side by side.
        const Sum2 a2 = {pk2(a.hi, a.hi), pk2(a.lo, a.lo)};
        const uint64_t minus = pk2(-a.hi, -a.hi);
#pragma unroll
        for (int t = 0; t < kTiles / 2; ++t) {
            float x0[VEC], x1[VEC], y0[VEC], y1[VEC];
            widen<T>(x[t], x0);
            widen<T>(x[t + kTiles / 2], x1);
            if (with_q) {
                widen<T>(y[DRAFT ? t : 0], y0);
                widen<T>(y[DRAFT ? t + kTiles / 2 : 0], y1);
            }
            Sum2 both;
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                Sum2 w;
                if (with_q)
                    w = weight(pk2(x0[k], x1[k]), pk2(fmaxf(y0[k], 0.f), fmaxf(y1[k], 0.f)), a2, minus);
                else
                    w = Sum2{pk2(fmaxf(x0[k], 0.f), fmaxf(x1[k], 0.f)), 0ull};
                if (k == 0)
                    both = w;
                else
                    add(both, w);
            }
            unpk2(both.hi, tile[t].hi, tile[t + kTiles / 2].hi);
            unpk2(both.lo, tile[t].lo, tile[t + kTiles / 2].lo);
        }
        // Halving: a lane keeps half of its tiles and gives the others away, until it has one.
#pragma unroll
        for (int m = kTiles / 2, bit = 16; m > 0; m /= 2, bit /= 2)
#pragma unroll
            for (int k = 0; k < m; ++k) {
                const bool up = lane & bit;
                const Sum give = up ? tile[k] : tile[m + k];
                tile[k] = up ? tile[m + k] : tile[k];
                add(tile[k], __shfl_xor_sync(kFull, give.hi, bit), __shfl_xor_sync(kFull, give.lo, bit));
            }
        Sum one = tile[0];
#pragma unroll
        for (int o = kStep / 2; o > 0; o >>= 1) {
            const float h = __shfl_xor_sync(kFull, one.hi, o), l = __shfl_xor_sync(kFull, one.lo, o);
            add(one, h, l);
        }
        return one;
    };
    int turn = 0;
    // With one CTA a sequence there is nobody to wait for beyond it.
    auto barrier = [&] {
        if (cluster > 1)
            cluster_barrier();
        else
            __syncthreads();
    };
    // Every CTA's word: lane c gets that of CTA c.
    auto exchange = [&](unsigned long long mine) {
        if (cluster == 1)
            return mine;
        if (tid == 0)
            s_cta[turn] = mine;
        cluster_barrier();
        return lane < cluster ? load_from(&s_cta[turn], lane) : 0ull;
    };
    // The sum of max(p - a q, 0) over the row. Leaves what draw needs: lane w's
    // sum of this CTA's warp w and those up to it, lane c's of CTA c, and the
    // sums of this warp's tiles in s_tile (of groups of whole chunks where they
    // are more than kEntries).
    Sum warp_share, warp_upto, cta_share, cta_upto;
    auto tiles_per_entry = [&](const Row &r) {
        const int tiles = (r.v1 - r.v0 + 31) / 32;
        return tiles <= kEntries ? 1 : (tiles + kEntries * kTiles - 1) / (kEntries * kTiles) * kTiles;
    };
    auto total_of = [&](const Row &r, const Sum &a) {
        const int group = tiles_per_entry(r);
        Sum mine = {0.f, 0.f}, entry = {0.f, 0.f};
        __syncwarp();
        for (int v = r.v0, t = 0; v < r.v1; v += 32 * kTiles, t += kTiles) {
            const Sum one = chunk(r, v, a);
            const Sum all = shfl(running<kStep>(one), 31);
            add(mine, all.hi, all.lo);
            if (group == 1) {
                if (lane % kStep == 0 && t + lane / kStep < kEntries)
                    s_tile[warp][t + lane / kStep] = make_float2(one.hi, one.lo);
            } else {
                if (t % group == 0)
                    entry = Sum{0.f, 0.f};
                add(entry, all.hi, all.lo);
                if (lane == 0)
                    s_tile[warp][t / group] = make_float2(entry.hi, entry.lo);
            }
        }
        turn ^= 1;
        if (lane == 0)
            s_warp[turn][warp] = bits_of(mine);
        __syncthreads();
        warp_share = lane < kVerifyWarps ? sum_of(s_warp[turn][lane]) : Sum{0.f, 0.f};
        warp_upto = running<1>(warp_share);
        cta_share = sum_of(exchange(bits_of(shfl(warp_upto, 31))));
        if (cluster == 1 && lane > 0)
            cta_share = Sum{0.f, 0.f};
        cta_upto = running<1>(cta_share);
        return shfl(cta_upto, 31);
    };
    // Of the lanes' shares the first whose running sum, on top of `run`, passes t;
    // run becomes the sum before it. Where rounding leaves none, the last share
    // above 0, and `sure` is false.
    auto holder = [&](const Sum &share, const Sum &upto, const Sum &t, Sum &run, bool &sure) {
        Sum here = run;
        add(here, upto.hi, upto.lo);
        const unsigned some = __ballot_sync(kFull, share.hi > 0.f);
        const unsigned over = __ballot_sync(kFull, share.hi > 0.f && above(here, t));
        sure = over != 0u;
        const int at = over ? __ffs(over) - 1 : some ? 31 - __clz(some) : 0;
        const Sum before = shfl(upto, at ? at - 1 : 0);
        if (at)
            add(run, before.hi, before.lo);
        return at;
    };
    // A token drawn from max(p - a q, 0), whose sum z total_of has just given.
    auto draw = [&](const Row &r, const Sum &a, const Sum &z, float u) {
        const Sum t = times(u, z);
        Sum run = {0.f, 0.f};
        bool sure = true;
        const int owner = holder(cta_share, cta_upto, t, run, sure);
        if (rank == owner && warp == holder(warp_share, warp_upto, t, run, sure)) {
            const bool with_q = DRAFT && a.hi != 0.f;
            const int group = tiles_per_entry(r), entries = ((r.v1 - r.v0 + 31) / 32 + group - 1) / group;
            int found = -1, at = -1;
            for (int e0 = 0; sure && e0 < entries; e0 += 32) {
                const float2 e = e0 + lane < entries ? s_tile[warp][e0 + lane] : make_float2(0.f, 0.f);
                const Sum share = {e.x, e.y}, upto = running<1>(share);
                Sum before = run;
                bool here;
                const int k = holder(share, upto, t, before, here);
                if (here) {
                    run = before;
                    at = e0 + k;
                    break;
                }
                const Sum all = shfl(upto, 31);
                add(run, all.hi, all.lo);
            }
            for (int k = 0; at >= 0 && k < group && found < 0; ++k) {
                const int v = r.v0 + 32 * (at * group + k) + lane;
                Sum e[VEC], w = {0.f, 0.f};
                if (v < r.v1)
                    weights(load(r.p, r.mis, v, true), with_q ? load(r.q, r.mis, v, r.q_vec) : none, a, e);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    if (v >= r.v1)
                        e[j] = Sum{0.f, 0.f};
                    add(w, e[j].hi, e[j].lo);
                }
                const Sum upto = running<1>(w);
                Sum before = run;
                bool here;
                const int l = holder(w, upto, t, before, here);
                const unsigned some = __ballot_sync(kFull, w.hi > 0.f);
                if (here || (group == 1 && some)) {  // this lane's entries, one after the other
                    int mine = -1;
                    bool done = false;
#pragma unroll
                    for (int j = 0; j < VEC; ++j)
                        if (e[j].hi > 0.f && !done) {
                            add(before, e[j].hi, e[j].lo);
                            mine = v * VEC + j - r.mis;
                            done = above(before, t);
                        }
                    found = __shfl_sync(kFull, mine, l);
                }
                const Sum all = shfl(upto, 31);
                add(run, all.hi, all.lo);
            }
            if (found < 0) {
                // Rounding: a sum passed t that another order of its terms does not
                // pass. The border is at the end of what was found last, the group of
                // tiles or the part: its last positive entry.
                const int lo = at >= 0 ? r.v0 + 32 * at * group : r.v0;
                const int hi = at >= 0 ? min(r.v1, lo + 32 * group) : r.v1;
                for (int v = lo + lane; v < hi; v += 32) {
                    Sum e[VEC];
                    weights(load(r.p, r.mis, v, true), with_q ? load(r.q, r.mis, v, r.q_vec) : none, a, e);
#pragma unroll
                    for (int j = 0; j < VEC; ++j)
                        if (e[j].hi > 0.f)
                            found = v * VEC + j - r.mis;
                }
                found = max(0, __reduce_max_sync(kFull, found));
            }
            if (lane < cluster)
                store_to(&s_drawn[turn], lane, found);
        }
        barrier();
        return *const_cast<volatile int *>(&s_drawn[turn]);
    };
    // The row's first largest entry, NaN passed over.
    auto largest = [&](const Row &r) {
        float best = -INFINITY;
        int at = 0x7fffffff;
        for (int v = r.v0; v < r.v1; v += 32 * kTiles) {
            uint4 raw[kTiles];
#pragma unroll
            for (int t = 0; t < kTiles; ++t)
                raw[t] = v + 32 * t + lane < r.v1 ? load(r.p, r.mis, v + 32 * t + lane, true) : none;
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
                float x[VEC];
                widen<T>(raw[t], x);
                const int i0 = (v + 32 * t + lane) * VEC - r.mis;
#pragma unroll
                for (int k = 0; k < VEC; ++k)
                    if (v + 32 * t + lane < r.v1 && i0 + k >= 0 && i0 + k < V && x[k] > best) {
                        best = x[k];
                        at = i0 + k;
                    }
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
            s_warp[turn][warp] = key;
        __syncthreads();
        auto most = [&] {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                key = max(key, __shfl_xor_sync(kFull, key, o));
        };
        key = lane < kVerifyWarps ? s_warp[turn][lane] : 0ull;
        most();
        if (cluster > 1) {
            key = exchange(key);
            most();
        }
        const int i = (int)(0x7fffffffu - (uint32_t)key);
        return i < V ? i : 0;
    };

    int node = 0;
    for (int k = 0; k < n; ++k) {  // each step goes to a later node
        int next = n, token = 0;
        const Row r = row_at(node);
        if constexpr (MODE == kGreedy) {
            token = largest(r);
        } else {
            Sum a = {0.f, 0.f}, z = {1.f, 0.f};  // draft: see above
            int kid = DRAFT ? child_of(node, node) : n;
            for (;;) {
                if constexpr (DRAFT) {
                    if (kid < n) {
                        const Sum rx = a.hi > 0.f ? weight(s_p[kid], s_q[kid], a) : Sum{s_p[kid], 0.f};
                        // u q, a pair, times Z
                        const float h = __fmul_rn(s_u[kid], s_q[kid]);
                        Sum bar = times(h, z);
                        bar.lo += fmaf(s_u[kid], s_q[kid], -h) * z.hi;
                        if (above(rx, bar)) {
                            next = kid;
                            break;
                        }
                        add(a, z.hi, z.lo);
                        const float lead = a.hi + a.lo;
                        a = Sum{lead, a.lo - (lead - a.hi)};
                        kid = child_of(node, kid);
                    }
                }
                z = total_of(r, a);
                if (DRAFT && kid < n)
                    continue;
                if (z.hi > 0.f && z.hi <= FLT_MAX) {
                    token = draw(r, a, z, p.uniforms[2 * (q0 + node) + 1]);
                    break;
                }
                if (a.hi == 0.f) {
                    if (rank == 0 && tid == 0)
                        tree_raise(PA_DEVERR_TREE);
                    break;
                }
                a = Sum{0.f, 0.f};  // nothing is left of the row: the target's own
            }
        }
        if constexpr (!DRAFT) {
            next = child_of(node, node);
            while (next < n && s_token[next] != token)
                next = child_of(node, next);
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
    barrier();  // nobody leaves while its shared memory may be read
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

constexpr int kMoveThreads = 256, kMoveBatch = 8, kMoveCtas = 16;

// Moves: a thread takes one 16-byte column of one layer's K or V rows (then
// another) and all of a sequence's accepted tokens, in ascending order,
// kMoveBatch of them read before the first is written. Token path[j] >= j goes
// to place j, so a write never reaches a row that a later batch still reads, and
// no other thread touches the column: no copy in between, no barrier. HBM bounds
// it: 64 sequences, 192 moved tokens, 40 layers of 40 heads of 128 fp16 (315 MB
// read and written) 57 us, 5.5 TB/s; 69 us with a CTA for every 256 columns,
// whose look-ups of the slots (count, path, table, one after the other) then
// took as long as its copies.
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
    const int columns = 2 * p.num_layers * p.row_vecs;
    for (int c = blockIdx.x * kMoveThreads + tid; c < columns; c += gridDim.x * kMoveThreads) {
        const int lk = c / p.row_vecs, v = c - lk * p.row_vecs;
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

// The current device's SM count, asked for once per device.
int sm_count_of(const char *who, int *sms_out)
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
        if (e != cudaSuccess)
            return set_error(PA_ERR_CUDA, "%s: SM count: %s", who, cudaGetErrorString(e));
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
    // A thread per word of 32 nodes' masks.
    int lane_words = 1;
    while (lane_words < std::min(mask_words, kGroupWords))
        lane_words *= 2;
    const dim3 grid(num_seqs, (mask_words + kGroupWords - 1) / kGroupWords);
    build_tree_kernel<<<grid, 32 * lane_words, (size_t)32 * mask_words * lane_words * 4, reinterpret_cast<cudaStream_t>(stream)>>>(
        parents, cu_seqlens_q, seq_lens, total_q, mask_words, lane_words, positions, reinterpret_cast<uint32_t *>(tree_masks));
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
    const int rc = sm_count_of(who, &sms);
    if (rc != PA_OK)
        return rc;
    // CTAs a sequence: as many as run at once, up to those that leave a warp one
    // chunk of a row. Measured with 1 / 2 / 4 / 8 of them: 256 sequences, drafter's
    // rows, 32000 entries 19.9 / 28.6 / 42.9 / 77.0 us; 48 sequences, drawn, 100003
    // entries 62 / 38 / 28.8 / 24.3; one, greedy, 131072 entries 30.6 / 19.4 / 12.8 /
    // 9.4 (clusters of 16, or CTAs of 512 threads, are slower in each).
    const int mode = !uniforms ? kGreedy : draft ? kDraft : kSample;
    const long long chunk = kVerifyWarps * kTiles * 512 / (int)elem, room = (long long)sms * verify_ctas(mode);
    int cluster = 1;
    while (cluster < kMaxCluster && cluster * chunk < vocab_size && 2LL * num_seqs * cluster <= room)
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
    const cudaError_t e = cudaLaunchKernelExC(&cfg, verify_kernel(dtype, mode), args);
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
    if (columns > 0x3fffffffLL)
        return set_error(PA_ERR_UNSUPPORTED, "%s: %d layers of rows of %lld bytes are too many columns", who, num_layers, row_bytes);
    int sms = 0;
    const int rc = sm_count_of(who, &sms);
    if (rc != PA_OK)
        return rc;
    // A CTA looks its sequence's slots up once and then takes several columns a
    // thread: about kMoveCtas CTAs an SM in all.
    const long long most = (columns + kMoveThreads - 1) / kMoveThreads;
    const dim3 grid((unsigned)std::min(most, std::max(1LL, (long long)sms * kMoveCtas / num_seqs)), num_seqs);
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
