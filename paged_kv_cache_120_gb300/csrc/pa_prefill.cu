// pa_prefill, pa_cross_attention and pa_tree_attention on the chunk kernel:
// tensor maps, launch plans and the C ABI. The kernel is in
// pa_prefill_kernel.cuh; its causal and cross kinds are instantiated here, the
// tree kinds in pa_tree_attention.cu.
#include "pa_prefill_kernel.cuh"

namespace pa {

namespace {

// 2^x0, 2^x1 on the FMA pipe, without the MUFU unit that ex2 uses: x = j + f
// with j = round(x) (adding and subtracting 1.5 * 2^23 rounds to an integer
// in fp32 for |x| < 2^22) and f in [-1/2, 1/2] exact, then p(f) ~ 2^f by the
// minimax polynomial of degree DEG (coefficients from a Remez exchange fit of
// the relative error, printed by paged_kv_cache_120_gb300/exp2_poly.py; max
// relative error 7.5e-5 at degree 3, 2.7e-6 at degree 4), then j added to
// p's exponent field. Inputs below -126 are clamped there (2^-126 or less
// rounds to zero or to a negligible subnormal in the 16-bit P); NaN stays
// NaN (max.NaN keeps it, and the exponent add leaves NaN bits NaN).
template <int DEG>
__device__ __forceinline__ void exp2_poly2(uint64_t x2, float &y0, float &y1)
{
    float x0, x1;
    unpk2(x2, x0, x1);
    asm("max.NaN.f32 %0, %0, 0fC2FC0000;" : "+f"(x0));  // -126
    asm("max.NaN.f32 %0, %0, 0fC2FC0000;" : "+f"(x1));
    const uint64_t xv = pk2(x0, x1);
    const uint64_t magic = pk2(12582912.f, 12582912.f), nmagic = pk2(-12582912.f, -12582912.f);
    const uint64_t j = add2(xv, magic);           // round(x) in the low mantissa bits
    const uint64_t t = add2(j, nmagic);           // round(x) as a float
    uint64_t f;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(f) : "l"(xv), "l"(t));
    uint64_t p;
    if constexpr (DEG == 4) {
        p = fma2(pk2(0x1.3997d6p-7f, 0x1.3997d6p-7f), f, pk2(0x1.ca1440p-5f, 0x1.ca1440p-5f));
        p = fma2(p, f, pk2(0x1.ec06dap-3f, 0x1.ec06dap-3f));
        p = fma2(p, f, pk2(0x1.62e0dcp-1f, 0x1.62e0dcp-1f));
        p = fma2(p, f, pk2(0x1.ffffe8p-1f, 0x1.ffffe8p-1f));
    } else {
        static_assert(DEG == 3, "degree 3 or 4");
        p = fma2(pk2(0x1.c3f760p-5f, 0x1.c3f760p-5f), f, pk2(0x1.f0de1ap-3f, 0x1.f0de1ap-3f));
        p = fma2(p, f, pk2(0x1.62f31ap-1f, 0x1.62f31ap-1f));
        p = fma2(p, f, pk2(0x1.fff692p-1f, 0x1.fff692p-1f));
    }
    float p0, p1, j0, j1;
    unpk2(p, p0, p1);
    unpk2(j, j0, j1);
    y0 = __uint_as_float(__float_as_uint(p0) + (__float_as_uint(j0) << 23));
    y1 = __uint_as_float(__float_as_uint(p1) + (__float_as_uint(j1) << 23));
}

// ================================================================ host side

PFN_cuTensorMapEncodeTiled_v12000 encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

// Pool as rank 5 (head_size, kv_heads, block slots, blocks, K|V), box of 64
// dims x one head x 16 slots x one block x one of K/V: 2 KB, 128-byte swizzle.
int encode_kv_map(CUtensorMap *m, const void *kv, int num_blocks, int block_size, int num_kv_heads, int d)
{
    const cuuint64_t e = 2, hd = (cuuint64_t)d;
    cuuint64_t dims[5] = {hd, (cuuint64_t)num_kv_heads, (cuuint64_t)block_size, (cuuint64_t)num_blocks, 2};
    cuuint64_t strides[4] = {hd * e, (cuuint64_t)num_kv_heads * hd * e,
                             (cuuint64_t)block_size * num_kv_heads * hd * e,
                             (cuuint64_t)num_blocks * block_size * num_kv_heads * hd * e};
    cuuint32_t box[5] = {64, 1, (cuuint32_t)kBoxTokens, 1, 1};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    // A row of a 64-wide head is 128 bytes: promoted to 256, its load would pull
    // the next head's row from DRAM as well (512 queries over 8000 states, 32
    // heads: 66.1 us promoted, 65.2 us not; equal where heads share the L2).
    CUresult r = encoder()(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 5, const_cast<void *>(kv), dims, strides, box,
                           estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           d == kD ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? PA_OK : set_error(PA_ERR_CUDA, "pa_prefill: K/V tensor map (%d)", (int)r);
}

// An FP8 pool as rank 5 (head_size bytes, kv_heads, block slots, blocks,
// K|V), box of the d codes of one head x 16 slots: 128-byte rows with the
// 128-byte swizzle at d = 128 (2 KB), plain 64-byte rows at d = 64 (1 KB).
// Tree attention's MMAs read the codes as they lie: 64-byte rows are swizzled there.
int encode_kv_map_fp8(CUtensorMap *m, const void *kv, int num_blocks, int block_size, int num_kv_heads, int d, bool swizzle64)
{
    const cuuint64_t hd = (cuuint64_t)d;
    cuuint64_t dims[5] = {hd, (cuuint64_t)num_kv_heads, (cuuint64_t)block_size, (cuuint64_t)num_blocks, 2};
    cuuint64_t strides[4] = {hd, (cuuint64_t)num_kv_heads * hd, (cuuint64_t)block_size * num_kv_heads * hd,
                             (cuuint64_t)num_blocks * block_size * num_kv_heads * hd};
    cuuint32_t box[5] = {(cuuint32_t)d, 1, (cuuint32_t)kBoxTokens, 1, 1};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    CUresult r = encoder()(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void *>(kv), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE,
                           d == kD ? CU_TENSOR_MAP_SWIZZLE_128B : swizzle64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? PA_OK : set_error(PA_ERR_CUDA, "pa_prefill_fp8: K/V tensor map (%d)", (int)r);
}

// Queries as rank 3 (head_size, q_heads, tokens), box of 64 dims x one head x
// rows_per_head tokens.
int encode_q_map(CUtensorMap *m, const void *q, int total_q, int num_q_heads, int rows, int d)
{
    const cuuint64_t e = 2, hd = (cuuint64_t)d;
    cuuint64_t dims[3] = {hd, (cuuint64_t)num_q_heads, (cuuint64_t)total_q};
    cuuint64_t strides[2] = {hd * e, (cuuint64_t)num_q_heads * hd * e};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)rows};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = encoder()(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void *>(q), dims, strides, box,
                           estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? PA_OK : set_error(PA_ERR_CUDA, "pa_prefill: query tensor map (%d)", (int)r);
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

int prefill_take_device_error(int *bits)
{
    int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_prefill_error, sizeof(int));
    if (e == cudaSuccess)
        e = cudaMemcpyToSymbol(g_prefill_error, &zero, sizeof(int));
    *bits = e == cudaSuccess ? v : 0;
    return (int)e;
}

}  // namespace pa

using namespace pa;

namespace {

// A launch's work units and scheduling. With enough units, persistent CTAs
// take whole units, heaviest first, from the launch's grid. With few (at most kSplitUnitsPerSm per SM, and a workspace), the
// units' K/V tiles are dealt out in equal contiguous shares (stream-K) to
// one CTA per SM, however many pieces that cuts a unit into (the merge
// spreads a unit's pieces over several threads per row).
constexpr int kSplitUnitsPerSm = 4;

struct LaunchPlan {
    int heads_per_cta, head_tiles, rows_per_head, q_pairs;
    long long units;
    int split_grid;     // G under stream-K, 0 when the launch takes whole units
    size_t split_bytes; // workspace stream-K needs
};

LaunchPlan plan_launch(int num_seqs, int max_seqlen_q, int num_q_heads, int num_kv_heads, int head_size, int sms)
{
    LaunchPlan lp;
    const int group = num_q_heads / num_kv_heads;
    lp.heads_per_cta = group < 16 ? group : 16;
    lp.head_tiles = group / lp.heads_per_cta;
    lp.rows_per_head = (kM / lp.heads_per_cta) & ~7;
    const long long q_tiles = ((long long)max_seqlen_q + lp.rows_per_head - 1) / lp.rows_per_head;
    lp.q_pairs = (int)((q_tiles + 1) / 2);
    lp.units = (long long)lp.q_pairs * num_seqs * num_kv_heads * lp.head_tiles;
    lp.split_grid = 0;
    lp.split_bytes = 0;
    if (lp.units > 0 && lp.units <= std::min<long long>(kMaxSplitUnits, (long long)kSplitUnitsPerSm * sms)) {
        lp.split_grid = sms;
        // Per CTA two slots of two 128-row tiles: O rows (head_size fp32)
        // and (m, l) pairs; then one job record per CTA.
        lp.split_bytes = (size_t)lp.split_grid * 2 * 2 * kM * ((size_t)head_size * 4 + 8) + (size_t)lp.split_grid * 16;
    }
    return lp;
}

// Launch with programmatic stream serialisation: the kernel may be scheduled
// while the previous one in the stream finishes and waits for it with
// griddepcontrol.wait before reading what it wrote.
cudaError_t launch_pdl(const void *fn, dim3 grid, dim3 block, void **args, size_t smem, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

// SM count of the current device (cached per device).
int current_sms(const char *who, int *dev_out, int *sms_out)
{
    static std::mutex mu;
    static int sm_count[64] = {};
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return set_error(PA_ERR_CUDA, "%s: cudaGetDevice: %s", who, cudaGetErrorString(e));
    std::lock_guard<std::mutex> lock(mu);
    sms = dev < 64 ? sm_count[dev] : 0;
    if (sms <= 0) {
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess || sms <= 0)
            return set_error(PA_ERR_CUDA, "%s: SM count: %s", who, cudaGetErrorString(e));
        if (dev < 64)
            sm_count[dev] = sms;
    }
    *dev_out = dev;
    *sms_out = sms;
    return PA_OK;
}

int check_heads(const char *who, int num_q_heads, int num_kv_heads, int head_size)
{
    if (head_size != kD && head_size != 64)
        return set_error(PA_ERR_UNSUPPORTED, "%s: head_size %d (built: 64 and 128)", who, head_size);
    if (num_kv_heads <= 0 || num_q_heads <= 0 || num_q_heads % num_kv_heads != 0)
        return set_error(PA_ERR_INVALID_ARG,
                         "%s: num_q_heads %d must be a positive multiple of num_kv_heads %d", who,
                         num_q_heads, num_kv_heads);
    const int group = num_q_heads / num_kv_heads;
    if (group > 16 && group % 16 != 0)
        return set_error(PA_ERR_UNSUPPORTED, "%s: query group %d (want <= 16 or a multiple of 16)", who,
                         group);
    return PA_OK;
}

// Checks shared by the causal and the cross calls; *empty: nothing to do.
int check_call(const char *who, const void *out, const void *query, const void *kv_cache, const int32_t *block_tables,
               int max_blocks_per_seq, const int32_t *cu_seqlens_q, const int32_t *seq_lens, int num_seqs, int total_q,
               int max_seqlen_q, float scale, int num_q_heads, int num_kv_heads, int head_size, int num_blocks,
               int block_size, int dtype, bool *empty)
{
    *empty = false;
    if (dtype != PA_F16 && dtype != PA_BF16)
        return set_error(PA_ERR_UNSUPPORTED, "%s: dtype %d (want PA_F16 or PA_BF16)", who, dtype);
    int rc = check_heads(who, num_q_heads, num_kv_heads, head_size);
    if (rc != PA_OK)
        return rc;
    if (block_size < kBoxTokens || block_size % kBoxTokens != 0)
        return set_error(PA_ERR_INVALID_ARG, "%s: block_size %d must be a positive multiple of 16", who,
                         block_size);
    if (num_seqs < 0 || total_q < 0 || max_seqlen_q < 0 || num_blocks <= 0 || max_blocks_per_seq <= 0)
        return set_error(PA_ERR_INVALID_ARG, "%s: bad sizes", who);
    if ((long long)max_blocks_per_seq * block_size > (1LL << 30))
        return set_error(PA_ERR_INVALID_ARG, "%s: max_blocks_per_seq * block_size too large", who);
    if (!std::isfinite(scale))
        return set_error(PA_ERR_INVALID_ARG, "%s: scale is not finite", who);
    *empty = num_seqs == 0 || total_q == 0 || max_seqlen_q == 0;
    if (*empty)
        return PA_OK;
    if (!out || !query || !kv_cache || !block_tables || !cu_seqlens_q || !seq_lens)
        return set_error(PA_ERR_INVALID_ARG, "%s: null pointer argument", who);
    if (!aligned16(out) || !aligned16(query) || !aligned16(kv_cache) ||
        (reinterpret_cast<uintptr_t>(block_tables) & 3) || (reinterpret_cast<uintptr_t>(cu_seqlens_q) & 3) ||
        (reinterpret_cast<uintptr_t>(seq_lens) & 3))
        return set_error(PA_ERR_INVALID_ARG, "%s: misaligned pointer (query/out/pool 16 B)", who);
    return PA_OK;
}

// Whether a cross batch of few units shares their tiles out or takes them
// whole. Whole units leave SMs idle in the last round: ceil(u) - 0.75 u units
// an SM (u: units per SM; 0.75: sequences are rarely all of the longest
// length), of the longest possible sequence's tiles (max_len, the width of the
// table: the host knows no lengths) and the two that a unit costs itself. Sharing costs about 9 + 5 u tiles (partial results, their merge, the
// cut units). Measured, 8 heads of 128, FP8 cache, shared against whole: 0.8
// units an SM over 400 / 1404 / 6404 states 35 / 51 / 117 and 18 / 31 / 118 us
// (78 and 102 over 1 .. 6404), 0.1 an SM 20 / 23 / 33 and 17 / 29 / 100, 2.1 an
// SM 57 / 91 / 262 and 45 / 87 / 336.
// Trees: 9 + 12 u, as a tile of theirs takes less than one of a cross batch
// beside what a cut unit costs. Shared against whole: 0.1 units an SM over
// 23371 tokens 33 and 194, 0.2 over 4425 37 and 54, 0.7 over 1 .. 5935 55 and
// 72, 3.4 over 4096 267 and 273; 1.05 over 57 .. 1139 26 and 18, 3.9 over 1 ..
// 4801 (FP8) 176 and 160 us. (2.5 over 0 .. 8191, FP8: 163 and 153, shared:
// were all of the longest, whole units would take three rounds for 2.5.)
bool cross_splits(long long units, int sms, long long max_len, bool tree)
{
    const double u = (double)units / sms, tiles = (double)((max_len + kN - 1) / kN) + 2.0;
    return (std::ceil(u) - 0.75 * u) * tiles > 9.0 + (tree ? 12.0 : 5.0) * u;
}

// What a call's queries see.
enum class Sees { kCausal, kAll, kTree };

int prefill_impl(const char *who, void *out, const void *query, const void *kv_cache, const int32_t *block_tables,
                 int max_blocks_per_seq, const int32_t *cu_seqlens_q, const int32_t *seq_lens, int num_seqs,
                 int total_q, int max_seqlen_q, float scale, int num_q_heads, int num_kv_heads, int head_size,
                 int num_blocks, int block_size, int dtype, bool fp8, float k_scale, float v_scale,
                 void *workspace, size_t workspace_bytes, Sees sees, const int32_t *tree_masks, int mask_words,
                 pa_stream_t stream)
{
    bool empty = false;
    int rc = check_call(who, out, query, kv_cache, block_tables, max_blocks_per_seq, cu_seqlens_q, seq_lens, num_seqs, total_q,
                        max_seqlen_q, scale, num_q_heads, num_kv_heads, head_size, num_blocks, block_size, dtype, &empty);
    if (rc != PA_OK || empty)
        return rc;
    const int group = num_q_heads / num_kv_heads;
    if (!encoder())
        return set_error(PA_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");

    int dev = 0, sms = 0;
    rc = current_sms(who, &dev, &sms);
    if (rc != PA_OK)
        return rc;
    LaunchPlan lp = plan_launch(num_seqs, max_seqlen_q, num_q_heads, num_kv_heads, head_size, sms);
    // A bound above total_q says no more than total_q: whole units are planned
    // for that, so that none is looked at in vain (the split, whose workspace
    // was sized by the caller's bound, keeps to it: it has few units).
    if (lp.split_grid == 0 && max_seqlen_q > total_q) {
        max_seqlen_q = total_q;
        lp = plan_launch(num_seqs, max_seqlen_q, num_q_heads, num_kv_heads, head_size, sms);
        lp.split_grid = 0;
    }
    if (lp.units > 0x7fffffffLL)
        return set_error(PA_ERR_UNSUPPORTED, "%s: too many query tiles", who);
    // Stream-K needs the workspace; without one the launch takes whole units.
    bool split = lp.split_grid > 0 && workspace != nullptr;
    if (split && (workspace_bytes < lp.split_bytes || (reinterpret_cast<uintptr_t>(workspace) & 255)))
        return set_error(PA_ERR_WORKSPACE, "%s: workspace of %zu bytes at %p (need %zu, 256-byte aligned)", who,
                         workspace_bytes, workspace, lp.split_bytes);
    if (sees != Sees::kCausal)
        split = split && cross_splits(lp.units, sms, (long long)max_blocks_per_seq * block_size, sees == Sees::kTree);

    TreeParams prm;  // the other kinds take its first part
    prm.out = out;
    prm.block_tables = block_tables;
    prm.cu_q = cu_seqlens_q;
    prm.seq_lens = seq_lens;
    prm.max_blocks_per_seq = max_blocks_per_seq;
    prm.num_seqs = num_seqs;
    prm.num_q_heads = num_q_heads;
    prm.group = group;
    prm.heads_per_cta = lp.heads_per_cta;
    prm.head_tiles = lp.head_tiles;
    const bool solo = max_seqlen_q <= lp.rows_per_head;
    // A tree's one query tile holds no more rows of a head than it needs, so
    // that whole warps are without one.
    prm.rows_per_head = sees == Sees::kTree && solo ? (max_seqlen_q + 7) & ~7 : lp.rows_per_head;
    prm.q_pairs = lp.q_pairs;
    prm.max_q = max_seqlen_q;
    prm.num_blocks = num_blocks;
    prm.block_size = block_size;
    prm.total_q = total_q;
    prm.max_len = max_blocks_per_seq * block_size;
    prm.scale_log2 = scale * 1.4426950408889634f * (fp8 ? k_scale : 1.f);
    prm.v_scale = fp8 ? v_scale : 1.f;
    prm.tree_masks = reinterpret_cast<const uint32_t *>(tree_masks);
    prm.mask_words = mask_words;
    prm.kv_cache = kv_cache;
    prm.query = query;
    prm.num_kv_heads = num_kv_heads;
    prm.num_units = (int)lp.units;
    prm.part_o = split ? static_cast<float *>(workspace) : nullptr;
    prm.part_ml = split ? reinterpret_cast<float2 *>(static_cast<float *>(workspace) +
                                                     (size_t)lp.split_grid * 2 * 2 * kM * head_size)
                        : nullptr;
    prm.jobs = split ? reinterpret_cast<int4 *>(prm.part_ml + (size_t)lp.split_grid * 2 * 2 * kM) : nullptr;

    CUtensorMap kv_map, q_map;
    rc = fp8 ? encode_kv_map_fp8(&kv_map, kv_cache, num_blocks, block_size, num_kv_heads, head_size, sees == Sees::kTree)
                 : encode_kv_map(&kv_map, kv_cache, num_blocks, block_size, num_kv_heads, head_size);
    if (rc != PA_OK)
        return rc;
    rc = encode_q_map(&q_map, query, total_q, num_q_heads, prm.rows_per_head, head_size);
    if (rc != PA_OK)
        return rc;

    const bool bf = dtype == PA_BF16, d64 = head_size == 64;
    // Instances by (kind, stream-K, FP8 cache, head size 64, bf16).
#define PA_PREFILL_INSTANCES(SK, KIND)                                                          \
    reinterpret_cast<const void *>(&paged_prefill_kernel<false, false, 128, SK, KIND>),          \
        reinterpret_cast<const void *>(&paged_prefill_kernel<true, false, 128, SK, KIND>),       \
        reinterpret_cast<const void *>(&paged_prefill_kernel<false, false, 64, SK, KIND>),       \
        reinterpret_cast<const void *>(&paged_prefill_kernel<true, false, 64, SK, KIND>),        \
        reinterpret_cast<const void *>(&paged_prefill_kernel<false, true, 128, SK, KIND>),       \
        reinterpret_cast<const void *>(&paged_prefill_kernel<true, true, 128, SK, KIND>),        \
        reinterpret_cast<const void *>(&paged_prefill_kernel<false, true, 64, SK, KIND>),        \
        reinterpret_cast<const void *>(&paged_prefill_kernel<true, true, 64, SK, KIND>)
    static const void *const kernels[48] = {PA_PREFILL_INSTANCES(false, kCausal), PA_PREFILL_INSTANCES(true, kCausal),
                                            PA_PREFILL_INSTANCES(false, kCross), PA_PREFILL_INSTANCES(true, kCross),
                                            PA_PREFILL_INSTANCES(false, kCrossSolo), PA_PREFILL_INSTANCES(true, kCrossSolo)};
#undef PA_PREFILL_INSTANCES
    const int kind = sees == Sees::kCausal ? kCausal : sees == Sees::kAll ? (solo ? kCrossSolo : kCross) : solo ? kTreeSolo : kTree;
    const int type = (split ? 8 : 0) + (fp8 ? 4 : 0) + (d64 ? 2 : 0) + (bf ? 1 : 0);
    const int variant = kind * 16 + type;
    const void *fn = sees == Sees::kTree ? tree_kernel(solo, type) : kernels[variant];
    // Raise the kernel's shared-memory limit once per device (a call being
    // captured into a CUDA graph then makes no attribute call; the SM count
    // is cached likewise).
    static std::mutex mu;
    static bool raised[80][64] = {};
    cudaError_t e;
    {
        std::lock_guard<std::mutex> lock(mu);
        bool &done = raised[variant][dev & 63];
        if (!done) {
            e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
            if (e != cudaSuccess)
                return set_error(PA_ERR_CUDA, "%s: cudaFuncSetAttribute: %s", who, cudaGetErrorString(e));
            done = dev < 64;
        }
    }
    // One CTA per SM runs at a time (it holds 225 KB of shared memory): G
    // CTAs under stream-K, else a CTA per unit, claimed by those that run.
    const dim3 grid(split ? (unsigned)lp.split_grid : (unsigned)lp.units);
    void *args[] = {&kv_map, &q_map, &prm};
    e = cudaLaunchKernel(fn, grid, dim3(threads_for(fp8)), args, kSmemBytes, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess)
        return set_error(PA_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
    if (split) {
        // Merge planes: enough that each thread folds about 8 pieces of a
        // unit cut into G / units + 1 pieces.
        const long long pieces = ((long long)lp.split_grid + lp.units - 1) / lp.units + 1;
        const int qi = pieces <= 8 ? 0 : pieces <= 16 ? 1 : pieces <= 32 ? 2 : 3;
#define PA_MERGE_INSTANCES(Q)                                                                      \
    reinterpret_cast<const void *>(&paged_prefill_merge_kernel<false, 128, Q>),                    \
        reinterpret_cast<const void *>(&paged_prefill_merge_kernel<true, 128, Q>),                 \
        reinterpret_cast<const void *>(&paged_prefill_merge_kernel<false, 64, Q>),                 \
        reinterpret_cast<const void *>(&paged_prefill_merge_kernel<true, 64, Q>)
        static const void *const merges[16] = {PA_MERGE_INSTANCES(1), PA_MERGE_INSTANCES(2), PA_MERGE_INSTANCES(4),
                                               PA_MERGE_INSTANCES(8)};
#undef PA_MERGE_INSTANCES
        static const int blocks128[4] = {MergeGeo<128, 1>::kBlocks, MergeGeo<128, 2>::kBlocks,
                                         MergeGeo<128, 4>::kBlocks, MergeGeo<128, 8>::kBlocks};
        static const int blocks64[4] = {MergeGeo<64, 1>::kBlocks, MergeGeo<64, 2>::kBlocks, MergeGeo<64, 4>::kBlocks,
                                        MergeGeo<64, 8>::kBlocks};
        int grid_main = lp.split_grid;
        const long long jobs = std::min<long long>(lp.units, grid_main);  // at most one per unit and per CTA
        const int merge_grid = (int)(jobs * 2 * (d64 ? blocks64[qi] : blocks128[qi]));
        void *margs[] = {&prm, &grid_main};
        e = launch_pdl(merges[qi * 4 + (d64 ? 2 : 0) + (bf ? 1 : 0)], dim3(merge_grid), dim3(256), margs, 0,
                       reinterpret_cast<cudaStream_t>(stream));
        if (e != cudaSuccess)
            return set_error(PA_ERR_CUDA, "%s: merge launch: %s", who, cudaGetErrorString(e));
    }
    return PA_OK;
}

// Cross attention: with a workspace, a few rows per kv head (the decode step
// of one query or a few candidates per sequence) are bound by reading K and V
// and take the decode kernels' ragged form, whose warps stream them; more rows
// take the prefill kernel without its causal limit. Arguments are checked
// alike either way.
int cross_impl(const char *who, void *out, const void *query, const void *kv_cache, const int32_t *block_tables,
               int max_blocks_per_seq, const int32_t *cu_seqlens_q, const int32_t *kv_lens, int num_seqs, int total_q,
               int max_seqlen_q, float scale, int num_q_heads, int num_kv_heads, int head_size, int num_blocks,
               int block_size, int dtype, bool fp8, float k_scale, float v_scale, void *workspace,
               size_t workspace_bytes, unsigned flags, pa_stream_t stream)
{
    if (flags & ~PA_DECODE_SHARED_BLOCKS)
        return set_error(PA_ERR_INVALID_ARG, "%s: unknown flags 0x%x", who, flags);
    bool empty = false;
    const int rc = check_call(who, out, query, kv_cache, block_tables, max_blocks_per_seq, cu_seqlens_q, kv_lens, num_seqs,
                              total_q, max_seqlen_q, scale, num_q_heads, num_kv_heads, head_size, num_blocks, block_size,
                              dtype, &empty);
    if (rc != PA_OK || empty)
        return rc;
    if (workspace && cross_rows_fit(num_seqs, max_seqlen_q, num_q_heads, num_kv_heads, block_size)) {
        if (reinterpret_cast<uintptr_t>(workspace) & 255)
            return set_error(PA_ERR_WORKSPACE, "%s: workspace at %p (256-byte aligned)", who, workspace);
        return cross_rows(who, out, query, kv_cache, block_tables, max_blocks_per_seq, cu_seqlens_q, kv_lens, num_seqs,
                          total_q, max_seqlen_q, scale, num_q_heads, num_kv_heads, head_size, num_blocks, block_size, dtype,
                          fp8, k_scale, v_scale, nullptr, 0, workspace, workspace_bytes, flags, stream);
    }
    return prefill_impl(who, out, query, kv_cache, block_tables, max_blocks_per_seq, cu_seqlens_q, kv_lens, num_seqs,
                        total_q, max_seqlen_q, scale, num_q_heads, num_kv_heads, head_size, num_blocks, block_size, dtype,
                        fp8, k_scale, v_scale, workspace, workspace_bytes, Sees::kAll, nullptr, 0, stream);
}

// Tree attention: the same choice, each with the masks.
int tree_impl(const char *who, void *out, const void *query, const void *kv_cache, const int32_t *block_tables,
              int max_blocks_per_seq, const int32_t *cu_seqlens_q, const int32_t *seq_lens, const int32_t *tree_masks,
              int mask_words, int num_seqs, int total_q, int max_seqlen_q, float scale, int num_q_heads, int num_kv_heads,
              int head_size, int num_blocks, int block_size, int dtype, bool fp8, float k_scale, float v_scale, void *workspace,
              size_t workspace_bytes, unsigned flags, pa_stream_t stream)
{
    if (flags & ~PA_DECODE_SHARED_BLOCKS)
        return set_error(PA_ERR_INVALID_ARG, "%s: unknown flags 0x%x", who, flags);
    bool empty = false;
    const int rc = check_call(who, out, query, kv_cache, block_tables, max_blocks_per_seq, cu_seqlens_q, seq_lens, num_seqs,
                              total_q, max_seqlen_q, scale, num_q_heads, num_kv_heads, head_size, num_blocks, block_size,
                              dtype, &empty);
    if (rc != PA_OK)
        return rc;
    if (max_seqlen_q > PA_MAX_TREE_NODES || mask_words < 1 || max_seqlen_q > 32LL * mask_words)
        return set_error(PA_ERR_INVALID_ARG, "%s: max_seqlen_q %d (at most %d, and 32 for each of %d mask words)", who,
                         max_seqlen_q, PA_MAX_TREE_NODES, mask_words);
    if (empty)
        return PA_OK;
    if (!tree_masks || (reinterpret_cast<uintptr_t>(tree_masks) & 3))
        return set_error(PA_ERR_INVALID_ARG, "%s: null or misaligned tree_masks", who);
    if (workspace && cross_rows_fit(num_seqs, max_seqlen_q, num_q_heads, num_kv_heads, block_size)) {
        if (reinterpret_cast<uintptr_t>(workspace) & 255)
            return set_error(PA_ERR_WORKSPACE, "%s: workspace at %p (256-byte aligned)", who, workspace);
        return cross_rows(who, out, query, kv_cache, block_tables, max_blocks_per_seq, cu_seqlens_q, seq_lens, num_seqs,
                          total_q, max_seqlen_q, scale, num_q_heads, num_kv_heads, head_size, num_blocks, block_size, dtype,
                          fp8, k_scale, v_scale, tree_masks, mask_words, workspace, workspace_bytes, flags, stream);
    }
    return prefill_impl(who, out, query, kv_cache, block_tables, max_blocks_per_seq, cu_seqlens_q, seq_lens, num_seqs,
                        total_q, max_seqlen_q, scale, num_q_heads, num_kv_heads, head_size, num_blocks, block_size, dtype,
                        fp8, k_scale, v_scale, workspace, workspace_bytes, Sees::kTree, tree_masks, mask_words, stream);
}

}  // namespace

extern "C" int pa_prefill(void *out, const void *query, const void *kv_cache, const int32_t *block_tables,
                          int max_blocks_per_seq, const int32_t *cu_seqlens_q, const int32_t *seq_lens,
                          int num_seqs, int total_q, int max_seqlen_q, float scale, int num_q_heads,
                          int num_kv_heads, int head_size, int num_blocks, int block_size, int dtype,
                          void *workspace, size_t workspace_bytes, pa_stream_t stream)
{
    return prefill_impl("pa_prefill", out, query, kv_cache, block_tables, max_blocks_per_seq, cu_seqlens_q,
                        seq_lens, num_seqs, total_q, max_seqlen_q, scale, num_q_heads, num_kv_heads, head_size,
                        num_blocks, block_size, dtype, false, 1.f, 1.f, workspace, workspace_bytes, Sees::kCausal, nullptr, 0, stream);
}

extern "C" int pa_prefill_fp8(void *out, const void *query, const void *kv_cache, const int32_t *block_tables,
                              int max_blocks_per_seq, const int32_t *cu_seqlens_q, const int32_t *seq_lens,
                              int num_seqs, int total_q, int max_seqlen_q, float scale, int num_q_heads,
                              int num_kv_heads, int head_size, int num_blocks, int block_size, int dtype,
                              float k_scale, float v_scale, void *workspace, size_t workspace_bytes,
                              pa_stream_t stream)
{
    if (!(std::isfinite(k_scale) && k_scale > 0.f && std::isfinite(v_scale) && v_scale > 0.f))
        return set_error(PA_ERR_INVALID_ARG, "pa_prefill_fp8: k_scale and v_scale must be finite and > 0");
    return prefill_impl("pa_prefill_fp8", out, query, kv_cache, block_tables, max_blocks_per_seq, cu_seqlens_q,
                        seq_lens, num_seqs, total_q, max_seqlen_q, scale, num_q_heads, num_kv_heads, head_size,
                        num_blocks, block_size, dtype, true, k_scale, v_scale, workspace, workspace_bytes, Sees::kCausal, nullptr, 0,
                        stream);
}

extern "C" int pa_prefill_workspace_size(int num_seqs, int max_seqlen_q, int num_q_heads, int num_kv_heads,
                                         int head_size, size_t *bytes)
{
    const char *who = "pa_prefill_workspace_size";
    if (!bytes)
        return set_error(PA_ERR_INVALID_ARG, "%s: null bytes", who);
    *bytes = 0;
    int rc = check_heads(who, num_q_heads, num_kv_heads, head_size);
    if (rc != PA_OK)
        return rc;
    if (num_seqs < 0 || max_seqlen_q < 0)
        return set_error(PA_ERR_INVALID_ARG, "%s: bad sizes", who);
    if (num_seqs == 0 || max_seqlen_q == 0)
        return PA_OK;
    int dev = 0, sms = 0;
    rc = current_sms(who, &dev, &sms);
    if (rc != PA_OK)
        return rc;
    *bytes = plan_launch(num_seqs, max_seqlen_q, num_q_heads, num_kv_heads, head_size, sms).split_bytes;
    return PA_OK;
}

extern "C" int pa_cross_attention(void *out, const void *query, const void *kv_cache, const int32_t *block_tables,
                                  int max_blocks_per_seq, const int32_t *cu_seqlens_q, const int32_t *kv_lens,
                                  int num_seqs, int total_q, int max_seqlen_q, float scale, int num_q_heads,
                                  int num_kv_heads, int head_size, int num_blocks, int block_size, int dtype,
                                  void *workspace, size_t workspace_bytes, unsigned flags, pa_stream_t stream)
{
    return cross_impl("pa_cross_attention", out, query, kv_cache, block_tables, max_blocks_per_seq, cu_seqlens_q, kv_lens,
                      num_seqs, total_q, max_seqlen_q, scale, num_q_heads, num_kv_heads, head_size, num_blocks, block_size,
                      dtype, false, 1.f, 1.f, workspace, workspace_bytes, flags, stream);
}

extern "C" int pa_cross_attention_fp8(void *out, const void *query, const void *kv_cache, const int32_t *block_tables,
                                      int max_blocks_per_seq, const int32_t *cu_seqlens_q, const int32_t *kv_lens,
                                      int num_seqs, int total_q, int max_seqlen_q, float scale, int num_q_heads,
                                      int num_kv_heads, int head_size, int num_blocks, int block_size, int dtype,
                                      float k_scale, float v_scale, void *workspace, size_t workspace_bytes,
                                      unsigned flags, pa_stream_t stream)
{
    if (!(std::isfinite(k_scale) && k_scale > 0.f && std::isfinite(v_scale) && v_scale > 0.f))
        return set_error(PA_ERR_INVALID_ARG, "pa_cross_attention_fp8: k_scale and v_scale must be finite and > 0");
    return cross_impl("pa_cross_attention_fp8", out, query, kv_cache, block_tables, max_blocks_per_seq, cu_seqlens_q,
                      kv_lens, num_seqs, total_q, max_seqlen_q, scale, num_q_heads, num_kv_heads, head_size, num_blocks,
                      block_size, dtype, true, k_scale, v_scale, workspace, workspace_bytes, flags, stream);
}

namespace {

int few_or_chunk_workspace(const char *who, bool tree, int num_seqs, int max_seqlen_q, int num_q_heads, int num_kv_heads,
                           int head_size, int block_size, int dtype, int cache_dtype, size_t *bytes)
{
    if (!bytes)
        return set_error(PA_ERR_INVALID_ARG, "%s: null bytes", who);
    *bytes = 0;
    if (dtype != PA_F16 && dtype != PA_BF16)
        return set_error(PA_ERR_UNSUPPORTED, "%s: dtype %d (want PA_F16 or PA_BF16)", who, dtype);
    if (cache_dtype != dtype && cache_dtype != PA_FP8_E4M3)
        return set_error(PA_ERR_UNSUPPORTED, "%s: cache_dtype %d (want dtype or PA_FP8_E4M3)", who, cache_dtype);
    if (block_size < kBoxTokens || block_size % kBoxTokens != 0)
        return set_error(PA_ERR_INVALID_ARG, "%s: block_size %d must be a positive multiple of 16", who, block_size);
    const int rc = check_heads(who, num_q_heads, num_kv_heads, head_size);
    if (rc != PA_OK)
        return rc;
    if (num_seqs > 0 && max_seqlen_q > 0 && cross_rows_fit(num_seqs, max_seqlen_q, num_q_heads, num_kv_heads, block_size))
        return cross_rows_workspace(num_seqs, max_seqlen_q, num_q_heads, num_kv_heads, head_size, dtype,
                                    cache_dtype == PA_FP8_E4M3, tree, bytes);
    return pa_prefill_workspace_size(num_seqs, max_seqlen_q, num_q_heads, num_kv_heads, head_size, bytes);
}

}  // namespace

extern "C" int pa_cross_attention_workspace_size(int num_seqs, int max_seqlen_q, int num_q_heads, int num_kv_heads,
                                                 int head_size, int block_size, int dtype, int cache_dtype, size_t *bytes)
{
    return few_or_chunk_workspace("pa_cross_attention_workspace_size", false, num_seqs, max_seqlen_q, num_q_heads, num_kv_heads,
                                  head_size, block_size, dtype, cache_dtype, bytes);
}

extern "C" int pa_tree_attention(void *out, const void *query, const void *kv_cache, const int32_t *block_tables,
                                 int max_blocks_per_seq, const int32_t *cu_seqlens_q, const int32_t *seq_lens,
                                 const int32_t *tree_masks, int mask_words, int num_seqs, int total_q, int max_seqlen_q,
                                 float scale, int num_q_heads, int num_kv_heads, int head_size, int num_blocks, int block_size,
                                 int dtype, void *workspace, size_t workspace_bytes, unsigned flags, pa_stream_t stream)
{
    return tree_impl("pa_tree_attention", out, query, kv_cache, block_tables, max_blocks_per_seq, cu_seqlens_q, seq_lens,
                     tree_masks, mask_words, num_seqs, total_q, max_seqlen_q, scale, num_q_heads, num_kv_heads, head_size,
                     num_blocks, block_size, dtype, false, 1.f, 1.f, workspace, workspace_bytes, flags, stream);
}

extern "C" int pa_tree_attention_fp8(void *out, const void *query, const void *kv_cache, const int32_t *block_tables,
                                     int max_blocks_per_seq, const int32_t *cu_seqlens_q, const int32_t *seq_lens,
                                     const int32_t *tree_masks, int mask_words, int num_seqs, int total_q, int max_seqlen_q,
                                     float scale, int num_q_heads, int num_kv_heads, int head_size, int num_blocks,
                                     int block_size, int dtype, float k_scale, float v_scale, void *workspace,
                                     size_t workspace_bytes, unsigned flags, pa_stream_t stream)
{
    if (!(std::isfinite(k_scale) && k_scale > 0.f && std::isfinite(v_scale) && v_scale > 0.f))
        return set_error(PA_ERR_INVALID_ARG, "pa_tree_attention_fp8: k_scale and v_scale must be finite and > 0");
    return tree_impl("pa_tree_attention_fp8", out, query, kv_cache, block_tables, max_blocks_per_seq, cu_seqlens_q, seq_lens,
                     tree_masks, mask_words, num_seqs, total_q, max_seqlen_q, scale, num_q_heads, num_kv_heads, head_size,
                     num_blocks, block_size, dtype, true, k_scale, v_scale, workspace, workspace_bytes, flags, stream);
}

extern "C" int pa_tree_attention_workspace_size(int num_seqs, int max_seqlen_q, int num_q_heads, int num_kv_heads,
                                                int head_size, int block_size, int dtype, int cache_dtype, size_t *bytes)
{
    return few_or_chunk_workspace("pa_tree_attention_workspace_size", true, num_seqs, max_seqlen_q, num_q_heads, num_kv_heads,
                                  head_size, block_size, dtype, cache_dtype, bytes);
}
