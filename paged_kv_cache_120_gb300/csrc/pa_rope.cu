// pa_rope_and_cache: rotary positions on this step's queries and keys, and
// the write of the keys and values into the cache by slot, in one pass.
//
// A head's first rot dimensions are rot / 2 pairs (x1, x2); pair i turns by
// the angle pos[axis(i)] * f_i:
//
//   (x1, x2) -> (x1 cos - x2 sin, x1 sin + x2 cos)
//
// with the pairs (i, i + rot / 2) or (2 i, 2 i + 1); the other dimensions pass.
// The write by slot is [book] chapter 4's §4.4.3 / §4.5 step 1, as in
// pa_reshape_and_cache.
//
// Angles. Only the fraction of a turn matters, so f_i / 2 pi is kept as a
// 64-bit fraction of a turn (pa_rope_plan) and multiplied by the integer
// position modulo 2^64: the wrap-around is exact, and for any 32-bit position
// the angle is off by at most 2^-32 turns, where an fp32 product would be off
// by a radian at a position of 10^7. The upper 32 bits as a signed number are
// the angle in [-1, 1) half turns.
//
// HBM-bound: per token the q row is read and written, the k and v rows read
// and written once; the sines are computed once per token, not per head.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "../../include/pa.h"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

__device__ int g_rope_error;  // PA_DEVERR_* bits of the rotary kernels

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxPairs = 256;  // rot <= 512
constexpr int kRopeMaxAxes = 4;     // the axis is kept in a plan word's low 2 bits

__device__ __forceinline__ void rope_raise(int bit) { atomicOr(&g_rope_error, bit); }

struct RopeParams {
    void *q_out;
    const void *q, *k, *v;
    void *kv;
    const int32_t *slots, *positions;
    const uint64_t *plan;
    long long q_out_stride, q_stride, k_stride, v_stride;  // 8-element vectors per token
    long long pos_stride;                                  // entries per axis
    long long num_slots;
    int num_tokens, num_q_heads, num_kv_heads, head_vecs, rot_vecs, num_axes;
    float k_scale, v_scale;
};

struct F8 {
    float f[8];
};

template <bool BF16>
__device__ __forceinline__ F8 unpack8(const uint4 x)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    F8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2<BF16>(w[i]);
        r.f[2 * i] = f.x;
        r.f[2 * i + 1] = f.y;
    }
    return r;
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const F8 &x)
{
    return make_uint4(pack2<BF16>(x.f[0], x.f[1]), pack2<BF16>(x.f[2], x.f[3]), pack2<BF16>(x.f[4], x.f[5]),
                      pack2<BF16>(x.f[6], x.f[7]));
}

// Eight values to E4M3 codes of value / scale (IEEE fp32 division, nearest
// even, saturating), as pa_reshape_and_cache_fp8 rounds.
__device__ __forceinline__ uint2 codes8(const F8 &x, float scale)
{
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("{\n\t.reg .b16 r;\n\tcvt.rn.satfinite.e4m3x2.f32 r, %1, %2;\n\tcvt.u32.u16 %0, r;\n\t}"
            : "=r"(c[i])
            : "f"(__fdiv_rn(x.f[2 * i + 1], scale)), "f"(__fdiv_rn(x.f[2 * i], scale)));
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// Sine and cosine of pair `word`'s angle at the token's positions.
__device__ __forceinline__ float2 turn_of(uint64_t word, const int32_t *positions, long long stride, int num_axes, int t)
{
    const int axis = min((int)(word & 3u), num_axes - 1);
    const long long pos = positions[axis * stride + t];
    const uint64_t frac = (uint64_t)pos * (word & ~3ull);
    float s, c;
    sincospif((float)(int32_t)(frac >> 32) * 0x1p-31f, &s, &c);
    return make_float2(c, s);
}

// One CTA per token.
template <bool BF16, bool FP8, bool ADJ>
__global__ void __launch_bounds__(kRopeThreads) rope_and_cache_kernel(const RopeParams p)
{
    __shared__ __align__(16) float s_cos[kRopeMaxPairs], s_sin[kRopeMaxPairs];
    const int t = blockIdx.x;
    // Launched with a programmatic dependency: nothing is read before the
    // preceding kernel (which may write the slots) is done, and only then may
    // the next one start, so that what it may read early is older still.
    grid_dependency_wait();
    grid_launch_dependents();
    for (int i = threadIdx.x; i < p.rot_vecs * 4; i += kRopeThreads) {
        const float2 cs = turn_of(p.plan[i], p.positions, p.pos_stride, p.num_axes, t);
        s_cos[i] = cs.x;
        s_sin[i] = cs.y;
    }
    const long long slot = p.slots[t];
    const bool write = slot >= 0 && slot < p.num_slots;
    if (slot >= p.num_slots && threadIdx.x == 0)
        rope_raise(PA_DEVERR_SLOT);
    __syncthreads();
    const int hv = p.head_vecs, rv = p.rot_vecs, half = rv / 2;
    const long long kv_row = (long long)p.num_kv_heads * hv;
    const uint4 *q = static_cast<const uint4 *>(p.q) + t * p.q_stride, *k = static_cast<const uint4 *>(p.k) + t * p.k_stride,
                *v = static_cast<const uint4 *>(p.v) + t * p.v_stride;
    uint4 *q_out = static_cast<uint4 *>(p.q_out) + t * p.q_out_stride;
    using Out = typename std::conditional<FP8, uint2, uint4>::type;
    Out *k_out = static_cast<Out *>(p.kv) + slot * kv_row, *v_out = k_out + p.num_slots * kv_row;
    auto put_k = [&](long long i, const F8 &x) {
        if constexpr (FP8)
            k_out[i] = codes8(x, p.k_scale);
        else
            k_out[i] = pack8<BF16>(x);
    };
    // Units of a head: rotated vectors (in pairs, unless the pairs are
    // adjacent), then those that pass.
    const int per_head = ADJ ? hv : half + (hv - rv);
    const int heads = p.num_q_heads + (write ? p.num_kv_heads : 0);
    for (int i = threadIdx.x; i < heads * per_head; i += kRopeThreads) {
        const int h = i / per_head, u = i - h * per_head;
        const bool is_q = h < p.num_q_heads;
        const long long at = (long long)(is_q ? h : h - p.num_q_heads) * hv;
        const uint4 *src = is_q ? q : k;
        if constexpr (ADJ) {
            F8 x = unpack8<BF16>(src[at + u]);
            if (u < rv) {
                F8 y;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float c = s_cos[4 * u + e], s = s_sin[4 * u + e];
                    y.f[2 * e] = x.f[2 * e] * c - x.f[2 * e + 1] * s;
                    y.f[2 * e + 1] = x.f[2 * e] * s + x.f[2 * e + 1] * c;
                }
                x = y;
            }
            if (is_q)
                q_out[at + u] = pack8<BF16>(x);
            else
                put_k(at + u, x);
        } else if (u < half) {
            const F8 a = unpack8<BF16>(src[at + u]), b = unpack8<BF16>(src[at + half + u]);
            F8 y, z;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float c = s_cos[8 * u + e], s = s_sin[8 * u + e];
                y.f[e] = a.f[e] * c - b.f[e] * s;
                z.f[e] = a.f[e] * s + b.f[e] * c;
            }
            if (is_q) {
                q_out[at + u] = pack8<BF16>(y);
                q_out[at + half + u] = pack8<BF16>(z);
            } else {
                put_k(at + u, y);
                put_k(at + half + u, z);
            }
        } else {
            const int w = rv + (u - half);
            const uint4 x = src[at + w];
            if (is_q)
                q_out[at + w] = x;
            else
                put_k(at + w, unpack8<BF16>(x));
        }
    }
    if (write)
        for (int i = threadIdx.x; i < kv_row; i += kRopeThreads) {
            if constexpr (FP8)
                v_out[i] = codes8(unpack8<BF16>(v[i]), p.v_scale);
            else
                v_out[i] = v[i];
        }
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int rope_impl(const char *who, void *query_out, const void *query, const void *key, const void *value, void *kv_cache,
              const int32_t *slot_mapping, const int32_t *positions, int num_axes, long long position_stride,
              const uint64_t *plan, int rot_dim, int adjacent, int num_tokens, long long query_out_stride,
              long long query_stride, long long key_stride, long long value_stride, int num_q_heads, int num_kv_heads,
              int head_size, int num_blocks, int block_size, int dtype, bool fp8, float k_scale, float v_scale,
              pa_stream_t stream)
{
    if (dtype != PA_F16 && dtype != PA_BF16)
        return set_error(PA_ERR_UNSUPPORTED, "%s: dtype %d (want PA_F16 or PA_BF16)", who, dtype);
    if (num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads > 65535 || num_kv_heads > 65535 ||
        num_blocks <= 0 || block_size < 16 || block_size % 16 != 0)
        return set_error(PA_ERR_INVALID_ARG, "%s: bad sizes", who);
    if (head_size <= 0 || head_size % 8 != 0 || head_size > 1024)
        return set_error(PA_ERR_UNSUPPORTED, "%s: head_size %d (want a multiple of 8, at most 1024)", who, head_size);
    if (rot_dim <= 0 || rot_dim % 16 != 0 || rot_dim > head_size || rot_dim > 2 * kRopeMaxPairs)
        return set_error(PA_ERR_UNSUPPORTED, "%s: rot_dim %d (want a multiple of 16, at most head_size and %d)", who, rot_dim,
                         2 * kRopeMaxPairs);
    if (num_axes < 1 || num_axes > kRopeMaxAxes || (num_axes > 1 && position_stride < num_tokens))
        return set_error(PA_ERR_INVALID_ARG, "%s: num_axes %d (1 to %d), position_stride %lld (at least num_tokens)", who,
                         num_axes, kRopeMaxAxes, position_stride);
    const long long q_row = (long long)num_q_heads * head_size, kv_row = (long long)num_kv_heads * head_size;
    if (query_out_stride < q_row || query_stride < q_row || key_stride < kv_row || value_stride < kv_row ||
        ((query_out_stride | query_stride | key_stride | value_stride) & 7))
        return set_error(PA_ERR_INVALID_ARG, "%s: a token stride is shorter than its row or no multiple of 8", who);
    if ((long long)num_blocks * block_size > 0x7fffffffLL)
        return set_error(PA_ERR_INVALID_ARG, "%s: num_blocks * block_size does not fit an int32 slot", who);
    if (num_tokens == 0)
        return PA_OK;
    if (!query_out || !query || !key || !value || !kv_cache || !slot_mapping || !positions || !plan)
        return set_error(PA_ERR_INVALID_ARG, "%s: null pointer argument", who);
    if (!aligned(query_out, 16) || !aligned(query, 16) || !aligned(key, 16) || !aligned(value, 16) || !aligned(kv_cache, 16) ||
        !aligned(slot_mapping, 4) || !aligned(positions, 4) || !aligned(plan, 8))
        return set_error(PA_ERR_INVALID_ARG, "%s: misaligned pointer (rows and pool 16 B, plan 8 B)", who);
    if (query_out == query && query_out_stride != query_stride)
        return set_error(PA_ERR_INVALID_ARG, "%s: in place, query_out_stride must equal query_stride", who);

    RopeParams prm;
    prm.q_out = query_out;
    prm.q = query;
    prm.k = key;
    prm.v = value;
    prm.kv = kv_cache;
    prm.slots = slot_mapping;
    prm.positions = positions;
    prm.plan = plan;
    prm.q_out_stride = query_out_stride / 8;
    prm.q_stride = query_stride / 8;
    prm.k_stride = key_stride / 8;
    prm.v_stride = value_stride / 8;
    prm.pos_stride = position_stride;
    prm.num_slots = (long long)num_blocks * block_size;
    prm.num_tokens = num_tokens;
    prm.num_q_heads = num_q_heads;
    prm.num_kv_heads = num_kv_heads;
    prm.head_vecs = head_size / 8;
    prm.rot_vecs = rot_dim / 8;
    prm.num_axes = num_axes;
    prm.k_scale = k_scale;
    prm.v_scale = v_scale;
    static const void *const kernels[8] = {
        reinterpret_cast<const void *>(&rope_and_cache_kernel<false, false, false>),
        reinterpret_cast<const void *>(&rope_and_cache_kernel<true, false, false>),
        reinterpret_cast<const void *>(&rope_and_cache_kernel<false, true, false>),
        reinterpret_cast<const void *>(&rope_and_cache_kernel<true, true, false>),
        reinterpret_cast<const void *>(&rope_and_cache_kernel<false, false, true>),
        reinterpret_cast<const void *>(&rope_and_cache_kernel<true, false, true>),
        reinterpret_cast<const void *>(&rope_and_cache_kernel<false, true, true>),
        reinterpret_cast<const void *>(&rope_and_cache_kernel<true, true, true>)};
    void *args[] = {&prm};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_tokens);
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelExC(&cfg, kernels[(adjacent ? 4 : 0) + (fp8 ? 2 : 0) + (dtype == PA_BF16 ? 1 : 0)], args);
    if (e != cudaSuccess)
        return set_error(PA_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
    return PA_OK;
}

}  // namespace

int rope_take_device_error(int *bits)
{
    int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_rope_error, sizeof(int));
    if (e == cudaSuccess)
        e = cudaMemcpyToSymbol(g_rope_error, &zero, sizeof(int));
    *bits = e == cudaSuccess ? v : 0;
    return (int)e;
}

}  // namespace pa

using namespace pa;

extern "C" int pa_rope_plan(const double *inv_freq, const int32_t *pair_axes, int num_pairs, uint64_t *plan)
{
    if (num_pairs < 0 || (num_pairs > 0 && (!inv_freq || !plan)))
        return set_error(PA_ERR_INVALID_ARG, "pa_rope_plan: null pointer argument or num_pairs %d", num_pairs);
    for (int i = 0; i < num_pairs; ++i) {
        if (!(std::fabs(inv_freq[i]) <= 4294967296.0))
            return set_error(PA_ERR_INVALID_ARG, "pa_rope_plan: inv_freq[%d] is not within +-2^32", i);
        if (pair_axes && (pair_axes[i] < 0 || pair_axes[i] >= kRopeMaxAxes))
            return set_error(PA_ERR_INVALID_ARG, "pa_rope_plan: pair_axes[%d] = %d outside [0, %d)", i, pair_axes[i],
                             kRopeMaxAxes);
    }
    for (int i = 0; i < num_pairs; ++i) {
        // f / 2 pi as an unevaluated sum (1 / 2 pi to 106 bits, the product's
        // rounding error by fma), each part reduced to a fraction of a turn
        // and added modulo 2^64.
        constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
        const double f = inv_freq[i], p = f * kHi, e = std::fma(f, kHi, -p) + f * kLo;
        auto fraction = [](double x) -> uint64_t {  // of |x|, exact to 2^-64, with x's sign
            const double a = std::fabs(x), r = a - std::floor(a);
            const uint64_t w = (uint64_t)std::ldexp(r, 64);
            return x < 0 ? 0 - w : w;
        };
        // 62 bits of the fraction, rounded; the axis takes the low two.
        plan[i] = ((fraction(p) + fraction(e) + 2) & ~3ull) | (uint64_t)(pair_axes ? pair_axes[i] : 0);
    }
    return PA_OK;
}

extern "C" int pa_rope_and_cache(void *query_out, const void *query, const void *key, const void *value, void *kv_cache,
                                 const int32_t *slot_mapping, const int32_t *positions, int num_axes,
                                 int64_t position_stride, const uint64_t *plan, int rot_dim, int adjacent, int num_tokens,
                                 int64_t query_out_stride, int64_t query_stride, int64_t key_stride, int64_t value_stride,
                                 int num_q_heads, int num_kv_heads, int head_size, int num_blocks, int block_size, int dtype,
                                 pa_stream_t stream)
{
    return rope_impl("pa_rope_and_cache", query_out, query, key, value, kv_cache, slot_mapping, positions, num_axes,
                     position_stride, plan, rot_dim, adjacent, num_tokens, query_out_stride, query_stride, key_stride,
                     value_stride, num_q_heads, num_kv_heads, head_size, num_blocks, block_size, dtype, false, 1.f, 1.f,
                     stream);
}

extern "C" int pa_rope_and_cache_fp8(void *query_out, const void *query, const void *key, const void *value, void *kv_cache,
                                     const int32_t *slot_mapping, const int32_t *positions, int num_axes,
                                     int64_t position_stride, const uint64_t *plan, int rot_dim, int adjacent, int num_tokens,
                                     int64_t query_out_stride, int64_t query_stride, int64_t key_stride,
                                     int64_t value_stride, int num_q_heads, int num_kv_heads, int head_size, int num_blocks,
                                     int block_size, int dtype, float k_scale, float v_scale, pa_stream_t stream)
{
    if (!(std::isfinite(k_scale) && k_scale > 0.f && std::isfinite(v_scale) && v_scale > 0.f))
        return set_error(PA_ERR_INVALID_ARG, "pa_rope_and_cache_fp8: k_scale and v_scale must be finite and > 0");
    return rope_impl("pa_rope_and_cache_fp8", query_out, query, key, value, kv_cache, slot_mapping, positions, num_axes,
                     position_stride, plan, rot_dim, adjacent, num_tokens, query_out_stride, query_stride, key_stride,
                     value_stride, num_q_heads, num_kv_heads, head_size, num_blocks, block_size, dtype, true, k_scale,
                     v_scale, stream);
}
