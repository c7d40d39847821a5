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
// 62-bit fraction of a turn (pa_rope_plan) and multiplied by the integer
// position modulo 2^64: the wrap-around is exact, and for any 32-bit position
// the product is off by at most 2^-31 turns, where an fp32 product would be off
// by a radian at a position of 10^7. The upper 32 bits as a signed number are
// the angle in [-1, 1) half turns; rounded to fp32 for the sines it is off by
// up to 2^-26 turns (1e-7 radians), far below a 16-bit rounding of the result.
//
// HBM-bound: per token the q row is read and written, the k and v rows read
// and written once; the sines are computed once per unit, not per head.
// Measured (GB300, of the 6.80 TB/s copy rate): 8192 tokens of 40/40 heads of
// 128, 503 MB in 80 us (6.3 TB/s, 92 %); 16383 tokens of 32/8 heads, 396 MB in
// 61 us (6.5 TB/s, 95 %); 5001 tokens of 32/8 heads into an FP8 cache, 113 MB
// in 22 us (5.1 TB/s, 75 %: a fifth of it is the launch and the first loads).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "../../include/pa.h"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

__device__ int g_rope_error;  // PA_DEVERR_* bits of the rotary kernels

namespace {

constexpr int kRopeWarps = 8;                         // that turn and store
constexpr int kRopeThreads = 32 * (kRopeWarps + 2);   // and one that copies, one for the sines
constexpr int kRopeMaxStages = 8, kRopeMaxTokens = 8;  // of the ring, of a unit
// A unit's rows at most (but a group of heads at least), and a CTA's ring, two
// CTAs an SM: about 80 KB of rows in flight an SM. Both less and more is
// slower: the units in flight are the stretch of memory that is read and
// written at a time (measured at 16383 tokens of 32 + 2 x 8 heads, rings of
// 24 / 36 / 40 / 57 / 96 KB: 108 / 71 / 61 / 69 / 73 us).
constexpr int kRopeUnitBytes = 12288, kRopeSmemBytes = 40960;
constexpr int kRopeMaxDims = 512;  // that turn
constexpr int kRopeMaxAxes = 4;    // the axis is kept in a plan word's low 2 bits

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
    int units;
    int parts, tokens_per_unit, heads_per_unit;  // units a token, or tokens a unit
    int stages, stage_bytes, sines_at;  // a stage: the unit's rows, then each token's rot / 2 cosines and sines
    float k_scale, v_scale, k_inv, v_inv;  // inv: 1 / scale, 0 where quotients are to be divided
};

// Two fp32 lanes in a register pair: one packed instruction for both.
__device__ __forceinline__ uint64_t pair(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ float2 lanes(uint64_t x)
{
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(x));
    return f;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// Eight elements as four fp32 pairs, and back.
struct F8 {
    uint64_t p[4];
};

template <bool BF16>
__device__ __forceinline__ F8 unpack8(const uint4 x)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    F8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = BF16 ? make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u))
                              : unpack2<false>(w[i]);
        r.p[i] = pair(f.x, f.y);
    }
    return r;
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const F8 &x)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = lanes(x.p[i]);
        w[i] = pack2<BF16>(f.x, f.y);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint4 negated(const uint4 x)  // eight 16-bit elements
{
    return make_uint4(x.x ^ 0x80008000u, x.y ^ 0x80008000u, x.z ^ 0x80008000u, x.w ^ 0x80008000u);
}

// E4M3 codes (nearest even, saturating) of the IEEE fp32 quotients of eight
// values by the scale, as pa_reshape_and_cache_fp8 rounds; nx holds the values
// NEGATED. With inv = 1 / scale correctly rounded, Markstein's theorem
// ("Computation of elementary functions on the IBM RISC System/6000
// processor", 1990) gives the correctly rounded quotient as
// q - (q scale - x) inv, q = x inv, as long as the residual is exact. It is
// for scale within 2^+-64 and |x / scale| >= 2^-12; smaller quotients have
// code 0 of their sign whatever their last bits are (the residual of a zero is
// taken with the sign that leaves -0 alone). q is held to 2^24 so that an
// infinite x stays one instead of becoming NaN; all such quotients saturate.
// Other scales (inv 0) are divided, which takes about three times the
// instructions.
__device__ __forceinline__ uint2 codes8(const F8 &nx, float scale, float inv)
{
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 r;
        if (inv != 0.f) {
            const uint64_t ninv = pair(-inv, -inv);
            const float2 q0 = lanes(mul2(nx.p[i], ninv));
            const uint64_t q = pair(fmaxf(fminf(q0.x, 0x1p24f), -0x1p24f), fmaxf(fminf(q0.y, 0x1p24f), -0x1p24f));
            r = lanes(fma2(fma2(q, pair(scale, scale), nx.p[i]), ninv, q));
        } else {
            const float2 n = lanes(nx.p[i]);
            r = make_float2(__fdiv_rn(-n.x, scale), __fdiv_rn(-n.y, scale));
        }
        asm("{\n\t.reg .b16 r;\n\tcvt.rn.satfinite.e4m3x2.f32 r, %1, %2;\n\tcvt.u32.u16 %0, r;\n\t}"
            : "=r"(c[i])
            : "f"(r.y), "f"(r.x));
    }
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}

struct RopeBars {
    uint64_t full[kRopeMaxStages], empty[kRopeMaxStages];
    int slot[kRopeMaxStages][kRopeMaxTokens];  // of the unit's tokens, -1 where no K and V are written
};

// Persistent CTAs over units: a unit is a few tokens, a token, or
// heads_per_unit of its heads (q, then k, then v heads, counted through). One
// warp brings the units' rows into a ring of shared-memory stages by bulk
// copies, so that the bytes in flight do not depend on registers; another
// computes the tokens' sines into the stage meanwhile; the others turn the
// heads and store.
//
// A lane of those holds one place of a head: 16 bytes of it (adjacent pairs),
// or two times 16 bytes that lie rot / 2 apart, or of the dimensions that
// pass; `per` lanes a head and 32 / per heads side by side make a group, and
// the warps take the groups of all units in turn.
// MANY: several tokens a unit.
template <bool BF16, bool FP8, bool ADJ, bool MANY>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_and_cache_kernel(const RopeParams p)
{
    constexpr int kPairs = ADJ ? 4 : 8;  // of a lane
    constexpr int kVecs = ADJ ? 1 : 2;   // 16-byte vectors of a lane
    extern __shared__ __align__(128) uint8_t rope_smem[];
    __shared__ RopeBars bars;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = smem_addr(rope_smem);
    if (threadIdx.x == 0) {
        for (int st = 0; st < p.stages; ++st) {
            mbar_init(smem_addr(&bars.full[st]), 2);  // the copies' bytes, the sines
            mbar_init(smem_addr(&bars.empty[st]), kRopeWarps);
        }
        fence_barrier_init();
    }
    __syncthreads();
    // Launched with a programmatic dependency: nothing is read before the
    // preceding kernel (which may write the slots) is done, and only then may
    // the next one start, so that what it may read early is older still.
    grid_dependency_wait();
    grid_launch_dependents();

    const int hv = p.head_vecs, rv = p.rot_vecs, hq = p.num_q_heads, hk = hq + p.num_kv_heads, heads = hk + p.num_kv_heads;
    const int pairs = rv * 4, tokens = MANY ? p.tokens_per_unit : 1;
    // Unit u: tokens t0 .. t0 + tokens - 1 (those below num_tokens), heads from h0 on.
    auto unit_at = [&](int u, int &t0, int &h0) {
        const int k = p.parts == 1 ? u : u / p.parts;
        t0 = k * tokens;
        h0 = (u - k * p.parts) * p.heads_per_unit;
    };
    const int grid = gridDim.x;
    // From a unit to this CTA's next without a division.
    const int t_step = (p.parts == 1 ? grid : grid / p.parts) * tokens, h_step = (p.parts == 1 ? 0 : grid % p.parts) * p.heads_per_unit;
    const int h_end = p.parts * p.heads_per_unit;
    auto next_unit = [&](int &t0, int &h0) {
        t0 += t_step;
        h0 += h_step;
        if (h0 >= h_end) {
            h0 -= h_end;
            t0 += tokens;
        }
    };
    const int window = 32 / tokens;  // units whose tokens' indexes a warp loads at a time, a token a lane
    if (warp == kRopeWarps) {
        // ---------------------------------------------------------- copies
        // The slot of this lane's token in the window of units from u on.
        auto window_slot = [&](int u) {
            const int mine = u + (lane / tokens) * grid;
            if (lane >= window * tokens || mine >= p.units)
                return -1;
            int t0, h0;
            unit_at(mine, t0, h0);
            const int t = t0 + lane % tokens;
            return t < p.num_tokens ? p.slots[t] : -1;
        };
        int slot = -1, slot_next = window_slot(blockIdx.x);
        int st = 0, ahead = 0;
        uint32_t used = 0;  // rounds of the ring behind this stage
        int t0, h0;
        unit_at(blockIdx.x, t0, h0);
        for (int u = blockIdx.x; u < p.units; u += grid, next_unit(t0, h0)) {
            if (ahead == 0) {
                slot = slot_next;
                slot_next = window_slot(u + window * grid);
                if (slot >= p.num_slots) {
                    rope_raise(PA_DEVERR_SLOT);
                    slot = -1;
                }
            }
            const int j = lane - ahead * tokens;  // this lane's token of the unit
            const bool mine = j >= 0 && j < tokens && t0 + j < p.num_tokens;
            const int h1 = min(h0 + p.heads_per_unit, slot >= 0 ? heads : hq), n = mine ? max(h1 - h0, 0) : 0;
            const uint32_t full = smem_addr(&bars.full[st]), data = base + st * p.stage_bytes;
            if (used > 0 && !__all_sync(kFull, mbar_wait(smem_addr(&bars.empty[st]), (used - 1) & 1))) {
                if (lane == 0)
                    rope_raise(PA_DEVERR_TIMEOUT);
                return;  // the other warps wait (bounded) for what is in flight
            }
            uint32_t bytes = (uint32_t)(n * hv) * 16u;
            if (j >= 0 && j < tokens)
                bars.slot[st][j] = slot;
            if constexpr (MANY) {
                __syncwarp();
                bytes = __reduce_add_sync(kFull, bytes);
            }
            if (j == 0)
                mbar_expect_tx(full, bytes);
            if constexpr (MANY)
                __syncwarp();
            if (n > 0) {
                fence_proxy_async();  // the stage's last reads, before it is written again
                const int t = t0 + j;
                const uint32_t row_at = data + (uint32_t)(j * p.heads_per_unit * hv) * 16u;
                auto load = [&](const void *row, long long stride, int a, int b, int from) {  // heads [a, b) of the unit's
                    if (a < b)
                        bulk_load(row_at + (uint32_t)((a - h0) * hv) * 16u,
                                  static_cast<const uint4 *>(row) + t * stride + (long long)(a - from) * hv,
                                  (uint32_t)((b - a) * hv) * 16u, full);
                };
                load(p.q, p.q_stride, h0, min(h1, hq), 0);
                load(p.k, p.k_stride, max(h0, hq), min(h1, hk), hq);
                load(p.v, p.v_stride, max(h0, hk), h1, hk);
            }
            __syncwarp();
            if (++ahead == window)
                ahead = 0;
            if (++st == p.stages) {
                st = 0;
                ++used;
            }
        }
        return;
    }
    if (warp > kRopeWarps) {
        // ----------------------------------------------------------- sines
        uint64_t words[kRopeMaxDims / 64];  // a lane's plan words
#pragma unroll
        for (int k = 0; k < kRopeMaxDims / 64; ++k)
            words[k] = lane + 32 * k < pairs ? p.plan[lane + 32 * k] : 0;
        int pos[kRopeMaxAxes], pos_next[kRopeMaxAxes] = {0, 0, 0, 0};  // as the slots above
        auto window_pos = [&](int u) {
            const int mine = u + (lane / tokens) * grid;
            if (lane >= window * tokens || mine >= p.units)
                return;
            int t0, h0;
            unit_at(mine, t0, h0);
            const int t = t0 + lane % tokens;
#pragma unroll
            for (int a = 0; a < kRopeMaxAxes; ++a)
                if (a < p.num_axes && t < p.num_tokens)
                    pos_next[a] = p.positions[a * p.pos_stride + t];
        };
        window_pos(blockIdx.x);
        int st = 0, ahead = 0;
        uint32_t used = 0;
        for (int u = blockIdx.x; u < p.units; u += grid) {
            if (ahead == 0) {
#pragma unroll
                for (int a = 0; a < kRopeMaxAxes; ++a)
                    pos[a] = pos_next[a];
                window_pos(u + window * grid);
            }
            if (used > 0 && !__all_sync(kFull, mbar_wait(smem_addr(&bars.empty[st]), (used - 1) & 1))) {
                if (lane == 0)
                    rope_raise(PA_DEVERR_TIMEOUT);
                return;
            }
            float *cs = reinterpret_cast<float *>(rope_smem + st * p.stage_bytes + p.sines_at), *sn = cs + pairs;
            for (int j = 0; j < tokens; ++j, cs += 2 * pairs, sn += 2 * pairs) {
                int at[kRopeMaxAxes];
#pragma unroll
                for (int a = 0; a < kRopeMaxAxes; ++a)
                    at[a] = __shfl_sync(kFull, pos[a], ahead * tokens + j);
#pragma unroll
                for (int k = 0; k < kRopeMaxDims / 64; ++k) {
                    const int e = lane + 32 * k;
                    if (e < pairs) {
                        const int axis = min((int)(words[k] & 3u), p.num_axes - 1);
                        const long long x = axis == 0 ? at[0] : axis == 1 ? at[1] : axis == 2 ? at[2] : at[3];
                        const uint64_t turn = (uint64_t)x * (words[k] & ~3ull);
                        sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, sn + e, cs + e);
                    }
                }
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_addr(&bars.full[st]));
            if (++ahead == window)
                ahead = 0;
            if (++st == p.stages) {
                st = 0;
                ++used;
            }
        }
        return;
    }

    // ---------------------------------------------------- turn and store
    using Out = typename std::conditional<FP8, uint2, uint4>::type;
    const long long kv_row = (long long)p.num_kv_heads * hv;
    // Places of a head: those that turn, then those that pass.
    const int turning = rv / kVecs, rest = hv - rv, passing = (rest + kVecs - 1) / kVecs, places = turning + passing;
    const int segs = (places + 31) / 32, per = min(places, 32), side = 32 / per;
    const int h_in = lane / per, in = lane - h_in * per;
    int next = warp;  // this warp's next group, counted from the unit's first
    int st = 0;
    uint32_t phase = 0;
    int t0, first;
    unit_at(blockIdx.x, t0, first);
    for (int un = blockIdx.x; un < p.units; un += grid, next_unit(t0, first)) {
        if (!__all_sync(kFull, mbar_wait(smem_addr(&bars.full[st]), phase))) {
            if (lane == 0)
                rope_raise(PA_DEVERR_TIMEOUT);
            return;
        }
        const int count = min(p.heads_per_unit, heads - first);  // heads of the unit
        const int across = (count + side - 1) / side, groups = across * segs;  // of a token
        for (int j = 0; j < tokens; ++j, next -= groups) {  // next stays this warp's turn from token to token
            const int t = t0 + j, slot = bars.slot[st][j];
            const int n = t < p.num_tokens ? min(count, (slot >= 0 ? heads : hq) - first) : 0;
            const uint32_t data = base + st * p.stage_bytes + (uint32_t)(j * p.heads_per_unit * hv) * 16u;
            const uint32_t sines = base + st * p.stage_bytes + p.sines_at + (uint32_t)(j * pairs) * 8u;
            uint4 *q_out = static_cast<uint4 *>(p.q_out) + t * p.q_out_stride;
            Out *k_out = static_cast<Out *>(p.kv) + slot * kv_row, *v_out = k_out + p.num_slots * kv_row;
            for (; next < groups; next += kRopeWarps) {
                const int seg = segs == 1 ? 0 : next / across;
                const int h = (next - seg * across) * side + h_in;  // of the unit
                const int u = seg * 32 + in;
                if (h_in >= side || h >= n || u >= places)
                    continue;
                const bool turns = u < turning;
                const int v0 = turns ? u : rv + (u - turning), v1 = turns ? turning + u : v0 + passing;
                const bool two = !ADJ && v1 < hv;  // the second may be missing among those that pass
                const int head = first + h;
                const bool turn = turns && head < hk, code = FP8 && head >= hq;
                uint4 a[kVecs];
                a[0] = lds128(data + (uint32_t)(h * hv + v0) * 16u);
                if constexpr (!ADJ)
                    a[1] = two ? lds128(data + (uint32_t)(h * hv + v1) * 16u) : make_uint4(0u, 0u, 0u, 0u);
                if (code) {  // codes8 takes negated values
#pragma unroll
                    for (int c = 0; c < kVecs; ++c)
                        a[c] = negated(a[c]);
                }
                F8 y[kVecs];
#pragma unroll
                for (int c = 0; c < kVecs; ++c)
                    y[c] = unpack8<BF16>(a[c]);
                if (turn) {
                    float cs[kPairs], sn[kPairs];
#pragma unroll
                    for (int e = 0; e < kPairs; e += 4) {
                        const uint4 c4 = lds128(sines + (uint32_t)(u * kPairs + e) * 4u);
                        const uint4 s4 = lds128(sines + (uint32_t)(pairs + u * kPairs + e) * 4u);
                        const uint32_t cw[4] = {c4.x, c4.y, c4.z, c4.w}, sw[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                        for (int f = 0; f < 4; ++f) {
                            cs[e + f] = __uint_as_float(cw[f]);
                            sn[e + f] = __uint_as_float(sw[f]);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if constexpr (ADJ) {
                            // (x0, x1) (c, c) + (x1, x0) (-s, s)
                            const float2 x = lanes(y[0].p[e]);
                            y[0].p[e] = fma2(y[0].p[e], pair(cs[e], cs[e]), mul2(pair(x.y, x.x), pair(-sn[e], sn[e])));
                        } else {
                            const uint64_t x = y[0].p[e], z = y[1].p[e], c = pair(cs[2 * e], cs[2 * e + 1]);
                            y[0].p[e] = fma2(x, c, mul2(z, pair(-sn[2 * e], -sn[2 * e + 1])));
                            y[1].p[e] = fma2(z, c, mul2(x, pair(sn[2 * e], sn[2 * e + 1])));
                        }
                    }
                }
                const long long row = (long long)(head < hq ? head : head < hk ? head - hq : head - hk) * hv;
                if (code) {
                    uint2 *to = reinterpret_cast<uint2 *>((head < hk ? k_out : v_out) + row);
                    const float scale = head < hk ? p.k_scale : p.v_scale, inv = head < hk ? p.k_inv : p.v_inv;
                    to[v0] = codes8(y[0], scale, inv);
                    if constexpr (!ADJ)
                        if (two)
                            to[v1] = codes8(y[1], scale, inv);
                } else {
                    uint4 *to = head < hq ? q_out + row : reinterpret_cast<uint4 *>((head < hk ? k_out : v_out) + row);
                    to[v0] = turn ? pack8<BF16>(y[0]) : a[0];
                    if constexpr (!ADJ)
                        if (two)
                            to[v1] = turn ? pack8<BF16>(y[1]) : a[1];
                }
            }
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(smem_addr(&bars.empty[st]));
        if (++st == p.stages) {
            st = 0;
            phase ^= 1;
        }
    }
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The current device and its SM count (cached per device).
int rope_device(const char *who, int *dev, int *sms)
{
    static std::mutex mu;
    static int count[64] = {};
    cudaError_t e = cudaGetDevice(dev);
    std::lock_guard<std::mutex> lock(mu);
    *sms = e == cudaSuccess && *dev < 64 ? count[*dev] : 0;
    if (e == cudaSuccess && *sms <= 0) {
        e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev);
        if (e == cudaSuccess && *dev < 64)
            count[*dev] = *sms;
    }
    return e == cudaSuccess && *sms > 0 ? PA_OK : set_error(PA_ERR_CUDA, "%s: device: %s", who, cudaGetErrorString(e));
}

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
    if (num_tokens > (1 << 30))
        return set_error(PA_ERR_UNSUPPORTED, "%s: too many tokens (%d)", who, num_tokens);
    if (head_size <= 0 || head_size % 8 != 0 || head_size > 1024)
        return set_error(PA_ERR_UNSUPPORTED, "%s: head_size %d (want a multiple of 8, at most 1024)", who, head_size);
    if (rot_dim <= 0 || rot_dim % 16 != 0 || rot_dim > head_size || rot_dim > kRopeMaxDims)
        return set_error(PA_ERR_UNSUPPORTED, "%s: rot_dim %d (want a multiple of 16, at most head_size and %d)", who, rot_dim,
                         kRopeMaxDims);
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
    auto inverse = [](float scale) { return scale >= 0x1p-64f && scale <= 0x1p64f ? 1.f / scale : 0.f; };
    prm.k_inv = inverse(k_scale);
    prm.v_inv = inverse(v_scale);
#define PA_ROPE_INSTANCES(ADJ, MANY)                                                \
    reinterpret_cast<const void *>(&rope_and_cache_kernel<false, false, ADJ, MANY>),    \
        reinterpret_cast<const void *>(&rope_and_cache_kernel<true, false, ADJ, MANY>), \
        reinterpret_cast<const void *>(&rope_and_cache_kernel<false, true, ADJ, MANY>), \
        reinterpret_cast<const void *>(&rope_and_cache_kernel<true, true, ADJ, MANY>)
    static const void *const kernels[16] = {PA_ROPE_INSTANCES(false, false), PA_ROPE_INSTANCES(true, false),
                                            PA_ROPE_INSTANCES(false, true), PA_ROPE_INSTANCES(true, true)};
#undef PA_ROPE_INSTANCES
    int dev = 0, sms = 0;
    int rc = rope_device(who, &dev, &sms);
    if (rc != PA_OK)
        return rc;
    // Units: a token, in equal parts if its rows are longer than a unit's, or
    // if there are too few tokens for the CTAs (not below a group for each
    // warp); several tokens if they are short and there are plenty (measured
    // at 64703 tokens of 16/4 heads of 64: 126 us one at a time, 98 us four).
    const int heads = num_q_heads + 2 * num_kv_heads, head_bytes = head_size * 2;
    const int vecs = adjacent ? 1 : 2, places = rot_dim / 8 / vecs + ((head_size - rot_dim) / 8 + vecs - 1) / vecs;
    const int side = places < 32 ? 32 / places : 1;
    int parts = std::max(1, (heads * head_bytes + kRopeUnitBytes - 1) / kRopeUnitBytes);
    const long long wanted = (2LL * sms + num_tokens - 1) / num_tokens;
    const int most = std::max(parts, heads / (side * kRopeWarps));
    parts = (int)std::min<long long>(std::max<long long>(parts, wanted), most);
    parts = std::min(parts, heads);
    prm.heads_per_unit = ((heads + parts - 1) / parts + side - 1) / side * side;
    prm.parts = (heads + prm.heads_per_unit - 1) / prm.heads_per_unit;
    const int rows = prm.heads_per_unit * head_bytes, sines = rot_dim * 4;
    prm.tokens_per_unit = 1;
    if (prm.parts == 1)
        prm.tokens_per_unit = std::max(1, std::min({kRopeMaxTokens, kRopeUnitBytes / rows, num_tokens / (8 * sms)}));
    const long long units = ((long long)num_tokens + prm.tokens_per_unit - 1) / prm.tokens_per_unit * prm.parts;
    if (units > (1LL << 30))
        return set_error(PA_ERR_UNSUPPORTED, "%s: too many tokens (%d)", who, num_tokens);
    prm.units = (int)units;
    prm.sines_at = prm.tokens_per_unit * rows;
    prm.stage_bytes = (prm.sines_at + prm.tokens_per_unit * sines + 127) & ~127;
    prm.stages = std::max(1, std::min(kRopeMaxStages, kRopeSmemBytes / prm.stage_bytes));
    const int smem = prm.stages * prm.stage_bytes;
    const int variant = (prm.tokens_per_unit > 1 ? 8 : 0) + (adjacent ? 4 : 0) + (fp8 ? 2 : 0) + (dtype == PA_BF16 ? 1 : 0);
    const void *fn = kernels[variant];
    // Allow the largest ring once per kernel and device, so that a call being
    // captured into a CUDA graph makes no attribute call.
    {
        static std::mutex mu;
        static bool raised[16][64] = {};
        std::lock_guard<std::mutex> lock(mu);
        if (dev >= 64 || !raised[variant][dev]) {
            cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kRopeSmemBytes);
            if (e != cudaSuccess)
                return set_error(PA_ERR_CUDA, "%s: cudaFuncSetAttribute: %s", who, cudaGetErrorString(e));
            if (dev < 64)
                raised[variant][dev] = true;
        }
    }
    void *args[] = {&prm};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min(prm.units, 2 * sms));
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
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
