// int8.cuh -- device helpers of the 8-bit integer products: the tcgen05 integer
// MMA, its instruction descriptor, and the rounding of a row to 8 bits.
#pragma once
#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx.cuh"

namespace bffn {

// D[tmem] (+)= A[smem desc] * B[smem desc]^T, kind::i8 (int8 in, int32 out), K = 32
__device__ __forceinline__ void umma_i8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The same by a pair of blocks (cta_group::2): 256 rows of A and D, half in each block, and
// each block's half of B's rows; issued by the pair's first block.
__device__ __forceinline__ void umma_i8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// arrive on the mbarrier at this place in both blocks of the pair when every MMA of the
// pair that this thread issued so far is done
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}
// 2-D tiled load into this block's shared memory, its bytes counted on an mbarrier of either
// block of the pair (a shared::cluster address)
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* m, uint32_t cluster_bar, int c0, int c1,
                                                 uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        ".L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(cluster_bar), "r"(c0), "r"(c1), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// Instruction descriptor, kind::i8: A = B = signed 8 bits, D = int32, both K-major.
__host__ __device__ constexpr uint32_t idesc_i8_s32(int M, int N) {
    return (2u << 4)                                   // D format int32
           | (1u << 7)                                 // A format signed
           | (1u << 10)                                // B format signed
           | (static_cast<uint32_t>(N >> 3) << 17)     // N / 8
           | (static_cast<uint32_t>(M >> 4) << 24);    // M / 16
}

// A warp's wait for a barrier phase that it tested some time ago (`tested`: the test's
// result, so that its latency runs under other work); false after a timeout or abort.
__device__ __forceinline__ bool wait_tested(uint32_t tested, uint64_t* bar, uint32_t parity, uint64_t limit_ns,
                                            volatile int* abort, Ctl* ctl, int32_t detail) {
    if (__all_sync(0xffffffffu, tested != 0)) return true;
    return wait_bar_warp(bar, parity, limit_ns, abort, ctl, detail);
}

__device__ __forceinline__ int ld_shared_cluster_s32(uint32_t cluster_addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
    return v;
}

// --------------------------------------------------------------- workspace --
// The 8-bit calls keep nothing in a workspace but its status word, so they share one
// freely among themselves; one that a forward call keeps its counters in is not theirs (and
// a forward refuses one of theirs in the same way: its shape key differs).
constexpr unsigned long long kInt8Key = 0x3862697473ull | 1ull;

// What a thread of a call's first kernel reads of the control block at its start, so that
// the read runs beside its inputs' (waited for alone it cost a decode call 0.4 us).
struct Int8Gate {
    Ctl* ctl;    // nullptr: a call without a workspace
    int32_t status;
    unsigned long long key;
};
__device__ __forceinline__ Int8Gate int8_gate(Ctl* ctl) {
    Int8Gate g{ctl, 0, kInt8Key};
    if (ctl != nullptr) {
        g.status = __ldcg(&ctl->status);
        g.key = __ldcg(&ctl->shape_key);
    }
    return g;
}
// May this thread write?  Not after an earlier error, nor into a forward's workspace, which
// is recorded.  Threads may read the status while a dependent kernel records a wait that
// ran out, so they need not agree: no barrier follows, or the block decides together.
__device__ __forceinline__ bool int8_gate_open(const Int8Gate& g) {
    if (g.status != 0) return false;
    if (g.key == kInt8Key) return true;
    if (g.key == 0) {
        if (threadIdx.x == 0) claim_shape_key(g.ctl, kInt8Key);
        return true;
    }
    if (threadIdx.x == 0) record_error(g.ctl, kErrWorkspace, kShapeKey);
    return false;
}

// ------------------------------------------------- 8-bit rounding of a row --
// q = rint(127 v / amax), scale = amax / 127.  A row that is all zero (or below
// 2^-120, where 127 / amax would overflow) has q = 0 and scale 0; a row with an
// infinity or a NaN has scale NaN, so that what is computed from it shows it.
struct RowScale {
    float inv;      // 127 / amax, or 0
    float scale;    // amax / 127, or 0, or NaN
    float amax;
};
// amax_bits: the largest |v| of the row as bits (NaN above infinity above numbers)
__device__ __forceinline__ RowScale row_scale(uint32_t amax_bits) {
    RowScale r;
    r.amax = __uint_as_float(amax_bits);
    r.inv = 0.f;
    r.scale = 0.f;
    if (amax_bits >= 0x7f800000u) {
        r.scale = __uint_as_float(0x7fc00000u);
    } else if (amax_bits >= 0x03800000u) {   // 2^-120
        r.inv = 127.f / r.amax;
        r.scale = r.amax / 127.f;
    }
    return r;
}
// The product v * inv is off by less than 127 * 2^-22; a value that near the border of two
// whole numbers is divided again in 64 bits, so q is rint of the exact quotient.
__device__ __forceinline__ int quantize_exact(float v, const RowScale& r) {
    const float p = v * r.inv;
    float q = rintf(p);
    if (fabsf(fabsf(p - q) - 0.5f) < 1e-4f) q = (float)rint((double)v * 127.0 / (double)r.amax);
    return (int)q;
}
__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// The magnitude of the largest of 16 bytes of values, as bits of an fp32 (a bf16 is its
// upper half); NaN above infinity above numbers.
template <typename T>
__device__ __forceinline__ uint32_t chunk_max(uint32_t m, const uint4& u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2) m = __vmaxu2(m, w[i] & 0x7fff7fffu);   // (two running maxima)
        else m = max(m, w[i] & 0x7fffffffu);
    }
    return m;
}
template <typename T>
__device__ __forceinline__ uint32_t chunk_max_bits(uint32_t m) {
    return sizeof(T) == 2 ? max(m << 16, m & 0xffff0000u) : m;
}
template <typename T>
__device__ __forceinline__ float chunk_value(const uint4& u, int i) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (sizeof(T) == 2) return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    else return __uint_as_float(w[i]);
}

// 16 bytes of a row (V values) in 8 bits, packed.  v * inv is rounded by adding 1.5 * 2^23
// (the whole number is the sum's low byte); what was rounded off tells whether a value is
// near the border of two whole numbers, and such a chunk is done again exactly.  bf16
// values meet the border itself often (one in 256 where amax is a power of two), but
// 127 v - q amax is exact for them in fp32; fp32 values (one chunk in some hundred)
// are divided in 64 bits, in a function of its own so that it costs no registers here.
template <typename T>
__device__ __noinline__ uint2 quantize_chunk_exact(uint4 u, RowScale r) {
    constexpr int V = 16 / (int)sizeof(T);
    uint32_t p[2] = {0u, 0u};
#pragma unroll 1
    for (int i = 0; i < V; ++i)
        p[i >> 2] |= ((uint32_t)quantize_exact(chunk_value<T>(u, i), r) & 255u) << (8 * (i & 3));
    return make_uint2(p[0], p[1]);
}
template <typename T>
__device__ __forceinline__ uint2 quantize_chunk(const uint4& u, const RowScale& r) {
    constexpr int V = 16 / (int)sizeof(T);
    constexpr float kMagic = 12582912.f;
    uint32_t b[V];
    float worst = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float v = chunk_value<T>(u, i);
        const float t = fmaf(v, r.inv, kMagic);
        b[i] = __float_as_uint(t);
        worst = fmaxf(worst, fabsf(fmaf(v, r.inv, kMagic - t)));
    }
    // (inv is off by 2^-24 of itself: the product by 8e-6 at most)
    if (worst > 0.49998f) {
        if constexpr (sizeof(T) == 4) {
            return quantize_chunk_exact<T>(u, r);
        } else {
            const float down = r.amax > 1.f ? 0.00390625f : 1.f;   // (127 v stays finite, and exact)
            const float amax = r.amax * down, half = 0.5f * amax;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float q = __uint_as_float(b[i]) - kMagic;
                const float d = fmaf(-q, amax, 127.f * (chunk_value<T>(u, i) * down));
                // past the border, or on it with an odd number: the next one on d's side
                if (fabsf(d) > half || (fabsf(d) == half && (b[i] & 1u))) b[i] += d > 0.f ? 1u : ~0u;
            }
        }
    }
    uint32_t p[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < V / 4; ++i)
        p[i] = __byte_perm(__byte_perm(b[4 * i], b[4 * i + 1], 0x0040), __byte_perm(b[4 * i + 2], b[4 * i + 3], 0x0040),
                           0x5410);
    return make_uint2(p[0], p[1]);
}

// W threads (a multiple of 32; thread `t` of them, meeting at named barrier `bar` when
// they are more than a warp) round one row of K values.  C > 0: K values in whole
// 16-byte chunks, at most C * W of them, read once and kept in registers.  C == 0: any
// K, two passes.  red: a word per warp of the group.
template <typename T, int C>
__device__ __forceinline__ void quantize_row(const T* __restrict__ v, int K, int8_t* __restrict__ q, float* scale, int W,
                                             int t, int bar, uint32_t* red, const Int8Gate& gate) {
    constexpr int V = 16 / (int)sizeof(T);
    uint4 u[C > 0 ? C : 1];
    uint32_t m = 0;
    if constexpr (C > 0) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            u[c] = make_uint4(0u, 0u, 0u, 0u);
            if ((c * W + t) * V < K) u[c] = *reinterpret_cast<const uint4*>(v + (c * W + t) * V);
        }
#pragma unroll
        for (int c = 0; c < C; ++c) m = chunk_max<T>(m, u[c]);
        m = chunk_max_bits<T>(m);
    } else {
        for (int k = t; k < K; k += W) m = max(m, __float_as_uint(as_f32(v[k])) & 0x7fffffffu);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (W > 32) {
        if ((t & 31) == 0) red[t >> 5] = m;
        named_bar_sync(bar, W);
        for (int w = 0; w < W / 32; ++w) m = max(m, red[w]);
    }
    if (!int8_gate_open(gate)) return;   // (behind the last barrier)
    const RowScale r = row_scale(m);
    if (t == 0) *scale = r.scale;
    if constexpr (C > 0) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = (c * W + t) * V;
            if (k < K) {
                const uint2 p = r.inv != 0.f ? quantize_chunk<T>(u[c], r) : make_uint2(0u, 0u);
                if constexpr (V == 8) *reinterpret_cast<uint2*>(q + k) = p;
                else *reinterpret_cast<uint32_t*>(q + k) = p.x;
            }
        }
    } else {
        for (int k = t; k < K; k += W) q[k] = (int8_t)(r.inv != 0.f ? quantize_exact(as_f32(v[k]), r) : 0);
    }
}

// How a block of 256 threads rounds rows of K values: W threads a row, C chunks of 16
// bytes a thread (0: two passes).  Few rows are spread over more threads (what counts
// is the way through one row); many take fewer threads a row, four chunks each.
constexpr int kQThreads = 256;
struct QuantPlan {
    int lgW, C;    // W = 2^lgW
};
inline QuantPlan quantize_plan(int rows, int K, int elem_bytes) {
    const int V = 16 / elem_bytes;
    QuantPlan p{8, 0};
    if (K % V != 0 || K / V > 8 * kQThreads) return p;
    p.C = K / V > 4 * kQThreads ? 8 : (rows <= 296 && K / V <= 2 * kQThreads ? 2 : 4);
    p.lgW = 5;
    while ((p.C << p.lgW) < K / V) ++p.lgW;
    return p;
}

}  // namespace bffn
