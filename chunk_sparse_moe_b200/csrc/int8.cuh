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

// Instruction descriptor, kind::i8: A = B = signed 8 bits, D = int32, both K-major.
__host__ __device__ constexpr uint32_t idesc_i8_s32(int M, int N) {
    return (2u << 4)                                   // D format int32
           | (1u << 7)                                 // A format signed
           | (1u << 10)                                // B format signed
           | (static_cast<uint32_t>(N >> 3) << 17)     // N / 8
           | (static_cast<uint32_t>(M >> 4) << 24);    // M / 16
}

__device__ __forceinline__ int ld_shared_cluster_s32(uint32_t cluster_addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
    return v;
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
__device__ __forceinline__ uint32_t pack4_i8(int a, int b, int c, int d) {
    return (uint32_t)(a & 255) | (uint32_t)(b & 255) << 8 | (uint32_t)(c & 255) << 16 | (uint32_t)d << 24;
}

__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// 16 bytes of a row as fp32 values
__device__ __forceinline__ void load_chunk(const __nv_bfloat16* p, float (&f)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = *reinterpret_cast<const __nv_bfloat162*>(&w[i]);
        f[2 * i] = __low2float(h);
        f[2 * i + 1] = __high2float(h);
    }
}
__device__ __forceinline__ void load_chunk(const float* p, float (&f)[4]) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    f[0] = u.x;
    f[1] = u.y;
    f[2] = u.z;
    f[3] = u.w;
}
__device__ __forceinline__ void store_q(int8_t* p, const int (&q)[8]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack4_i8(q[0], q[1], q[2], q[3]), pack4_i8(q[4], q[5], q[6], q[7]));
}
__device__ __forceinline__ void store_q(int8_t* p, const int (&q)[4]) {
    *reinterpret_cast<uint32_t*>(p) = pack4_i8(q[0], q[1], q[2], q[3]);
}

// The block's largest |v| as bits; red: one word per warp, free again on return.
__device__ __forceinline__ uint32_t block_max_bits(uint32_t v, uint32_t* red) {
    v = __reduce_max_sync(0xffffffffu, v);
    const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    __syncthreads();
    uint32_t m = 0;
    for (int w = 0; w < nw; ++w) m = max(m, red[w]);
    __syncthreads();
    return m;
}

constexpr int kQChunks = 4;   // 16-byte chunks a thread keeps in registers

// One block rounds one row of K values.  VEC: K values in whole 16-byte chunks,
// K <= chunk values * kQChunks * threads, read once; otherwise two passes.
template <typename T, bool VEC>
__device__ __forceinline__ void quantize_row(const T* __restrict__ v, int K, int8_t* __restrict__ q, float* scale,
                                             uint32_t* red) {
    constexpr int V = 16 / (int)sizeof(T);
    const int tid = threadIdx.x, nt = blockDim.x;
    if constexpr (VEC) {
        float f[kQChunks][V];
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < kQChunks; ++c) {
            const int k = (c * nt + tid) * V;
            if (k < K) {
                load_chunk(v + k, f[c]);
#pragma unroll
                for (int i = 0; i < V; ++i) m = max(m, __float_as_uint(f[c][i]) & 0x7fffffffu);
            }
        }
        const RowScale r = row_scale(block_max_bits(m, red));
        if (tid == 0) *scale = r.scale;
#pragma unroll
        for (int c = 0; c < kQChunks; ++c) {
            const int k = (c * nt + tid) * V;
            if (k < K) {
                int o[V];
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] = r.inv != 0.f ? quantize_exact(f[c][i], r) : 0;
                store_q(q + k, o);
            }
        }
    } else {
        uint32_t m = 0;
        for (int k = tid; k < K; k += nt) m = max(m, __float_as_uint(as_f32(v[k])) & 0x7fffffffu);
        const RowScale r = row_scale(block_max_bits(m, red));
        if (tid == 0) *scale = r.scale;
        for (int k = tid; k < K; k += nt) q[k] = (int8_t)(r.inv != 0.f ? quantize_exact(as_f32(v[k]), r) : 0);
    }
}

// Threads of a block that rounds rows of K values, and whether one pass serves.
inline int quantize_threads(int K, int elem_bytes) {
    const int chunks = (K * elem_bytes + 15) / 16;
    const int t = ((chunks + 1) / 2 + 31) / 32 * 32;   // two chunks a thread where the row is long enough
    return t < 64 ? 64 : (t > 256 ? 256 : t);
}
inline bool quantize_one_pass(int K, int elem_bytes) {
    const int V = 16 / elem_bytes;
    return K % V == 0 && K <= V * kQChunks * quantize_threads(K, elem_bytes);
}

}  // namespace bffn
