// int8_linear.cu -- rows rounded to 8 bits, and the product of 8-bit integers with a
// scale for each token and each output channel on the sm_100a tensor cores.
//
//   q_t  = rint(127 x_t / amax_t),  s_t = amax_t / 127            (quantize kernel)
//   y[t, o] = s_t s_w[o] (sum_k q[t, k] W[o, k]) + bias[o]        (product kernel)
//
// The sums are exact: int8 x int8 into int32 (tcgen05 kind::i8), so the order of
// the K blocks, and how K is split, do not matter.  int32 -> fp32, the two scales
// and the bias are the only roundings before the one to y's type.
//
// Tiles.  128 output channels (M, the weight's rows) by N tokens (N = 16 .. 256):
// the weight is the operand that a small batch streams, so it fills the MMA's M
// whatever T is.  A pipeline stage is 128 bytes of K of both operands, or 256 (KP = 2)
// where K is whole 128-byte blocks: a TMA operation takes an SM's TMA unit about
// 0.15-0.27 us whatever it brings up to 32 KB, so fewer and larger ones.  TMA writes the
// 128-byte swizzle the MMA reads; K's tail and the rows behind O and T are zeros that it
// fills in.  (K = O = 4096: one token 8.0 -> 7.1 us with 256 bytes, weights 2.6 us.)
//
// Few tiles: a cluster of S blocks shares a tile, each multiplying a slice of K.  The
// int32 partial sums stay in each block's shared memory; after a cluster barrier
// each block adds N / S token columns over the S blocks.  Many tiles: one
// persistent block per SM, two accumulators in TMEM, so the epilogue of a tile runs
// under the MMAs of the next.
//
// Roles (384 threads): warp 0 loads, warp 1 issues the MMAs, warp 2 owns TMEM,
// warps 4-11 are the epilogue (a thread is one channel; two groups of four
// warps take alternate 16-column pieces).  The product kernel is a programmatic
// dependent of the quantize kernel: the weights' first tiles are loaded while that
// one still runs.
#include <cuda.h>
#include <cuda_runtime.h>

#include <mutex>

#include "int8.cuh"
#include "launch.h"

namespace bffn {

template <typename T, int C>
__global__ void __launch_bounds__(kQThreads) quantize_rows_kernel(const T* __restrict__ v, int rows, int K, int lgW,
                                                                  int8_t* __restrict__ q, float* __restrict__ scale,
                                                                  Ctl* ctl) {
    __shared__ uint32_t red[8];
    griddep_wait();
    griddep_launch_dependents();
    const Int8Gate gate = int8_gate(ctl);
    const int W = 1 << lgW, g = threadIdx.x >> lgW;   // the block's group of W threads
    const long long row = ((long long)blockIdx.x << (8 - lgW)) + g;
    if (row >= rows) return;
    quantize_row<T, C>(v + row * K, K, q + row * K, scale + row, W, threadIdx.x & (W - 1), 1 + g, red + (g << lgW >> 5),
                       gate);
}

namespace {
template <typename T>
cudaError_t launch_quantize_t(const T* v, int rows, int K, int8_t* q, float* scale, Ctl* ctl, cudaStream_t s) {
    const QuantPlan p = quantize_plan(rows, K, (int)sizeof(T));
    const int per = kQThreads >> p.lgW;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows + (long long)per - 1) / per));
    cfg.blockDim = dim3(kQThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (p.C == 0) return cudaLaunchKernelEx(&cfg, quantize_rows_kernel<T, 0>, v, rows, K, p.lgW, q, scale, ctl);
    if (p.C == 2) return cudaLaunchKernelEx(&cfg, quantize_rows_kernel<T, 2>, v, rows, K, p.lgW, q, scale, ctl);
    if (p.C == 4) return cudaLaunchKernelEx(&cfg, quantize_rows_kernel<T, 4>, v, rows, K, p.lgW, q, scale, ctl);
    return cudaLaunchKernelEx(&cfg, quantize_rows_kernel<T, 8>, v, rows, K, p.lgW, q, scale, ctl);
}
}  // namespace

cudaError_t launch_quantize_rows(const void* v, bool bf16, int rows, int K, int8_t* q, float* scale, Ctl* ctl,
                                 cudaStream_t s) {
    return bf16 ? launch_quantize_t(static_cast<const __nv_bfloat16*>(v), rows, K, q, scale, ctl, s)
                : launch_quantize_t(static_cast<const float*>(v), rows, K, q, scale, ctl, s);
}

namespace {

constexpr int kIlThreads = 384;
constexpr int kIlMaxStages = 12;
constexpr int kIlABytes = 128 * 128;          // weight tile: 128 rows x 128 int8
constexpr int kIlRing = 200 * 1024;           // shared memory of the stages

struct IlShared {
    uint64_t full[kIlMaxStages];
    uint64_t empty[kIlMaxStages];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint64_t mma_done;
    uint32_t tmem_base;
    volatile int abort;
    int refused;                          // an earlier error: written once, read behind named barrier 1
};
// warp 0 arrives there, the MMA warp and the epilogue wait: the block goes on, or does not, as one
constexpr int kIlAgree = 32 * (1 + 1 + 8);

__device__ __forceinline__ void il_put(float* y, float v) { *y = v; }
__device__ __forceinline__ void il_put(__nv_bfloat16* y, float v) { *y = __float2bfloat16_rn(v); }
__device__ __forceinline__ void il_put4(float* y, const float (&f)[4]) {
    *reinterpret_cast<float4*>(y) = make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void il_put4(__nv_bfloat16* y, const float (&f)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
    *reinterpret_cast<uint2*>(y) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

}  // namespace

// A stage's operand: KP blocks of 128 bytes of K of `rows` rows, one TMA operation.
template <int KP>
__device__ __forceinline__ void il_load(void* dst, const CUtensorMap* m, uint64_t* bar, int kb, int row, uint64_t pol) {
    if constexpr (KP == 1) tma_load_2d(dst, m, bar, kb * 128, row, pol);
    else tma_load_3d(dst, m, bar, 0, row, kb * KP, pol);
}

template <typename OutT, int KP>
__global__ void __launch_bounds__(kIlThreads, 1)
int8_linear_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                   const __grid_constant__ IlArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int N = a.N, S = a.S;
    constexpr int kA = KP * kIlABytes;
    const int b_tile = N * 128, stage_bytes = kA + KP * b_tile;
    IlShared& sh = *reinterpret_cast<IlShared*>(smem + (size_t)a.stages * stage_bytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = S > 1 ? (int)cluster_ctarank() : 0;
    const int first = S > 1 ? (int)cluster_id_x() : (int)blockIdx.x;
    const int step = (int)gridDim.x;   // (S > 1: a cluster has one tile)
    const int kb0 = a.kb_lo[rank], kb1 = a.kb_lo[rank + 1];
    const int tiles = a.tiles_o * a.tiles_t;

    if (threadIdx.x == 0) {
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.acc_full[i], 1);
            mbar_init(&sh.acc_empty[i], 8);
        }
        mbar_init(&sh.mma_done, 1);
        fence_mbar_init();
        sh.abort = 0;
        prefetch_tmap(&tm_w);
        prefetch_tmap(&tm_x);
    }
    if (warp == 2) {
        tmem_alloc(&sh.tmem_base, 2 * N);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_launch_dependents();
    const uint32_t tmem = sh.tmem_base;
    const uint64_t limit = a.wait_ns;

    bool refused = false;

    if (warp == 0) {
        // the first stages' weight tiles do not depend on the quantize kernel
        const int pre = first < tiles ? min(a.stages, kb1 - kb0) : 0;
        // (elect.sync, not lane 0: what one elected lane runs is issued at twice the rate)
        if (elect_one()) {
            const uint64_t pol = policy_evict_normal();
            const int to = first % a.tiles_o;
            for (int i = 0; i < pre; ++i) {
                mbar_arrive_expect_tx(&sh.full[i], (uint32_t)stage_bytes);
                il_load<KP>(smem + (size_t)i * stage_bytes, &tm_w, &sh.full[i], kb0 + i, to * 128, pol);
            }
        }
        __syncwarp();
        griddep_wait();
        refused = __shfl_sync(0xffffffffu, __ldcg(&a.ctl->status), 0) != 0;
        if (lane == 0) sh.refused = refused;
        named_bar_arrive(1, kIlAgree);
        if (elect_one()) {
            const uint64_t pol = policy_evict_normal();
            int st = 0;
            uint32_t ph = 0;
            bool stop = false;
            int issued = 0;
            for (int tile = first; tile < tiles && !stop; tile += step) {
                const int to = tile % a.tiles_o, tt = tile / a.tiles_o;
                for (int kb = kb0; kb < kb1; ++kb) {
                    uint8_t* sp = smem + (size_t)st * stage_bytes;
                    if (issued >= pre) {
                        // (refused: the stages begun are still completed, nobody reads them)
                        if (refused || !wait_bar(&sh.empty[st], ph ^ 1u, limit, &sh.abort, a.ctl, kWaitEmpty)) {
                            stop = true;
                            break;
                        }
                        mbar_arrive_expect_tx(&sh.full[st], (uint32_t)stage_bytes);
                        il_load<KP>(sp, &tm_w, &sh.full[st], kb, to * 128, pol);
                    }
                    il_load<KP>(sp + kA, &tm_x, &sh.full[st], kb, tt * N, pol);
                    ++issued;
                    if (++st == a.stages) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
            }
            // every load issued has landed before the block may end
            const int in_ring = min(issued, a.stages);
            for (int i = 0; i < in_ring; ++i) {
                st = st == 0 ? a.stages - 1 : st - 1;
                const int nth = (issued - 1 - i) / a.stages;   // how often the stage was filled before
                wait_bar_drain(&sh.full[st], (uint32_t)(nth & 1), limit, a.ctl);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        const uint32_t idesc = idesc_i8_s32(128, N);
        const uint64_t desc0 = sw128_kmajor_desc(smem_u32(smem));
        named_bar_sync(1, kIlAgree);
        refused = sh.refused != 0;
        if (elect_one()) {
            int st = 0, buf = 0;
            uint32_t ph = 0, bph = 0;
            bool ok = !refused;
            for (int tile = first; tile < tiles && ok; tile += step) {
                ok = wait_bar(&sh.acc_empty[buf], bph ^ 1u, limit, &sh.abort, a.ctl, kWaitAccEmpty);
                if (!ok) break;
                tc_fence_after();
                for (int kb = kb0; kb < kb1; ++kb) {
                    ok = wait_bar(&sh.full[st], ph, limit, &sh.abort, a.ctl, kWaitFullW);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t ad = desc0 + (uint64_t)((uint32_t)st * (uint32_t)stage_bytes >> 4);
                    const uint64_t bd = ad + (kA >> 4);
#pragma unroll
                    for (int h = 0; h < KP; ++h)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            umma_i8(tmem + (uint32_t)(buf * N), ad + h * (kIlABytes >> 4) + 2 * k,
                                    bd + (uint64_t)(h * (b_tile >> 4)) + 2 * k, idesc, kb > kb0 || h + k > 0);
                    umma_commit(&sh.empty[st]);
                    if (kb == kb1 - 1) umma_commit(&sh.acc_full[buf]);
                    if (++st == a.stages) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
                buf ^= 1;
                if (buf == 0) bph ^= 1u;
            }
            // no MMA is in flight when the accumulators are given back
            umma_commit(&sh.mma_done);
            wait_bar_drain(&sh.mma_done, 0u, limit, a.ctl);
        }
        __syncwarp();
    } else if (warp >= 4) {
        griddep_wait();   // the token scales
        named_bar_sync(1, kIlAgree);
        refused = sh.refused != 0;
        const int q = warp & 3, half = (warp - 4) >> 2, ch = q * 32 + lane;
        int buf = 0;
        uint32_t bph = 0;
        for (int tile = first; tile < tiles && !refused; tile += step) {
            const int to = tile % a.tiles_o, tt = tile / a.tiles_o;
            const int t0 = tt * N, o = to * 128 + ch;
            // lanes 0-15 hold the token scales of a piece's columns
            auto scales = [&](int c) {
                const int t = t0 + c + (lane & 15);
                return c < N && t < a.T ? __ldcg(a.sx + t) : 0.f;
            };
            float sx = S == 1 ? scales(half * 16) : 0.f;
            const float sw = o < a.O ? __ldg(a.sw + o) : 0.f;
            const float b = (a.bias != nullptr && o < a.O) ? __ldg(a.bias + o) : 0.f;
            if (!wait_bar_warp(&sh.acc_full[buf], bph, limit, &sh.abort, a.ctl, kWaitAccFull)) break;
            tc_fence_after();
            const uint32_t tacc = tmem + (uint32_t)(buf * N) + ((uint32_t)(q * 32) << 16);
            OutT* y = static_cast<OutT*>(a.y) + (size_t)t0 * a.O + o;
            if (S == 1) {
#pragma unroll 1
                for (int c = half * 16; c < N; c += 32) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x16(tacc + (uint32_t)c, v);
                    const float sx0 = sx;
                    sx = scales(c + 32);
                    tmem_ld_wait();
                    if (c + 32 >= N) {   // the group's last piece: its columns are in registers
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh.acc_empty[buf]);
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float st = __shfl_sync(0xffffffffu, sx0, i);
                        if (o < a.O && t0 + c + i < a.T)
                            il_put(y + (size_t)(c + i) * a.O, fmaf((float)(int)v[i] * sw, st, b));
                    }
                }
                if (half * 16 >= N) {   // no piece of 16 columns for this group
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.acc_empty[buf]);
                }
            } else {
                // this block's partial sums, [N][128] int32, over the stages (all read)
                int* part = reinterpret_cast<int*>(smem);
#pragma unroll 1
                for (int c = half * 16; c < N; c += 32) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x16(tacc + (uint32_t)c, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) part[(c + i) * 128 + ch] = (int)v[i];
                }
            }
            buf ^= 1;
            if (buf == 0) bph ^= 1u;
        }
    }
    if (S > 1) {
        // (every block of the cluster has the same tile: tiles == clusters)
        cluster_barrier_sync();
        if (warp >= 4 && first < tiles && !refused && sh.abort == 0) {
            // a warp adds a column at a time, a lane four channels of it over the S blocks
            const int to = first % a.tiles_o, tt = first / a.tiles_o;
            const int t0 = tt * N, o = to * 128 + lane * 4;
            float sw[4], bs[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sw[i] = o + i < a.O ? __ldg(a.sw + o + i) : 0.f;
                bs[i] = a.bias != nullptr && o + i < a.O ? __ldg(a.bias + o + i) : 0.f;
            }
            OutT* y = static_cast<OutT*>(a.y) + (size_t)t0 * a.O + o;
            const int c1 = min(N * (rank + 1) / S, a.T - t0);
            float st_next = 0.f;
            int c = N * rank / S + warp - 4;
            if (c < c1) st_next = __ldcg(a.sx + t0 + c);
#pragma unroll 1
            for (; c < c1; c += 8) {
                const float st = st_next;
                if (c + 8 < c1) st_next = __ldcg(a.sx + t0 + c + 8);
                const uint32_t off = smem_u32(smem) + (uint32_t)(c * 128 + lane * 4) * 4u;
                float4 u[8];   // (int32 bits; all blocks' sums in flight at once)
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    u[r] = r < S ? ld_shared_cluster_f4(mapa_shared(off, (uint32_t)r)) : make_float4(0.f, 0.f, 0.f, 0.f);
                int v[4] = {0, 0, 0, 0};
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    v[0] += __float_as_int(u[r].x);
                    v[1] += __float_as_int(u[r].y);
                    v[2] += __float_as_int(u[r].z);
                    v[3] += __float_as_int(u[r].w);
                }
                float f[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = fmaf((float)v[i] * sw[i], st, bs[i]);
                OutT* yc = y + (size_t)c * a.O;
                if ((a.O & 3) == 0) {   // (rows are then aligned to four values, and whole)
                    if (o < a.O) il_put4(yc, f);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (o + i < a.O) il_put(yc + i, f[i]);
                }
            }
        }
        cluster_barrier_sync_relaxed();   // no block leaves while its partial sums may be read
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) tmem_dealloc(tmem, 2 * N);
}

// Many tiles: a pair of blocks shares a tile of 256 channels x 256 tokens (cta_group::2).  Each
// block brings its 128 rows of W and half of the token rows, 32 KB a stage for the MMA work
// that takes a single block 48 KB, and has its 128 channels of all 256 tokens in its own
// TMEM.  L2's delivery is what bounds the single-block form (about 55 bytes a cycle and SM).
// The pair's first block issues the MMAs; the loads of both blocks are counted on its
// barriers, and finished MMAs are reported to both.  (Stages of 256 bytes of K, as above,
// measured 61.4 us against 60.1 with the rounding at 4096^3: three long stages for six.)
// 4096^3: the product alone 55 us (floor 42), the tensor pipe 61 % busy, 686 MB from L2;
// with the rounding 62 us in a burst, 71 us where the power cap holds the clock at 1680 MHz.
namespace {

constexpr int kIpStages = 6;
constexpr int kIpStage = 2 * kIlABytes;   // 128 rows of W, 128 token rows

struct IpShared {
    uint64_t full[kIpStages];             // first block: both blocks' loads of the stage (bytes)
    uint64_t empty[kIpStages];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];                // first block: both blocks' epilogue warps
    uint64_t mma_done;
    uint32_t tmem_base;
    volatile int abort;
};

}  // namespace

template <typename OutT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kIlThreads, 1)
int8_linear_pair_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                        const __grid_constant__ IlArgs a) {
    constexpr int N = 256;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    IpShared& sh = *reinterpret_cast<IpShared*>(smem + kIpStages * kIpStage);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();
    const int first = (int)cluster_id_x(), step = (int)gridDim.x >> 1;
    const int tiles = a.tiles_o * a.tiles_t;   // of 256 channels, 256 tokens

    if (threadIdx.x == 0) {
        for (int i = 0; i < kIpStages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.acc_full[i], 1);
            mbar_init(&sh.acc_empty[i], 16);
        }
        mbar_init(&sh.mma_done, 1);
        fence_mbar_init();
        sh.abort = 0;
        prefetch_tmap(&tm_w);
        prefetch_tmap(&tm_x);
    }
    if (warp == 2) tmem_alloc_pair(&sh.tmem_base, 2 * N);
    tc_fence_before();
    cluster_barrier_sync();   // barriers of both blocks are set up
    tc_fence_after();
    griddep_launch_dependents();
    const uint32_t tmem = sh.tmem_base;
    const uint64_t limit = a.wait_ns;

    if (warp == 0) {
        if (elect_one()) {
            const uint64_t pol = policy_evict_normal();
            int st = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            griddep_wait();
            if (__ldcg(&a.ctl->status) != 0) {   // an earlier error: no loads, so no sums and no y
                sh.abort = 1;
                ok = false;
            }
            const uint32_t full0 = mapa_shared(smem_u32(&sh.full[0]), 0u);   // the first block's
            for (int tile = first; tile < tiles && ok; tile += step) {
                const int o = (tile % a.tiles_o * 2 + rank) * 128, t = tile / a.tiles_o * N + rank * 128;
                for (int kb = 0; kb < a.KB; ++kb) {
                    ok = wait_bar(&sh.empty[st], ph ^ 1u, limit, &sh.abort, a.ctl, kWaitEmpty);
                    if (!ok) break;
                    uint8_t* sp = smem + st * kIpStage;
                    const uint32_t bar = full0 + 8u * (uint32_t)st;
                    // (the second block's bytes may be counted before they are expected: the phase
                    // ends with the arrival that expects them)
                    if (rank == 0) mbar_arrive_expect_tx(&sh.full[st], 2 * kIpStage);
                    tma_load_2d_pair(sp, &tm_w, bar, kb * 128, o, pol);
                    tma_load_2d_pair(sp + kIlABytes, &tm_x, bar, kb * 128, t, pol);
                    ++issued;
                    if (++st == kIpStages) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
            }
            // every load issued has landed before the pair may end: the first block waits for
            // both (the second is held by the closing cluster barrier)
            const int in_ring = rank == 0 ? min(issued, kIpStages) : 0;
            for (int i = 0; i < in_ring; ++i) {
                st = st == 0 ? kIpStages - 1 : st - 1;
                wait_bar_drain(&sh.full[st], (uint32_t)(((issued - 1 - i) / kIpStages) & 1), limit, a.ctl);
            }
            // after a timeout the blocks may have stopped at different stages, and loads of the
            // second one that the first does not expect cannot be waited for: give them time
            if (sh.abort && issued > 0) {
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
            }
        }
        __syncwarp();
    } else if (warp == 1 && rank == 0) {
        const uint32_t idesc = idesc_i8_s32(256, N);
        const uint64_t desc0 = sw128_kmajor_desc(smem_u32(smem));
        if (elect_one()) {
            int st = 0, buf = 0;
            uint32_t ph = 0, bph = 0;
            bool ok = true;
            for (int tile = first; tile < tiles && ok; tile += step) {
                ok = wait_bar_cluster(&sh.acc_empty[buf], bph ^ 1u, limit, &sh.abort, a.ctl, kWaitAccEmpty);
                if (!ok) break;
                for (int kb = 0; kb < a.KB; ++kb) {
                    ok = wait_bar(&sh.full[st], ph, limit, &sh.abort, a.ctl, kWaitFullW);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t ad = desc0 + (uint64_t)((uint32_t)(st * kIpStage) >> 4);
                    const uint64_t bd = ad + (kIlABytes >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_i8_pair(tmem + (uint32_t)(buf * N), ad + 2 * k, bd + 2 * k, idesc, kb > 0 || k > 0);
                    umma_commit_pair(&sh.empty[st]);
                    if (kb == a.KB - 1) umma_commit_pair(&sh.acc_full[buf]);
                    if (++st == kIpStages) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
                buf ^= 1;
                if (buf == 0) bph ^= 1u;
            }
            // no MMA is in flight when the accumulators are given back
            umma_commit_pair(&sh.mma_done);
            wait_bar_drain(&sh.mma_done, 0u, limit, a.ctl);
        }
        __syncwarp();
    } else if (warp >= 4) {
        griddep_wait();   // the token scales
        const int q = warp & 3, half = (warp - 4) >> 2, ch = q * 32 + lane;
        const uint32_t freed = mapa_shared(smem_u32(&sh.acc_empty[0]), 0u);   // (and the next 8 bytes)
        int buf = 0;
        uint32_t bph = 0;
        for (int tile = first; tile < tiles; tile += step) {
            const int t0 = tile / a.tiles_o * N, o = (tile % a.tiles_o * 2 + rank) * 128 + ch;
            // lanes 0-15 hold the token scales of a piece's columns
            auto scales = [&](int c) {
                const int t = t0 + c + (lane & 15);
                return c < N && t < a.T ? __ldcg(a.sx + t) : 0.f;
            };
            float sx = scales(half * 16);
            const float sw = o < a.O ? __ldg(a.sw + o) : 0.f;
            const float b = (a.bias != nullptr && o < a.O) ? __ldg(a.bias + o) : 0.f;
            if (!wait_bar_warp(&sh.acc_full[buf], bph, limit, &sh.abort, a.ctl, kWaitAccFull)) break;
            tc_fence_after();
            const uint32_t tacc = tmem + (uint32_t)(buf * N) + ((uint32_t)(q * 32) << 16);
            OutT* y = static_cast<OutT*>(a.y) + (size_t)t0 * a.O + o;
#pragma unroll 1
            for (int c = half * 16; c < N; c += 32) {
                uint32_t v[32];
                tmem_ld_32x32b_x16(tacc + (uint32_t)c, v);
                const float sx0 = sx;
                sx = scales(c + 32);
                tmem_ld_wait();
                if (c + 32 >= N) {   // the group's last piece: its columns are in registers
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(freed + 8u * (uint32_t)buf);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float st = __shfl_sync(0xffffffffu, sx0, i);
                    if (o < a.O && t0 + c + i < a.T)
                        il_put(y + (size_t)(c + i) * a.O, fmaf((float)(int)v[i] * sw, st, b));
                }
            }
            buf ^= 1;
            if (buf == 0) bph ^= 1u;
        }
    }
    tc_fence_before();
    cluster_barrier_sync();   // no block leaves while the pair's MMAs may read it or report to it
    tc_fence_after();
    if (warp == 2) tmem_dealloc_pair(tmem, 2 * N);
}

namespace {
size_t il_smem(const IlArgs& a) { return 1024 + (size_t)a.stages * a.KP * (kIlABytes + a.N * 128) + sizeof(IlShared); }

template <typename OutT, int KP>
cudaError_t launch_il(const IlArgs& a, const CUtensorMap* maps, int grid, cudaStream_t s) {
    const size_t smem = il_smem(a);
    auto kern = int8_linear_kernel<OutT, KP>;
    static SmemOptIn opt_in;
    cudaError_t e = opt_in(kern);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kIlThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)a.S;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = a.S > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, maps[0], maps[1], a);
}
}  // namespace

// [S]: how many clusters of S blocks of these kernels (one block per SM) can be resident at
// once on the current device; 0 if unknown.  (On a B200 that is 148, 74, 45, 33, 26, 22, 15, 15 for
// S = 1 .. 8: an SM that is left over in its GPC holds no cluster.)
const int* int8_cluster_capacity() {
    static int cache[65][9];
    static std::once_flag once[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cache[64];   // all 0
    std::call_once(once[dev], [dev]() {
        auto kern = int8_linear_kernel<float, 1>;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) != cudaSuccess) return;
        for (int c = 1; c <= 8; ++c) {
            cudaLaunchAttribute at[1];
            at[0].id = cudaLaunchAttributeClusterDimension;
            at[0].val.clusterDim.x = (unsigned)c;
            at[0].val.clusterDim.y = 1;
            at[0].val.clusterDim.z = 1;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3((unsigned)c);
            cfg.blockDim = dim3(kIlThreads);
            cfg.dynamicSmemBytes = 200 * 1024;
            cfg.attrs = at;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&cache[dev][c], kern, &cfg) != cudaSuccess) {
                cudaGetLastError();
                cache[dev][c] = 0;
            }
        }
    });
    return cache[dev];
}

// Tile width and K split.  A tile of N tokens costs about 2 N cycles of MMA for each
// 128 bytes of K, or the time of its (128 + N) * 128 bytes at about 48 bytes per cycle
// and SM, and some 1500 cycles of start and epilogue (more where a cluster meets);
// the pair (N, S) with the smallest time over all waves is taken.
// Pairs of blocks (tiles of 256 x 256) bring 64 KB for what single blocks' 256 x 256 takes 96.
void int8_linear_plan(int T, int K, int O, int sms, int* N_out, int* S_out, bool* pair_out) {
    const int KB = (K + 127) / 128, tiles_o = (O + 127) / 128;
    const int* const fit = int8_cluster_capacity();
    double best = 1e30;
    *N_out = 256;
    *S_out = 1;
    for (int N = 16; N <= 256; N *= 2) {
        const long long tiles = (long long)tiles_o * ((T + N - 1) / N);
        for (int S = 1; S <= 8; ++S) {
            if (S > 1 && (N > 128 || tiles > fit[S] || KB / S < 2)) continue;
            const double waves = S > 1 ? 1.0 : (double)((tiles + sms - 1) / sms);
            const double mma = 2.0 * N, load = (128.0 + N) * 128.0 / 48.0;
            const double per = (double)((KB + S - 1) / S) * (mma > load ? mma : load);
            const double cost = waves * (per + N * 4.0) + 1500.0 + (S > 1 ? 1200.0 + N / S * 80.0 : 0.0);
            if (cost < best) {
                best = cost;
                *N_out = N;
                *S_out = S;
            }
        }
    }
    const int pairs = fit[2];
    *pair_out = false;
    if (pairs > 0) {
        const long long tiles = (long long)((O + 255) / 256) * ((T + 255) / 256);
        const double waves = (double)((tiles + pairs - 1) / pairs);
        const double cost = waves * (KB * (256.0 * 128.0 / 48.0) + 1024.0) + 2500.0;
        if (cost < best) {
            *N_out = 256;
            *S_out = 1;
            *pair_out = true;
        }
    }
}

namespace {
template <typename OutT>
cudaError_t launch_ip(const IlArgs& a, const CUtensorMap* maps, int grid, cudaStream_t s) {
    auto kern = int8_linear_pair_kernel<OutT>;
    static SmemOptIn opt_in;
    cudaError_t e = opt_in(kern);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kIlThreads);
    cfg.dynamicSmemBytes = 1024 + (size_t)kIpStages * kIpStage + sizeof(IpShared);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, maps[0], maps[1], a);
}
}  // namespace

cudaError_t launch_int8_linear(IlArgs a, const CUtensorMap* maps, bool bf16_out, int sms, cudaStream_t s) {
    if (a.pair) {
        const int tiles = a.tiles_o * a.tiles_t, fit = int8_cluster_capacity()[2];
        const int grid = 2 * (tiles < fit ? tiles : fit);
        return bf16_out ? launch_ip<__nv_bfloat16>(a, maps, grid, s) : launch_ip<float>(a, maps, grid, s);
    }
    const int stage = a.KP * (kIlABytes + a.N * 128);
    a.stages = kIlRing / stage < kIlMaxStages ? kIlRing / stage : kIlMaxStages;
    const int tiles = a.tiles_o * a.tiles_t;
    for (int r = 0; r <= a.S; ++r) a.kb_lo[r] = (int)((long long)a.KB * r / a.S);
    const int grid = a.S > 1 ? tiles * a.S : (tiles < sms ? tiles : sms);
    if (a.KP == 2)
        return bf16_out ? launch_il<__nv_bfloat16, 2>(a, maps, grid, s) : launch_il<float, 2>(a, maps, grid, s);
    return bf16_out ? launch_il<__nv_bfloat16, 1>(a, maps, grid, s) : launch_il<float, 1>(a, maps, grid, s);
}

}  // namespace bffn
