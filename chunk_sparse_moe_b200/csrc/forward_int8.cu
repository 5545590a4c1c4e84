// forward_int8.cu -- the expert sum of the layer in 8-bit integers on the sm_100a
// tensor cores (tcgen05 kind::i8, int32 sums).
//
// For every token t and every expert e with g[t,e] != 0:
//   (xq_t, sx_t)   = x_t rounded to 8 bits
//   z[j]           = sx_t s_in[e,j] (sum_k xq_t[k] W_in[e,j,k]) + b_in[e,j]
//   h              = z / (1 + exp(-z))                       (Swish)
//   (hq, sh)       = h rounded to 8 bits, one scale per (token, expert)
//   y_t[o]        += g sh s_out[e,o] (sum_j hq[j] W_out[e,o,j]) + g b_out[e,o]
// Both integer sums are exact.  The scales differ from expert to expert, so the sum
// over experts runs in fp32, experts ascending (within a block's share, the
// shares in order): two calls give the same bits.
//
// Only tokens that use an expert are computed for it ("pairs"), so the work is that
// of the pairs whatever the length; the weights of an expert that no token uses are
// not read.
//
//   prepare    : the tokens' 8-bit rows; per expert the ascending list of its tokens
//                and, at every 32nd token, how many came before
//   experts_in : tiles of one expert x up to N of its tokens, all of d_e; x rows are
//                gathered by TMA (four rows an operation) straight into the MMA's
//                layout.  The tile holds whole rows of h, so the epilogue finds
//                their scales and writes 8-bit h.  Few tiles: a cluster's blocks
//                split d_h and add their int32 sums through distributed shared memory.
//   experts_out: a block owns TT consecutive tokens x 128 output channels as fp32
//                sums in shared memory and walks the experts; a token tile's tokens
//                are neighbours in every expert's list, so h comes in plain boxes of
//                16 rows.  Each int32 result column is scaled and added to its
//                token's row.  Few tiles: a cluster's blocks share the experts and
//                add their fp32 rows in rank order.
// The three kernels are programmatic dependents of one another.
#include <cuda.h>
#include <cuda_runtime.h>

#include "int8.cuh"
#include "launch.h"

namespace bffn {

namespace {

// ------------------------------------------------------------------ prepare --
// Blocks 0 .. E-1 list an expert's tokens, block E + t rounds token t.
constexpr int kPrepBatch = 8;   // gates a thread has in flight

template <bool VEC>
__global__ void __launch_bounds__(256) int8_prepare_kernel(const __nv_bfloat16* __restrict__ x,
                                                           const float* __restrict__ gates, int T, int d_h, int E,
                                                           const X8Bufs w) {
    __shared__ uint32_t red[8];
    griddep_wait();
    griddep_launch_dependents();
    if ((int)blockIdx.x >= E) {
        const int t = blockIdx.x - E;
        quantize_row<__nv_bfloat16, VEC>(x + (size_t)t * d_h, d_h, w.xq + (size_t)t * d_h, w.sx + t, red);
        return;
    }
    const int e = blockIdx.x, nt = blockDim.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nw = nt >> 5;
    int32_t* list = w.list + (size_t)e * w.Tcap;
    int32_t* tpos = w.tpos + (size_t)e * (w.C32 + 1);
    int base = 0;   // tokens listed so far
    for (int b0 = 0; b0 < T; b0 += nt * kPrepBatch) {
        float g[kPrepBatch];
#pragma unroll
        for (int i = 0; i < kPrepBatch; ++i) {
            const int t = b0 + i * nt + tid;
            g[i] = t < T ? __ldcg(gates + (size_t)t * E + e) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kPrepBatch; ++i) {
            const int t = b0 + i * nt + tid;
            if (b0 + i * nt >= T) break;
            const uint32_t on = __ballot_sync(0xffffffffu, g[i] != 0.f);
            if (lane == 0) red[warp] = (uint32_t)__popc(on);
            __syncthreads();
            int before = base, all = 0;
            for (int q = 0; q < nw; ++q) {
                const int c = (int)red[q];
                before += q < warp ? c : 0;
                all += c;
            }
            if (lane == 0 && t < T) tpos[t >> 5] = before;
            if (g[i] != 0.f) list[before + __popc(on & ((1u << lane) - 1u))] = t;
            base += all;
            __syncthreads();
        }
    }
    if (tid == 0) {
        tpos[w.C32] = base;
        w.counts[e] = base;
    }
}

// --------------------------------------------------------------- experts_in --
constexpr int kXThreads = 384;
constexpr int kXMaxStages = 10;
constexpr int kXTile = 128 * 128;            // 128 rows x 128 int8
constexpr int kXRing = 200 * 1024;

struct XiShared {
    uint64_t full[kXMaxStages];
    uint64_t empty[kXMaxStages];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint64_t mma_done;
    uint32_t tmem_base;
    volatile int abort;
    uint32_t colmax[2][2][4][16];            // by warp group, piece parity, warp
    int cnt[256];
    int first[257];                          // first tile of each expert
};

struct XiItem {
    int e, base, rows;
};
// Tile i: expert e, tokens base .. base + rows of its list.  An expert's tokens are dealt
// evenly to its tiles, in sixteens.
__device__ __forceinline__ XiItem xi_item(const XiShared& sh, int E, int N, int i) {
    int lo = 0, hi = E;
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (sh.first[m] <= i) lo = m;
        else hi = m;
    }
    XiItem it;
    it.e = lo;
    const int cnt = sh.cnt[lo], nt = (cnt + N - 1) / N;
    const int per = ((cnt + nt - 1) / nt + 15) & ~15;
    it.base = (i - sh.first[lo]) * per;
    it.rows = min(per, cnt - it.base);
    return it;
}

// all threads of the named barrier agree: true when every one's v is
__device__ __forceinline__ bool bar_all(int id, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %2, 0;\n\t"
        "bar.red.and.pred q, %1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(v ? 1u : 0u)
        : "memory");
    return r != 0;
}

// What the epilogue does with n <= 16 columns (tokens) of int32 sums: h, its scale over
// all of d_e (the four warps of the group meet in colmax), 8-bit h and the pair's factors.
// Lane i (of 16) holds column i's token scale and gate.
template <int MT>
__device__ __forceinline__ void xi_finish(const X8In& a, XiShared& sh, const int (&v)[MT][16], int n, int e,
                                          size_t pair0, float sx, float gate, const float (&si)[MT],
                                          const float (&bi)[MT], int group, int q, int lane, uint32_t& parity) {
    float h[MT][16];
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float s = __shfl_sync(0xffffffffu, sx, i);
        uint32_t m = 0;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const float z = fmaf((float)v[mt][i] * si[mt], s, bi[mt]);
            h[mt][i] = __fdividef(z, 1.f + __expf(-z));
            m = max(m, __float_as_uint(h[mt][i]) & 0x7fffffffu);
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == i) mine = m;
    }
    uint32_t (&cm)[4][16] = sh.colmax[group][parity];
    parity ^= 1u;   // (the other buffer next: this one is read until the next barrier)
    if (lane < 16) cm[q][lane] = mine;
    named_bar_sync(1 + group, 128);
    RowScale r = {0.f, 0.f, 0.f};
    if (lane < 16) r = row_scale(max(max(cm[0][lane], cm[1][lane]), max(cm[2][lane], cm[3][lane])));
    if (q == 0 && lane < n) a.w.fpair[pair0 + lane] = make_float2(gate * r.scale, gate);
    int8_t* out = a.w.hq + pair0 * a.d_e + q * 32 + lane;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float inv = __shfl_sync(0xffffffffu, r.inv, i);
        if (i < n) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) out[(size_t)i * a.d_e + mt * 128] = (int8_t)(int)rintf(h[mt][i] * inv);
        }
    }
}

}  // namespace

template <int MT>
__global__ void __launch_bounds__(kXThreads, 1)
int8_experts_in_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                       const X8In a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int N = a.N;
    const int a_bytes = MT * kXTile, stage_bytes = a_bytes + N * 128;
    XiShared& sh = *reinterpret_cast<XiShared*>(smem + (size_t)a.stages * stage_bytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int crank = a.CS > 1 ? (int)cluster_ctarank() : 0;
    const int cluster = (int)blockIdx.x / a.CS;
    uint32_t cols = 32;
    while ((int)cols < 2 * MT * N) cols *= 2;

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
        tmem_alloc(&sh.tmem_base, cols);
        tmem_relinquish();
    }
    griddep_wait();
    griddep_launch_dependents();
    if (warp == 3) {
        // tiles of each expert and their running count
        int run = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane;
            const int cnt = e < a.E ? __ldcg(a.w.counts + e) : 0;
            const int nt = (cnt + N - 1) / N;
            int inc = nt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, inc, o);
                inc += lane >= o ? u : 0;
            }
            if (e < a.E) {
                sh.cnt[e] = cnt;
                sh.first[e] = run + inc - nt;
            }
            run += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) {
            sh.first[a.E] = run;
            if (__ldcg(&a.ctl->status) != 0) sh.abort = 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;
    const uint64_t limit = a.wait_ns;
    const int all = sh.first[a.E], tiles = sh.abort ? 0 : all;

    // S blocks per tile: as many as fill the grid once (a power of two, at most the cluster)
    int S = 1;
    while (2 * S <= a.CS && all * 2 * S <= (int)gridDim.x && a.KB >= 4 * S) S *= 2;
    const int sub = crank % S;
    const int first = (cluster * a.CS + crank) / S;
    const int step = (int)gridDim.x / S;
    const int kb0 = a.KB * sub / S, kb1 = a.KB * (sub + 1) / S;

    if (warp == 0) {
        const uint64_t pol = policy_evict_normal();
        int st = 0;
        uint32_t ph = 0;
        int issued = 0;
        bool ok = true;
        for (int i = first; i < tiles && ok; i += step) {
            const XiItem it = xi_item(sh, a.E, N, i);
            // lane l gathers rows 4 l .. 4 l + 3 (behind the last: the first again)
            const int32_t* list = a.w.list + (size_t)it.e * a.w.Tcap + it.base;
            const int quads = (it.rows + 3) >> 2;
            int r[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) r[u] = __ldcg(list + (4 * lane + u < it.rows ? 4 * lane + u : 0));
            const uint32_t bytes = (uint32_t)(a_bytes + quads * 512);
            for (int kb = kb0; kb < kb1; ++kb) {
                ok = wait_bar_warp(&sh.empty[st], ph ^ 1u, limit, &sh.abort, a.ctl, kWaitEmpty);
                if (!ok) break;
                uint8_t* sp = smem + (size_t)st * stage_bytes;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&sh.full[st], bytes);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
                        tma_load_2d(sp + mt * kXTile, &tm_w, &sh.full[st], kb * 128, it.e * a.d_e + mt * 128, pol);
                }
                __syncwarp();
                if (lane < quads)
                    tma_gather4(sp + a_bytes + lane * 512, &tm_x, &sh.full[st], kb * 128, r[0], r[1], r[2], r[3], pol);
                __syncwarp();
                ++issued;
                if (++st == a.stages) {
                    st = 0;
                    ph ^= 1u;
                }
            }
        }
        if (lane == 0) {
            // every load issued has landed before the block may end
            const int in_ring = min(issued, a.stages);
            for (int i = 0; i < in_ring; ++i) {
                st = st == 0 ? a.stages - 1 : st - 1;
                wait_bar_drain(&sh.full[st], (uint32_t)(((issued - 1 - i) / a.stages) & 1), limit, a.ctl);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        const uint64_t desc0 = sw128_kmajor_desc(smem_u32(smem));
        int st = 0, buf = 0;
        uint32_t ph = 0, bph = 0;
        bool ok = true;
        for (int i = first; i < tiles && ok; i += step) {
            const XiItem it = xi_item(sh, a.E, N, i);
            const uint32_t idesc = idesc_i8_s32(128, (it.rows + 15) & ~15);
            ok = wait_bar_warp(&sh.acc_empty[buf], bph ^ 1u, limit, &sh.abort, a.ctl, kWaitAccEmpty);
            if (!ok) break;
            tc_fence_after();
            for (int kb = kb0; kb < kb1; ++kb) {
                ok = wait_bar_warp(&sh.full[st], ph, limit, &sh.abort, a.ctl, kWaitFullW);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t ad = desc0 + (uint64_t)((uint32_t)st * (uint32_t)stage_bytes >> 4);
                    const uint64_t bd = ad + (uint64_t)(a_bytes >> 4);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            umma_i8(tmem + (uint32_t)((buf * MT + mt) * N), ad + mt * (kXTile >> 4) + 2 * k, bd + 2 * k,
                                    idesc, kb > kb0 || k > 0);
                    umma_commit(&sh.empty[st]);
                    if (kb == kb1 - 1) umma_commit(&sh.acc_full[buf]);
                }
                __syncwarp();
                if (++st == a.stages) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            buf ^= 1;
            if (buf == 0) bph ^= 1u;
        }
        // no MMA is in flight when the accumulators are given back
        if (elect_one()) umma_commit(&sh.mma_done);
        __syncwarp();
        if (lane == 0) wait_bar_drain(&sh.mma_done, 0u, limit, a.ctl);
        __syncwarp();
    } else if (warp >= 4) {
        const int q = warp & 3, group = (warp - 4) >> 2, ch = q * 32 + lane;
        int buf = 0;
        uint32_t bph = 0, parity = 0;
        for (int i = first; i < tiles; i += step) {
            const XiItem it = xi_item(sh, a.E, N, i);
            const size_t pair = (size_t)it.e * a.w.Tcap + it.base;
            float si[MT], bi[MT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                si[mt] = __ldg(a.s_in + (size_t)it.e * a.d_e + mt * 128 + ch);
                bi[mt] = a.b_in != nullptr ? __ldg(a.b_in + (size_t)it.e * a.d_e + mt * 128 + ch) : 0.f;
            }
            float sx[4], gt[4];
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const int c = group * 16 + 32 * p + (lane & 15);
                sx[p] = gt[p] = 0.f;
                if (S == 1 && c < it.rows) {
                    const int t = __ldcg(a.w.list + pair + c);
                    sx[p] = __ldcg(a.w.sx + t);
                    gt[p] = __ldg(a.gates + (size_t)t * a.E + it.e);
                }
            }
            // (the group leaves its loop together)
            if (!bar_all(1 + group, wait_bar_warp(&sh.acc_full[buf], bph, limit, &sh.abort, a.ctl, kWaitAccFull))) break;
            tc_fence_after();
            const uint32_t tacc = tmem + (uint32_t)(buf * MT * N) + ((uint32_t)(q * 32) << 16);
            if (S == 1) {
                if (group * 16 >= it.rows && lane == 0) mbar_arrive(&sh.acc_empty[buf]);   // nothing for this group
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const int c = group * 16 + 32 * p;
                    if (c < it.rows) {
                        int v[MT][16];
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            uint32_t u[32];
                            tmem_ld_32x32b_x16(tacc + (uint32_t)(mt * N + c), u);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 16; ++j) v[mt][j] = (int)u[j];
                        }
                        if (c + 32 >= it.rows) {   // the group's last piece is in registers
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&sh.acc_empty[buf]);
                        }
                        xi_finish<MT>(a, sh, v, min(16, it.rows - c), it.e, pair + c, sx[p], gt[p], si, bi, group, q,
                                      lane, parity);
                    }
                }
            } else {
                // partial sums [column][MT * 128] int32 over the stages (all read)
                int* part = reinterpret_cast<int*>(smem);
                for (int c = group * 16; c < it.rows; c += 32)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        uint32_t u[32];
                        tmem_ld_32x32b_x16(tacc + (uint32_t)(mt * N + c), u);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (c + j < it.rows) part[((c + j) * MT + mt) * 128 + ch] = (int)u[j];
                    }
            }
            buf ^= 1;
            if (buf == 0) bph ^= 1u;
        }
    }
    if (a.CS > 1 && S > 1) {
        // (S is the same in every block: one tile each, or none)
        cluster_barrier_sync();
        if (warp >= 4 && first < tiles && sh.abort == 0) {
            const int q = warp & 3, group = (warp - 4) >> 2, ch = q * 32 + lane;
            const XiItem it = xi_item(sh, a.E, N, first);
            uint32_t parity = 0;
            // this block's columns, half of them for each warp group (at most 16)
            const int per = N / S, c0 = sub * per + group * ((per + 1) / 2);
            const int c1 = min(group == 0 ? c0 + (per + 1) / 2 : (sub + 1) * per, it.rows);
            const int n = max(0, c1 - c0);
            if (n > 0) {
                const size_t pair = (size_t)it.e * a.w.Tcap + it.base + c0;
                float si[MT], bi[MT], sx = 0.f, gt = 0.f;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    si[mt] = __ldg(a.s_in + (size_t)it.e * a.d_e + mt * 128 + ch);
                    bi[mt] = a.b_in != nullptr ? __ldg(a.b_in + (size_t)it.e * a.d_e + mt * 128 + ch) : 0.f;
                }
                if ((lane & 15) < n) {
                    const int t = __ldcg(a.w.list + pair + (lane & 15));
                    sx = __ldcg(a.w.sx + t);
                    gt = __ldg(a.gates + (size_t)t * a.E + it.e);
                }
                int v[MT][16];
#pragma unroll
                for (int j = 0; j < 16; ++j)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        v[mt][j] = 0;
                        if (j < n) {
                            const uint32_t off = smem_u32(smem) + (uint32_t)(((c0 + j) * MT + mt) * 128 + ch) * 4u;
                            for (int r = 0; r < S; ++r)
                                v[mt][j] += ld_shared_cluster_s32(mapa_shared(off, (uint32_t)(crank - sub + r)));
                        }
                    }
                xi_finish<MT>(a, sh, v, n, it.e, pair, sx, gt, si, bi, group, q, lane, parity);
            }
        }
        cluster_barrier_sync();   // no block leaves while its partial sums may be read
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) tmem_dealloc(tmem, cols);
}

// -------------------------------------------------------------- experts_out --
namespace {

constexpr int kXoMaxStages = 10;
constexpr int kXoNB = 64;        // pairs of one expert multiplied at a time, at most
constexpr int kXoAcc = 4;        // accumulators in TMEM
constexpr int kXoMaxEnt = 1024;

struct alignas(16) XoShared {
    uint64_t full[kXoMaxStages];
    uint64_t empty[kXoMaxStages];
    uint64_t acc_full[kXoAcc];
    uint64_t acc_empty[kXoAcc];
    uint64_t mma_done;
    uint32_t tmem_base;
    volatile int abort;
    int n_ent;
    uint32_t ent[kXoMaxEnt];                 // expert << 24 | (pairs - 1) << 16 | first pair in its list
    alignas(16) int2 meta[8][kXoNB];         // by epilogue warp: row offset of the token, factor bits
    float gate[8][kXoNB];
};

}  // namespace

__global__ void __launch_bounds__(kXThreads, 1)
int8_experts_out_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_h,
                        const X8Out a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int NB = a.NB, TT = a.TT, S = a.S;
    const int stage_bytes = kXTile + NB * 128;
    float* acc = reinterpret_cast<float*>(smem + (size_t)a.stages * stage_bytes);   // [TT][128]
    XoShared& sh = *reinterpret_cast<XoShared*>(reinterpret_cast<uint8_t*>(acc) + (size_t)TT * 512);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = S > 1 ? (int)cluster_ctarank() : 0;
    const int item = (int)blockIdx.x / S, slab = item % a.slabs, t0 = item / a.slabs * TT;

    if (threadIdx.x == 0) {
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < kXoAcc; ++i) {
            mbar_init(&sh.acc_full[i], 1);
            mbar_init(&sh.acc_empty[i], 8);
        }
        mbar_init(&sh.mma_done, 1);
        fence_mbar_init();
        sh.abort = 0;
        prefetch_tmap(&tm_w);
        prefetch_tmap(&tm_h);
    }
    if (warp == 2) {
        tmem_alloc(&sh.tmem_base, kXoAcc * kXoNB);
        tmem_relinquish();
    }
    for (int i = threadIdx.x; i < TT * 32; i += kXThreads) reinterpret_cast<float4*>(acc)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    griddep_wait();
    griddep_launch_dependents();
    if (warp == 3) {
        // the tile's pairs, by expert, in pieces of at most NB
        const int c0 = t0 >> 5, c1 = min(a.w.C32, (t0 + TT) >> 5);
        int lo[8], hi[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = 32 * i + lane;
            lo[i] = hi[i] = 0;
            if (e < a.E) {
                lo[i] = __ldcg(a.w.tpos + (size_t)e * (a.w.C32 + 1) + c0);
                hi[i] = __ldcg(a.w.tpos + (size_t)e * (a.w.C32 + 1) + c1);
            }
        }
        int run = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int ne = (hi[i] - lo[i] + NB - 1) / NB;
            int inc = ne;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, inc, o);
                inc += lane >= o ? u : 0;
            }
            for (int k = 0; k < ne; ++k) {
                const int p = lo[i] + k * NB;
                sh.ent[run + inc - ne + k] = (uint32_t)(32 * i + lane) << 24 |
                                             (uint32_t)(min(NB, hi[i] - p) - 1) << 16 | (uint32_t)p;
            }
            run += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) {
            sh.n_ent = run;
            if (__ldcg(&a.ctl->status) != 0) sh.abort = 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;
    const uint64_t limit = a.wait_ns;
    const int ents = sh.abort ? 0 : sh.n_ent;
    const int m0 = ents * rank / S, m1 = ents * (rank + 1) / S;

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol = policy_evict_normal();
            int st = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int m = m0; m < m1 && ok; ++m) {
                const uint32_t en = sh.ent[m];
                const int e = (int)(en >> 24), n16 = (int)((en >> 16 & 255u) + 16) >> 4;
                const int row = e * a.w.Tcap + (int)(en & 0xffffu);
                for (int kb = 0; kb < a.KBe; ++kb) {
                    ok = wait_bar(&sh.empty[st], ph ^ 1u, limit, &sh.abort, a.ctl, kWaitEmpty);
                    if (!ok) break;
                    uint8_t* sp = smem + (size_t)st * stage_bytes;
                    mbar_arrive_expect_tx(&sh.full[st], (uint32_t)(kXTile + n16 * 2048));
                    tma_load_2d(sp, &tm_w, &sh.full[st], kb * 128, e * a.d_h + slab * 128, pol);
                    for (int i = 0; i < n16; ++i)
                        tma_load_2d(sp + kXTile + i * 2048, &tm_h, &sh.full[st], kb * 128, row + 16 * i, pol);
                    ++issued;
                    if (++st == a.stages) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
            }
            const int in_ring = min(issued, a.stages);
            for (int i = 0; i < in_ring; ++i) {
                st = st == 0 ? a.stages - 1 : st - 1;
                wait_bar_drain(&sh.full[st], (uint32_t)(((issued - 1 - i) / a.stages) & 1), limit, a.ctl);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        const uint64_t desc0 = sw128_kmajor_desc(smem_u32(smem));
        int st = 0, buf = 0;
        uint32_t ph = 0, bph = 0;
        bool ok = true;
        for (int m = m0; m < m1 && ok; ++m) {
            const uint32_t idesc = idesc_i8_s32(128, (int)((sh.ent[m] >> 16 & 255u) + 16) & ~15);
            ok = wait_bar_warp(&sh.acc_empty[buf], bph ^ 1u, limit, &sh.abort, a.ctl, kWaitAccEmpty);
            if (!ok) break;
            tc_fence_after();
            for (int kb = 0; kb < a.KBe; ++kb) {
                ok = wait_bar_warp(&sh.full[st], ph, limit, &sh.abort, a.ctl, kWaitFullH);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t ad = desc0 + (uint64_t)((uint32_t)st * (uint32_t)stage_bytes >> 4);
                    const uint64_t bd = ad + (kXTile >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_i8(tmem + (uint32_t)(buf * kXoNB), ad + 2 * k, bd + 2 * k, idesc, kb > 0 || k > 0);
                    umma_commit(&sh.empty[st]);
                    if (kb == a.KBe - 1) umma_commit(&sh.acc_full[buf]);
                }
                __syncwarp();
                if (++st == a.stages) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            if (++buf == kXoAcc) {
                buf = 0;
                bph ^= 1u;
            }
        }
        if (elect_one()) umma_commit(&sh.mma_done);
        __syncwarp();
        if (lane == 0) wait_bar_drain(&sh.mma_done, 0u, limit, a.ctl);
        __syncwarp();
    } else if (warp >= 4) {
        // A warp group owns half of the tile's tokens (a thread one channel of them), so no
        // sum is touched by two warps and the groups need not meet.
        const int q = warp & 3, group = (warp - 4) >> 2, ch = q * 32 + lane, o = slab * 128 + ch;
        int2* meta = sh.meta[warp - 4];
        float* mgate = sh.gate[warp - 4];
        const bool biased = a.b_out != nullptr;
        int buf = 0;
        uint32_t bph = 0;
        uint8_t* const my = reinterpret_cast<uint8_t*>(acc) + ch * 4;
        for (int m = m0; m < m1; ++m) {
            const uint32_t en = sh.ent[m];
            const int e = (int)(en >> 24), n = (int)(en >> 16 & 255u) + 1;
            const size_t pair = (size_t)e * a.w.Tcap + (en & 0xffffu);
            const float so = __ldg(a.s_out + (size_t)e * a.d_h + o);
            const float bo = biased ? __ldg(a.b_out + (size_t)e * a.d_h + o) : 0.f;
            int below = 0;   // columns whose tokens are in the first half (tokens ascend)
            __syncwarp();
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int c = lane + 32 * u;
                int tl = TT;
                if (c < n) {
                    tl = __ldcg(a.w.list + pair + c) - t0;
                    const float2 f = __ldcg(a.w.fpair + pair + c);
                    meta[c] = make_int2(tl * 512, __float_as_int(f.x));
                    mgate[c] = f.y;
                }
                below += __popc(__ballot_sync(0xffffffffu, tl < TT / 2));
            }
            __syncwarp();
            const int ca = group == 0 ? 0 : below, cb = group == 0 ? below : n;
            if (!wait_bar_warp(&sh.acc_full[buf], bph, limit, &sh.abort, a.ctl, kWaitAccFull)) break;
            tc_fence_after();
            const uint32_t tacc = tmem + (uint32_t)(buf * kXoNB) + ((uint32_t)(q * 32) << 16);
            for (int c = ca & ~15; c < cb; c += 16) {
                uint32_t v[32];
                tmem_ld_32x32b_x16(tacc + (uint32_t)c, v);
                tmem_ld_wait();
#pragma unroll
                for (int b = 0; b < 16; b += 8) {
                    int2 mt[8];
                    float s[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        mt[i] = meta[c + b + i];
                        if (c + b + i >= ca && c + b + i < cb) s[i] = *reinterpret_cast<float*>(my + mt[i].x);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (c + b + i >= ca && c + b + i < cb) {
                            float r = fmaf((float)(int)v[b + i] * so, __int_as_float(mt[i].y), s[i]);
                            if (biased) r = fmaf(mgate[c + b + i], bo, r);
                            *reinterpret_cast<float*>(my + mt[i].x) = r;
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.acc_empty[buf]);
            if (++buf == kXoAcc) {
                buf = 0;
                bph ^= 1u;
            }
        }
    }
    // y: the blocks of the cluster add their rows in rank order, each its share of the tokens
    if (S > 1) cluster_barrier_sync();
    else __syncthreads();
    if (sh.abort == 0) {
        const int ra = TT * rank / S, rb = min(TT * (rank + 1) / S, a.T - t0);
        for (int i = ra * 16 + (int)threadIdx.x; i < rb * 16; i += kXThreads) {
            float f[8];
            const float* p = acc + i * 8;
            if (S == 1) {
                const float4 u = *reinterpret_cast<const float4*>(p), v = *reinterpret_cast<const float4*>(p + 4);
                f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
                f[4] = v.x; f[5] = v.y; f[6] = v.z; f[7] = v.w;
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] = 0.f;
                const uint32_t off = smem_u32(p);
                for (int r = 0; r < S; ++r) {
                    const uint32_t rp = mapa_shared(off, (uint32_t)r);
                    const float4 u = ld_shared_cluster_f4(rp), v = ld_shared_cluster_f4(rp + 16);
                    f[0] += u.x; f[1] += u.y; f[2] += u.z; f[3] += u.w;
                    f[4] += v.x; f[5] += v.y; f[6] += v.z; f[7] += v.w;
                }
            }
            __nv_bfloat162 b[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) b[k] = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
            *reinterpret_cast<uint4*>(a.y + (size_t)(t0 + (i >> 4)) * a.d_h + slab * 128 + (i & 15) * 8) =
                *reinterpret_cast<const uint4*>(b);
        }
    }
    if (S > 1) cluster_barrier_sync();   // no block leaves while its rows may be read
    tc_fence_before();
    __syncthreads();
    if (warp == 2) tmem_dealloc(tmem, kXoAcc * kXoNB);
}

// ----------------------------------------------------------------- launches --
namespace {

cudaLaunchConfig_t x8_config(int grid, int threads, size_t smem, cudaStream_t s, cudaLaunchAttribute* at, int cluster) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cfg;
}

constexpr int kMaxSmem = 227 * 1024;

template <int MT>
cudaError_t launch_in(const X8In& a, const CUtensorMap* maps, int grid, size_t smem, cudaStream_t s) {
    auto kern = int8_experts_in_kernel<MT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[2];
    cudaLaunchConfig_t cfg = x8_config(grid, kXThreads, smem, s, at, a.CS);
    return cudaLaunchKernelEx(&cfg, kern, maps[0], maps[1], a);
}

}  // namespace

cudaError_t launch_int8_prepare(const __nv_bfloat16* x, const float* gates, int T, int d_h, int E, const X8Bufs& w,
                                cudaStream_t s) {
    cudaLaunchAttribute at[2];
    cudaLaunchConfig_t cfg = x8_config(T + E, quantize_threads(d_h, 2), 0, s, at, 1);
    return quantize_one_pass(d_h, 2) ? cudaLaunchKernelEx(&cfg, int8_prepare_kernel<true>, x, gates, T, d_h, E, w)
                                     : cudaLaunchKernelEx(&cfg, int8_prepare_kernel<false>, x, gates, T, d_h, E, w);
}

// Tokens per tile and blocks per cluster.  A tile of all an expert's tokens reads its
// weight once, so N grows with T, up to what two accumulators of all d_e rows leave of
// TMEM (2 * d_e / 128 * N <= 512 columns) and a gather of one warp (128 rows).  Where
// the tiles may be fewer than the SMs, clusters let several blocks share a tile.
cudaError_t launch_int8_experts_in(X8In a, const CUtensorMap* maps, int sms, cudaStream_t s) {
    const int MT = a.d_e / 128, stage = MT * kXTile + a.N * 128;
    a.stages = kXRing / stage < kXMaxStages ? kXRing / stage : kXMaxStages;
    const size_t smem = 1024 + (size_t)a.stages * stage + sizeof(XiShared);
    // (clusters of 8 do not fill every SM: 16 of them fit)
    const int grid = a.CS == 8 ? 128 : sms / a.CS * a.CS;
    switch (MT) {
        case 1: return launch_in<1>(a, maps, grid, smem, s);
        case 2: return launch_in<2>(a, maps, grid, smem, s);
        case 3: return launch_in<3>(a, maps, grid, smem, s);
        default: return launch_in<4>(a, maps, grid, smem, s);
    }
}

cudaError_t launch_int8_experts_out(X8Out a, const CUtensorMap* maps, cudaStream_t s) {
    const int stage = kXTile + a.NB * 128;
    const int room = (kMaxSmem - 1024 - (int)sizeof(XoShared) - a.TT * 512) / stage;
    a.stages = room < kXoMaxStages ? room : kXoMaxStages;
    const size_t smem = 1024 + (size_t)a.stages * stage + (size_t)a.TT * 512 + sizeof(XoShared);
    auto kern = int8_experts_out_kernel;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[2];
    const int grid = a.slabs * ((a.T + a.TT - 1) / a.TT) * a.S;
    cudaLaunchConfig_t cfg = x8_config(grid, kXThreads, smem, s, at, a.S);
    return cudaLaunchKernelEx(&cfg, kern, maps[0], maps[1], a);
}

}  // namespace bffn
