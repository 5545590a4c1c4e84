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
//   experts_in : tiles of one expert x up to N of its tokens, all of d_e.  Up to 64 tokens
//                are all multiplied (what counts is the weights' bytes); else x rows are
//                gathered in 16-byte asynchronous copies straight into the MMA's
//                swizzled layout (TMA's gather of four rows an operation took about 60
//                cycles each, 18 us for a tile of 128 rows at d_h 2048).  The tile holds
//                whole rows of h, so the epilogue finds their scales and writes 8-bit h.
//                Few tiles: a cluster's blocks split d_h and add their int32 sums through
//                distributed shared memory.
//   experts_out: a block owns TT consecutive tokens x 128 output channels as fp32
//                sums in shared memory and walks the experts; a token tile's tokens
//                are neighbours in every expert's list, so h comes in plain boxes of
//                16, 32 or 64 rows.  Each int32 result column is scaled and added to its
//                token's row.  Few tiles: a cluster's blocks share the experts and
//                add their fp32 rows in rank order.
// The three kernels are programmatic dependents of one another.
//
// What bounds them.  Decode: the way through three dependent launches, each with a plan
// to read: at d_h 2048, 8 of 64 experts, 15 us for one token and 19.5 us for a 32-token
// chunk, whose bytes take 0.7 and 3.4 us.  Long inputs (117 us at 4096 tokens; the three
// kernels alone 12, 36 and 81 us, the bytes and the products 10.6 us each): the entries of
// experts_out, one expert's pairs in a tile of tokens.  A block takes some 1200 cycles for one of
// about 32 pairs, of which the sums' read-modify-write in shared memory, 8 bytes for every
// pair and channel, is 256 (57 % of the shared-memory pipe, 6 % of the tensor pipe; 256 blocks
// are 1.73 waves); the time follows the number of entries more than that of pairs.  Tried there
// and slower: entries in twos under
// one barrier with their pieces pipelined (118 -> 123 us), four epilogue groups instead
// of two (118 -> 123 us), 128-token tiles (142 -> 198 us: twice the entries).
#include <cuda.h>
#include <cuda_runtime.h>

#include "int8.cuh"
#include "launch.h"

namespace bffn {

namespace {

// ------------------------------------------------------------------ prepare --
// Blocks 0 .. E-1 list an expert's tokens; the blocks behind them round tokens.
constexpr int kPrepBatch = 16;   // gates a thread has in flight

template <int C>
__global__ void __launch_bounds__(kQThreads) int8_prepare_kernel(const __nv_bfloat16* __restrict__ x,
                                                                 const float* __restrict__ gates, int T, int d_h,
                                                                 int E, int lgW, const X8Bufs w, Ctl* ctl) {
    constexpr int kWarps = kQThreads / 32;
    __shared__ uint32_t red[kPrepBatch * kWarps + 1];
    griddep_wait();
    griddep_launch_dependents();
    const Int8Gate gate = int8_gate(ctl);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if ((int)blockIdx.x >= E) {
        const int W = 1 << lgW, g = tid >> lgW, t = (((int)blockIdx.x - E) << (8 - lgW)) + g;
        if (t < T)
            quantize_row<__nv_bfloat16, C>(x + (size_t)t * d_h, d_h, w.xq + (size_t)t * d_h, w.sx + t, W, tid & (W - 1),
                                           1 + g, red + (g << lgW >> 5), gate);
        return;
    }
    const int e = blockIdx.x;
    int32_t* list = w.list + (size_t)e * w.Tcap;
    int32_t* tpos = w.tpos + (size_t)e * (w.C32 + 1);
    int base = 0;   // tokens listed so far
    for (int b0 = 0; b0 < T; b0 += kQThreads * kPrepBatch) {
        uint32_t on[kPrepBatch];
#pragma unroll
        for (int i = 0; i < kPrepBatch; ++i) {
            const int t = b0 + i * kQThreads + tid;
            on[i] = t < T ? __float_as_uint(__ldcg(gates + (size_t)t * E + e)) : 0u;
        }
#pragma unroll
        for (int i = 0; i < kPrepBatch; ++i) {
            on[i] = __ballot_sync(0xffffffffu, __uint_as_float(on[i]) != 0.f);
            if (lane == 0) red[i * kWarps + warp] = (uint32_t)__popc(on[i]);
        }
        if (!__syncthreads_and(int8_gate_open(gate))) return;
        if (warp == 0) {   // running sums over the batch's warps, in token order
            constexpr int kPer = kPrepBatch * kWarps / 32;
            uint32_t c[kPer], s = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                c[i] = red[kPer * lane + i];
                s += c[i];
            }
            const uint32_t mine = s;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t u = __shfl_up_sync(0xffffffffu, s, o);
                s += lane >= o ? u : 0u;
            }
            uint32_t run = s - mine;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                red[kPer * lane + i] = run;
                run += c[i];
            }
            if (lane == 31) red[kPrepBatch * kWarps] = s;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPrepBatch; ++i) {
            const int t = b0 + i * kQThreads + tid;
            const int before = base + (int)red[i * kWarps + warp];
            if (lane == 0 && t < T) tpos[t >> 5] = before;
            if (on[i] >> lane & 1u) list[before + __popc(on[i] & ((1u << lane) - 1u))] = t;
        }
        base += (int)red[kPrepBatch * kWarps];
        __syncthreads();
    }
    if (tid == 0) {
        tpos[w.C32] = base;
        w.counts[e] = base;
    }
}

// --------------------------------------------------------------- experts_in --
// Gathering warps of experts_in (2, 3, 12, ..): as many as its registers leave room for.
template <int MT>
struct XiCfg {
    static constexpr int kGather = MT <= 2 ? 8 : 4;
    static constexpr int kThreads = 384 + 32 * (kGather - 2);
    static constexpr int kStep = 4 * kGather;         // token rows they copy at a time
    static constexpr int kRows = 128 / kStep;
};
constexpr int kXMaxStages = 10;
constexpr int kXTile = 128 * 128;            // 128 rows x 128 int8
constexpr int kXRing = 200 * 1024;

struct XiShared {
    uint64_t full[kXMaxStages];              // weight tiles landed (bytes)
    uint64_t gathered[kXMaxStages];          // token rows copied (the gathering warps)
    uint64_t empty[kXMaxStages];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint64_t mma_done;
    uint32_t tmem_base;
    volatile int abort;
    int refused;                             // an earlier error, written once, before the first barrier
    uint32_t colmax[2][2][4][16];            // by warp group, piece parity, warp
    int cnt[256];
    int per[256];                            // tokens of each of an expert's tiles
    int first[257];                          // first tile of each expert
};

struct XiItem {
    int e, base, rows;
};
// Tile i: expert e, tokens base .. base + rows of its list.  An expert's tokens are dealt
// evenly to its tiles, in sixteens.  Called by whole warps.
__device__ __forceinline__ XiItem xi_item(const XiShared& sh, int E, int i) {
    const int lane = threadIdx.x & 31;
    int e = -1;   // the last expert whose first tile is not behind i
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (32 * j >= E) break;
        e += __popc(__ballot_sync(0xffffffffu, 32 * j + lane < E && sh.first[32 * j + lane] <= i));
    }
    XiItem it;
    it.e = e;
    it.base = (i - sh.first[e]) * sh.per[e];
    it.rows = min(sh.per[e], sh.cnt[e] - it.base);
    return it;
}

// The same for the tile behind i0's (whose expert is known), by one thread: the next tiles
// of a block are a grid apart.
__device__ __forceinline__ XiItem xi_item_from(const XiShared& sh, int E, int i, int e0) {
    int lo = e0, hi = E;
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (sh.first[m] <= i) lo = m;
        else hi = m;
    }
    XiItem it;
    it.e = lo;
    it.base = (i - sh.first[lo]) * sh.per[lo];
    it.rows = min(sh.per[lo], sh.cnt[lo] - it.base);
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

__device__ __forceinline__ void tmem_ld_piece(uint32_t taddr, int (&v)[8]) {
    // (no copy: the registers hold their values only after tmem_ld_wait)
    tmem_ld_32x32b_x8(taddr, reinterpret_cast<uint32_t (&)[8]>(v));
}

// Swish, z / (1 + exp(-z)): expf (within 2 steps of fp32), the sum rounded once, and the quotient
// by a reciprocal and one step of refinement with the remainder, which leaves it within half a
// step and 2^-20 of one.  No branches, so a piece's columns run through it side by side.
// (Divisor and quotient are carried as d / 8 and 8 h: the reciprocal takes no divisor above
// 2^126, z below -87.  Below -88.7 exp(-z) is infinite and h -0; an infinite or NaN z gives NaN.)
__device__ __forceinline__ float xi_swish(float z) {
    const float d = fmaf(expf(-z), 0.125f, 0.125f);
    const float r = __fdividef(1.f, d), q = z * r;
    return d < INFINITY ? fmaf(fmaf(-q, d, z), r, q) * 0.125f : q;
}

// What the epilogue does with PW columns (tokens) of int32 sums: h, its scale over all of
// d_e (the four warps of the group meet in colmax), 8-bit h and the pair's factors.  Lane i
// (of PW) holds column i's token, its scale and gate, and the place of the pair in the
// expert's list (slot, -1: no pair); pair0: the list's first pair.
// z, Swish and 127 h / amax are evaluated as the formula reads, every step rounded once to fp32
// (near the border of two whole numbers, that is; elsewhere h * (127 / amax) rounds to the same
// number): a value on the other side of a border moves its token's whole row of y.  (From the
// approximate exponential and quotient alone that was one value in 700000, and h was 0 below
// z = -87.)
template <int MT, int PW>
__device__ __forceinline__ void xi_finish(const X8In& a, XiShared& sh, const int (&v)[MT][PW], size_t pair0, int slot,
                                          int token, float sx, float gate, const float (&si)[MT],
                                          const float (&bi)[MT], int group, int q, int lane, uint32_t& parity) {
    float h[MT][PW];
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < PW; ++i) {
        const float s = __shfl_sync(0xffffffffu, sx, i);
        uint32_t m = 0;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const float z = __fadd_rn(__fmul_rn((float)v[mt][i] * si[mt], s), bi[mt]);
            h[mt][i] = xi_swish(z);
            m = max(m, __float_as_uint(h[mt][i]) & 0x7fffffffu);
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == i) mine = m;
    }
    uint32_t (&cm)[4][16] = sh.colmax[group][parity];
    parity ^= 1u;   // (the other buffer next: this one is read until the next barrier)
    if (lane < PW) cm[q][lane] = mine;
    named_bar_sync(1 + group, 128);
    RowScale r = {0.f, 0.f, 0.f};
    if (lane < PW) r = row_scale(max(max(cm[0][lane], cm[1][lane]), max(cm[2][lane], cm[3][lane])));
    if (q == 0 && lane < PW && slot >= 0)
        a.w.pair[pair0 + slot] = make_float4(__int_as_float(token), gate * r.scale, gate, 0.f);
    int8_t* out = a.w.hq + pair0 * a.d_e + q * 32 + lane;
    // rounded by adding 1.5 * 2^23 (the whole number is the sum's low byte); what was rounded off
    // is off by 127 * 2^-24 at most, inv's share, and the formula's own steps by twice that
    constexpr float kMagic = 12582912.f, kNear = 0.49997f;
    float worst = 0.f;
#pragma unroll
    for (int i = 0; i < PW; ++i) {
        const float inv = __shfl_sync(0xffffffffu, r.inv, i);
        const int at = __shfl_sync(0xffffffffu, slot, i);
        if (at >= 0) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const float t = fmaf(h[mt][i], inv, kMagic);
                worst = fmaxf(worst, fabsf(fmaf(h[mt][i], inv, kMagic - t)));
                out[(size_t)at * a.d_e + mt * 128] = (int8_t)__float_as_uint(t);
            }
        }
    }
    if (__any_sync(0xffffffffu, worst > kNear)) {   // (one piece in a hundred)
#pragma unroll
        for (int i = 0; i < PW; ++i) {
            const float inv = __shfl_sync(0xffffffffu, r.inv, i), amax = __shfl_sync(0xffffffffu, r.amax, i);
            const int at = __shfl_sync(0xffffffffu, slot, i);
            if (at >= 0) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const float t = fmaf(h[mt][i], inv, kMagic);
                    if (fabsf(fmaf(h[mt][i], inv, kMagic - t)) > kNear)
                        out[(size_t)at * a.d_e + mt * 128] =
                            (int8_t)(int)rintf(__fdiv_rn(__fmul_rn(h[mt][i], 127.f), amax));
                }
            }
        }
    }
}

}  // namespace

template <int MT>
__global__ void __launch_bounds__(XiCfg<MT>::kThreads, 1)
int8_experts_in_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                       const X8In a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    // Columns the epilogue holds at a time.  (Small pieces in rolled loops: at a decode step every
    // instruction of the epilogue runs once, from a cold instruction cache.)
    constexpr int PW = 8, PWX = 4;
    const int N = 1 << a.lgN;
    const int a_bytes = MT * kXTile, stage_bytes = a_bytes + N * 128;
    XiShared& sh = *reinterpret_cast<XiShared*>(smem + (size_t)a.stages * stage_bytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int crank = a.CS > 1 ? (int)cluster_ctarank() : 0;
    uint32_t cols = 32;
    while ((int)cols < 2 * MT * N) cols *= 2;

    if (threadIdx.x == 0) {
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.gathered[i], a.T <= N ? 1 : XiCfg<MT>::kGather);
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
    if (warp == 1) {
        tmem_alloc(&sh.tmem_base, cols);
        tmem_relinquish();
    }
    griddep_wait();
    griddep_launch_dependents();
    if (warp == 0) {
        // tiles of each expert and their running count
        const int status = __ldcg(&a.ctl->status);
        int cnt[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) cnt[i] = 32 * i + lane < a.E ? __ldcg(a.w.counts + 32 * i + lane) : 0;
        int run = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (32 * i >= a.E) break;
            const int e = 32 * i + lane, nt = (cnt[i] + N - 1) >> a.lgN;
            int inc = nt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, inc, o);
                inc += lane >= o ? u : 0;
            }
            if (e < a.E) {
                sh.cnt[e] = cnt[i];
                // (at most 8192 tokens: the quotient by way of fp32 is exact, and quicker)
                sh.per[e] = nt > 0 ? ((int)__fdividef((float)(cnt[i] + nt) - 0.5f, (float)nt) + 15) & ~15 : 0;
                sh.first[e] = run + inc - nt;
            }
            run += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) {
            sh.first[a.E] = run;
            sh.refused = status != 0;
            if (status != 0) sh.abort = 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;
    const uint64_t limit = a.wait_ns;
    const int all = sh.first[a.E], tiles = sh.refused ? 0 : all;

    // A slice of at most N tokens is not gathered: column c of every tile is token c, all
    // of them are multiplied, and the epilogue takes the columns of the expert's tokens.
    const bool dense = a.T <= N;

    // S = 2^lgS blocks per tile: as many as fill the grid once, at most the cluster
    int lgS = 0;
    while ((2 << lgS) <= a.CS && (all << (lgS + 1)) <= (int)gridDim.x && a.KB >= (4 << lgS)) ++lgS;
    const int S = 1 << lgS, sub = crank & (S - 1);
    const int first = (int)blockIdx.x >> lgS, step = (int)gridDim.x >> lgS;
    const int kb0 = a.KB * sub >> lgS, kb1 = a.KB * (sub + 1) >> lgS;

    if (warp == 0) {
        XiItem it = {0, 0, 0};
        if (first < tiles) it = xi_item(sh, a.E, first);
        // (elect.sync, not lane 0: what one elected lane runs is issued at twice the rate)
        if (elect_one()) {
            const uint64_t pol = policy_evict_normal();
            int st = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int i = first; i < tiles && ok; i += step) {
                if (i != first) it = xi_item_from(sh, a.E, i, it.e);
                for (int kb = kb0; kb < kb1; ++kb) {
                    ok = wait_bar(&sh.empty[st], ph ^ 1u, limit, &sh.abort, a.ctl, kWaitEmpty);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&sh.full[st], (uint32_t)a_bytes);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
                        tma_load_2d(smem + (size_t)st * stage_bytes + mt * kXTile, &tm_w, &sh.full[st], kb * 128,
                                    it.e * a.d_e + mt * 128, pol);
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
                wait_bar_drain(&sh.full[st], (uint32_t)(((issued - 1 - i) / a.stages) & 1), limit, a.ctl);
            }
        }
        __syncwarp();
    } else if (dense && (warp == 2 || warp == 3 || warp >= 12)) {
        if (warp == 2 && elect_one()) {
            const uint64_t pol = policy_evict_normal();
            int st = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int i = first; i < tiles && ok; i += step) {
                for (int kb = kb0; kb < kb1; ++kb) {
                    ok = wait_bar(&sh.empty[st], ph ^ 1u, limit, &sh.abort, a.ctl, kWaitEmpty);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&sh.gathered[st], (uint32_t)(N * 128));
                    tma_load_2d(smem + (size_t)st * stage_bytes + a_bytes, &tm_x, &sh.gathered[st], kb * 128, 0, pol);
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
                wait_bar_drain(&sh.gathered[st], (uint32_t)(((issued - 1 - i) / a.stages) & 1), limit, a.ctl);
            }
        }
        __syncwarp();
    } else if (warp == 2 || warp == 3 || warp >= 12) {
        // Gather: eight lanes copy one token row's 128 bytes in 16-byte pieces into the
        // swizzled layout (piece c of row r lies at c ^ (r & 7)); the warps take four rows
        // each in turn.  A stage is announced once it has landed and the two behind it (fewer
        // in a short ring, which leaves the MMAs and the copies a stage each) are under way; the
        // MMA reads the rows through the async proxy, hence the fence.
        constexpr int kRows = XiCfg<MT>::kRows, kStep = XiCfg<MT>::kStep;
        const int gw = warp < 4 ? warp - 2 : warp - 10;
        const int r0 = gw * 4 + (lane >> 3), c = lane & 7;
        const uint32_t dst0 = (uint32_t)(r0 * 128 + ((c ^ (r0 & 7)) << 4));
        const int later = min(2, a.stages - 2);
        int st = 0, ann = 0, pending = 0;
        auto announce = [&]() {   // the oldest stage has landed
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.gathered[ann]);
            if (++ann == a.stages) ann = 0;
            --pending;
        };
        uint32_t ph = 0;
        bool ok = true;
        int next[kRows];   // the next tile's tokens, on their way
        XiItem it = {0, 0, 0};
        auto fetch = [&](int i) {
            if (i >= tiles) return;
            it = xi_item(sh, a.E, i);
            const int32_t* list = a.w.list + (size_t)it.e * a.w.Tcap + it.base;
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                next[u] = 0;
                if (kStep * u < it.rows) next[u] = __ldcg(list + min(kStep * u + r0, it.rows - 1));
            }
        };
        fetch(first);
        for (int i = first; i < tiles && ok; i += step) {
            uint32_t tok[kRows];
            const int rows = it.rows;
#pragma unroll
            for (int u = 0; u < kRows; ++u) tok[u] = (uint32_t)next[u] * (uint32_t)a.KB;   // in 128-byte rows
            fetch(i + step);
            for (int kb = kb0; kb < kb1; ++kb) {
                ok = wait_bar_warp(&sh.empty[st], ph ^ 1u, limit, &sh.abort, a.ctl, kWaitEmpty);
                if (!ok) break;
                uint8_t* sp = smem + (size_t)st * stage_bytes + a_bytes + dst0;
                const int8_t* src = a.w.xq + kb * 128 + c * 16;
#pragma unroll
                for (int u = 0; u < kRows; ++u)
                    if (kStep * u < rows) cp_async_16(sp + u * kStep * 128, src + (size_t)tok[u] * 128);
                if (++st == a.stages) {
                    st = 0;
                    ph ^= 1u;
                }
                cp_async_commit();
                if (++pending > later) {
                    if (later == 2) cp_async_wait<2>();
                    else if (later == 1) cp_async_wait<1>();
                    else cp_async_wait<0>();
                    announce();
                }
            }
        }
        cp_async_wait_all();
        while (pending > 0) announce();
        __syncwarp();
    } else if (warp == 1) {
        const uint64_t desc0 = sw128_kmajor_desc(smem_u32(smem));
        XiItem it = {0, 0, 0};
        if (first < tiles) it = xi_item(sh, a.E, first);
        if (elect_one()) {
            int st = 0, buf = 0;
            uint32_t ph = 0, bph = 0;
            bool ok = true;
            for (int i = first; i < tiles && ok; i += step) {
                if (i != first) it = xi_item_from(sh, a.E, i, it.e);
                const uint32_t idesc = idesc_i8_s32(128, ((dense ? a.T : it.rows) + 15) & ~15);
                ok = wait_bar(&sh.acc_empty[buf], bph ^ 1u, limit, &sh.abort, a.ctl, kWaitAccEmpty);
                if (!ok) break;
                tc_fence_after();
                for (int kb = kb0; kb < kb1; ++kb) {
                    ok = wait_bar(&sh.full[st], ph, limit, &sh.abort, a.ctl, kWaitFullW) &&
                         wait_bar(&sh.gathered[st], ph, limit, &sh.abort, a.ctl, kWaitFullW);
                    if (!ok) break;
                    tc_fence_after();
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
    } else {   // warps 4 .. 11
        const int q = warp & 3, group = (warp - 4) >> 2, ch = q * 32 + lane;
        int buf = 0;
        uint32_t bph = 0, parity = 0;
        for (int i = first; i < tiles; i += step) {
            const XiItem it = xi_item(sh, a.E, i);
            const size_t pair0 = (size_t)it.e * a.w.Tcap;
            const int width = dense ? a.T : it.rows;   // columns of the tile
            float si[MT], bi[MT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                si[mt] = __ldg(a.s_in + (size_t)it.e * a.d_e + mt * 128 + ch);
                bi[mt] = a.b_in != nullptr ? __ldg(a.b_in + (size_t)it.e * a.d_e + mt * 128 + ch) : 0.f;
            }
            // (dense) the expert's tokens as bits: N <= 128, a register for each 32
            uint32_t on[4] = {0u, 0u, 0u, 0u};
            if (dense && S == 1) {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int t = 32 * w + lane;
                    on[w] = __ballot_sync(0xffffffffu, t < a.T && __ldg(a.gates + (size_t)t * a.E + it.e) != 0.f);
                }
            }
            // What is known of the group's columns (at most 64: column j of the group is column
            // 16 (j / 8) + 8 group + j % 8 of the tile) before the sums are there: lane i holds
            // its columns i and i + 32.
            int tks[2] = {0, 0}, slots[2] = {-1, -1};
            float sxs[2] = {0.f, 0.f}, gts[2] = {0.f, 0.f};
            if (S == 1) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int j = lane + 32 * u, c = 16 * (j >> 3) + 8 * group + (j & 7);
                    if (c >= width) continue;
                    if (!dense) {
                        slots[u] = it.base + c;
                        tks[u] = __ldcg(a.w.list + pair0 + slots[u]);
                    } else {
                        const int w = c >> 5;
                        const uint32_t word = w == 0 ? on[0] : w == 1 ? on[1] : w == 2 ? on[2] : on[3];
                        if (!(word >> (c & 31) & 1u)) continue;
                        tks[u] = c;
                        slots[u] = __popc(word & ((1u << (c & 31)) - 1u)) + (w > 0 ? __popc(on[0]) : 0) +
                                   (w > 1 ? __popc(on[1]) : 0) + (w > 2 ? __popc(on[2]) : 0);
                    }
                }
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    if (slots[u] >= 0) {
                        sxs[u] = __ldcg(a.w.sx + tks[u]);
                        gts[u] = __ldg(a.gates + (size_t)tks[u] * a.E + it.e);
                    }
            }
            // (the group leaves its loop together)
            if (!bar_all(1 + group, wait_bar_warp(&sh.acc_full[buf], bph, limit, &sh.abort, a.ctl, kWaitAccFull))) break;
            tc_fence_after();
            const uint32_t tacc = tmem + (uint32_t)(buf * MT * N) + ((uint32_t)(q * 32) << 16);
            if (S == 1) {
                if (group * PW >= width && lane == 0) mbar_arrive(&sh.acc_empty[buf]);   // nothing for this group
#pragma unroll 1
                for (int p = 0, c = group * PW; c < width; ++p, c += 2 * PW) {
                    int v[MT][PW];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) tmem_ld_piece(tacc + (uint32_t)(mt * N + c), v[mt]);
                    // lane i of the piece: the group's column 8 p + i
                    const int from = (8 * p + (lane & (PW - 1))) & 31;
                    const bool hi = p >= 4;
                    const int slot = __shfl_sync(0xffffffffu, hi ? slots[1] : slots[0], from);
                    const int tk = __shfl_sync(0xffffffffu, hi ? tks[1] : tks[0], from);
                    const float sx = __shfl_sync(0xffffffffu, hi ? sxs[1] : sxs[0], from);
                    const float gt = __shfl_sync(0xffffffffu, hi ? gts[1] : gts[0], from);
                    tmem_ld_wait();
                    if (c + 2 * PW >= width) {   // the group's last piece is in registers
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh.acc_empty[buf]);
                    }
                    xi_finish<MT, PW>(a, sh, v, pair0, slot, tk, sx, gt, si, bi, group, q, lane, parity);
                }
            } else {
                // partial sums [column][MT * 128] int32 over the stages (all read)
                int* part = reinterpret_cast<int*>(smem);
#pragma unroll 1
                for (int c = group * PW; c < width; c += 2 * PW) {
                    int v[MT][PW];
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) tmem_ld_piece(tacc + (uint32_t)(mt * N + c), v[mt]);
                    tmem_ld_wait();
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int j = 0; j < PW; ++j)
                            if (c + j < width) part[((c + j) * MT + mt) * 128 + ch] = v[mt][j];
                }
            }
            buf ^= 1;
            if (buf == 0) bph ^= 1u;
        }
    }
    if (S > 1) {
        // (S is the same in every block: one tile each, or none)
        const int q = warp & 3, group = (warp - 4) >> 2, ch = q * 32 + lane;
        float si[MT], bi[MT], sx = 0.f, gt = 0.f;
        int c0 = 0, n = 0, tk = 0;
        size_t pair0 = 0;
        if (warp >= 4 && warp < 12 && first < tiles) {
            // this block's share of the listed tokens, half of them for each warp group (at
            // most 16: N <= 64 where clusters have more than one block)
            const XiItem it = xi_item(sh, a.E, first);
            const int per = (it.rows + S - 1) >> lgS, half = (per + 1) >> 1;
            c0 = sub * per + group * half;
            n = max(0, min(min(c0 + half, (sub + 1) * per), it.rows) - c0);
            c0 += it.base;
            pair0 = (size_t)it.e * a.w.Tcap;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                si[mt] = __ldg(a.s_in + (size_t)it.e * a.d_e + mt * 128 + ch);
                bi[mt] = a.b_in != nullptr ? __ldg(a.b_in + (size_t)it.e * a.d_e + mt * 128 + ch) : 0.f;
            }
            if ((lane & 15) < n) {
                tk = __ldcg(a.w.list + pair0 + c0 + (lane & 15));
                sx = __ldcg(a.w.sx + tk);
                gt = __ldg(a.gates + (size_t)tk * a.E + it.e);
            }
            // (the tile's column of this lane's token)
            c0 -= it.base;
        }
        const int col = dense ? tk : c0 + (lane & 15);
        cluster_barrier_sync();
        if (n > 0 && sh.abort == 0) {
            uint32_t parity = 0;
            const int base = xi_item(sh, a.E, first).base;
            const uint32_t off = smem_u32(smem) + (uint32_t)ch * 4u;
#pragma unroll 1
            for (int b = 0; b < n; b += PWX) {
                // lane i of the piece: pair b + i, held by lane b + i
                const int from = (b + lane) & 15;
                const int slot = lane < PWX && b + lane < n ? base + c0 + b + lane : -1;
                // (at most four blocks share a tile; all their partial sums in flight at once)
                int u[4][MT][PWX], v[MT][PWX];
#pragma unroll
                for (int j = 0; j < PWX; ++j) {
                    const int cj = __shfl_sync(0xffffffffu, col, (b + j) & 15);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
                            u[r][mt][j] = r < S && b + j < n
                                              ? ld_shared_cluster_s32(mapa_shared(off + (uint32_t)((cj * MT + mt) * 512),
                                                                                  (uint32_t)(crank - sub + r)))
                                              : 0;
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int j = 0; j < PWX; ++j) v[mt][j] = u[0][mt][j] + u[1][mt][j] + u[2][mt][j] + u[3][mt][j];
                xi_finish<MT, PWX>(a, sh, v, pair0, slot, __shfl_sync(0xffffffffu, tk, from),
                                   __shfl_sync(0xffffffffu, sx, from), __shfl_sync(0xffffffffu, gt, from), si, bi, group,
                                   q, lane, parity);
            }
        }
        cluster_barrier_sync_relaxed();   // no block leaves while its partial sums may be read
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, cols);
}

// -------------------------------------------------------------- experts_out --
namespace {

constexpr int kXoMaxStages = 10;
constexpr int kXoNB = 64;        // pairs of one expert multiplied at a time, at most
constexpr int kXoGroups = 2;     // epilogue warp groups: each owns that part of the tile's tokens
constexpr int kXoThreads = 256 + 128 * kXoGroups;
constexpr int kXoAcc = 6;        // accumulators in TMEM, and lists of their columns
constexpr int kXoTmem = 512;     // columns: the accumulators', and room behind the last for a whole piece
constexpr int kXoMaxEnt = 1024;

// An entry's columns by warp group: (byte offset of the token's row of sums, factor).
struct alignas(16) XoMeta {
    uint2 col[kXoGroups][kXoNB + 8];
    float gate[kXoGroups][kXoNB + 8];
    float so[128], bo[128];                  // the slab's channel scales and biases
    int2 span[kXoGroups];                    // first column, columns
};

struct alignas(16) XoShared {
    uint64_t full[2][kXoMaxStages];          // weight tile, pairs' rows landed (bytes)
    uint64_t empty[kXoMaxStages];
    uint64_t acc_full[kXoAcc];
    uint64_t acc_empty[kXoAcc];
    uint64_t mma_done;
    uint32_t tmem_base;
    volatile int abort;
    int refused;                             // an earlier error, written once, before the first barrier
    int n_ent;
    uint32_t ent[kXoMaxEnt];                 // expert << 24 | (pairs - 1) << 16 | first pair in its list
    XoMeta meta[kXoAcc];
};

// Eight columns of an accumulator scaled and added to their tokens' rows of sums (`my`: this
// channel's word of row 0).  The columns of one entry are different tokens (but for the
// spare row's, whose sum nobody reads), so all loads go before the stores.
__device__ __forceinline__ void xo_add(uint32_t taddr, const uint2* col, const float* gate, uint32_t my, float so,
                                       float bo, bool biased) {
    uint32_t v[8], at[8];
    float f[8], s[8];
    tmem_ld_32x32b_x8(taddr, v);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const uint4 u = *reinterpret_cast<const uint4*>(col + i);
        at[i] = my + u.x;
        f[i] = __uint_as_float(u.y);
        at[i + 1] = my + u.z;
        f[i + 1] = __uint_as_float(u.w);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = ld_shared_f32(at[i]);
    if (biased) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = fmaf(gate[i], bo, s[i]);
    }
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 8; ++i) st_shared_f32(at[i], fmaf((float)(int)v[i] * so, f[i], s[i]));
}

}  // namespace

__global__ void __launch_bounds__(kXoThreads, 1)
int8_experts_out_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_h16,
                        const __grid_constant__ CUtensorMap tm_h32, const __grid_constant__ CUtensorMap tm_h64,
                        const X8Out a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int NB = 1 << a.lgNB, TT = a.TT, S = a.S;
    const int stage_bytes = kXTile + (128 << a.lgNB);
    float* acc = reinterpret_cast<float*>(smem + (size_t)a.stages * stage_bytes);   // [TT + 1][128]
    XoShared& sh = *reinterpret_cast<XoShared*>(reinterpret_cast<uint8_t*>(acc) + (size_t)(TT + 1) * 512);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = S > 1 ? (int)cluster_ctarank() : 0;
    const int slab = S > 1 ? (int)cluster_id_x() : (int)blockIdx.x, t0 = (int)blockIdx.y * TT;

    if (threadIdx.x == 0) {
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(&sh.full[0][i], 1);
            mbar_init(&sh.full[1][i], 1);
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < kXoAcc; ++i) {
            mbar_init(&sh.acc_full[i], 2);                 // the MMAs and the list of columns
            mbar_init(&sh.acc_empty[i], 4 * kXoGroups);
        }
        mbar_init(&sh.mma_done, 1);
        fence_mbar_init();
        sh.abort = 0;
        prefetch_tmap(&tm_w);
        prefetch_tmap(&tm_h16);
        prefetch_tmap(&tm_h32);
        prefetch_tmap(&tm_h64);
    }
    if (warp == 2) {
        tmem_alloc(&sh.tmem_base, kXoTmem);
        tmem_relinquish();
    }
    for (int i = threadIdx.x; i < TT * 32; i += kXoThreads) reinterpret_cast<float4*>(acc)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    griddep_wait();
    griddep_launch_dependents();
    if (warp == 3) {
        // the tile's pairs, by expert, in pieces of at most NB
        const int c0 = t0 >> 5, c1 = min(a.w.C32, (t0 + TT) >> 5);
        const int status = __ldcg(&a.ctl->status);
        int lo[8], hi[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = 32 * i + lane;
            lo[i] = hi[i] = 0;
            // (after an earlier error the tables may be another call's: no entries then)
            if (e < a.E && status == 0) {
                lo[i] = __ldcg(a.w.tpos + (size_t)e * (a.w.C32 + 1) + c0);
                hi[i] = __ldcg(a.w.tpos + (size_t)e * (a.w.C32 + 1) + c1);
            }
        }
        int run = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (32 * i >= a.E) break;
            const int ne = (hi[i] - lo[i] + NB - 1) >> a.lgNB;
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
            sh.n_ent = run;   // (0 after an earlier error)
            sh.refused = status != 0;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;
    const uint64_t limit = a.wait_ns;
    const int ents = sh.n_ent;
    // this block's share (at most 1024 entries: fp32 quotients are exact)
    const float per_rank = __fdividef(1.f, (float)S);
    const int m0 = (int)(((float)(ents * rank) + 0.25f) * per_rank);
    const int m1 = (int)(((float)(ents * (rank + 1)) + 0.25f) * per_rank);

    if (warp == 0 || warp == 2) {
        // Warp 0 loads weight tiles, warp 2 the pairs' rows of h: one thread issues a TMA
        // copy every few hundred cycles, so the two operands have an issuer each.
        if (elect_one()) {
            uint64_t* const full = sh.full[warp >> 1];
            const uint64_t pol = policy_evict_normal();
            int st = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int m = m0; m < m1 && ok; ++m) {
                const uint32_t en = sh.ent[m];
                const int e = (int)(en >> 24), n = (int)(en >> 16 & 255u) + 1;
                const int row = e * a.w.Tcap + (int)(en & 0xffffu);
                for (int kb = 0; kb < a.KBe; ++kb) {
                    ok = wait_bar(&sh.empty[st], ph ^ 1u, limit, &sh.abort, a.ctl, kWaitEmpty);
                    if (!ok) break;
                    uint8_t* sp = smem + (size_t)st * stage_bytes;
                    if (warp == 0) {
                        mbar_arrive_expect_tx(&full[st], (uint32_t)kXTile);
                        tma_load_2d(sp, &tm_w, &full[st], kb * 128, e * a.d_h + slab * 128, pol);
                    } else if (n <= 16) {
                        mbar_arrive_expect_tx(&full[st], 16u * 128u);
                        tma_load_2d(sp + kXTile, &tm_h16, &full[st], kb * 128, row, pol);
                    } else if (n <= 32) {
                        mbar_arrive_expect_tx(&full[st], 32u * 128u);
                        tma_load_2d(sp + kXTile, &tm_h32, &full[st], kb * 128, row, pol);
                    } else {
                        mbar_arrive_expect_tx(&full[st], 64u * 128u);
                        tma_load_2d(sp + kXTile, &tm_h64, &full[st], kb * 128, row, pol);
                    }
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
                wait_bar_drain(&full[st], (uint32_t)(((issued - 1 - i) / a.stages) & 1), limit, a.ctl);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        const uint64_t desc0 = sw128_kmajor_desc(smem_u32(smem));
        if (elect_one()) {
            int st = 0, buf = 0;
            uint32_t ph = 0, bph = 0;
            bool ok = true;
            for (int m = m0; m < m1 && ok; ++m) {
                const uint32_t idesc = idesc_i8_s32(128, (int)((sh.ent[m] >> 16 & 255u) + 16) & ~15);
                ok = wait_bar(&sh.acc_empty[buf], bph ^ 1u, limit, &sh.abort, a.ctl, kWaitAccEmpty);
                if (!ok) break;
                for (int kb = 0; kb < a.KBe; ++kb) {
                    ok = wait_bar(&sh.full[0][st], ph, limit, &sh.abort, a.ctl, kWaitFullW) &&
                         wait_bar(&sh.full[1][st], ph, limit, &sh.abort, a.ctl, kWaitFullH);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t ad = desc0 + (uint64_t)((uint32_t)st * (uint32_t)stage_bytes >> 4);
                    const uint64_t bd = ad + (kXTile >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_i8(tmem + (uint32_t)(buf * kXoNB), ad + 2 * k, bd + 2 * k, idesc, kb > 0 || k > 0);
                    umma_commit(&sh.empty[st]);
                    if (kb == a.KBe - 1) umma_commit(&sh.acc_full[buf]);
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
            umma_commit(&sh.mma_done);
            wait_bar_drain(&sh.mma_done, 0u, limit, a.ctl);
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 8) {
        // What the epilogue needs of each entry (the four warps in turn, reading kAhead of their
        // entries ahead: the loads' latency is several entries' time): the channels' scales
        // and biases, and every epilogue group's columns as (byte offset of the token's row of
        // sums, factor).  Tokens ascend, so a group's columns are neighbours.  Columns of the
        // spare row follow each list: the epilogue takes eight at a time.
        constexpr int kAhead = 2;
        float4 p0[kAhead], p1[kAhead], so[kAhead], bo[kAhead];
        const bool biased = a.b_out != nullptr;
        auto fetch = [&](int m, int k) {
            if (m >= m1) return;
            const uint32_t en = sh.ent[m];
            const int n = (int)(en >> 16 & 255u) + 1;
            const float4* src = a.w.pair + (size_t)(en >> 24) * a.w.Tcap + (en & 0xffffu);
            if (lane < n) p0[k] = __ldcg(src + lane);
            if (lane + 32 < n) p1[k] = __ldcg(src + lane + 32);
            const size_t ch = (size_t)(en >> 24) * a.d_h + slab * 128 + lane * 4;
            so[k] = __ldg(reinterpret_cast<const float4*>(a.s_out + ch));
            if (biased) bo[k] = __ldg(reinterpret_cast<const float4*>(a.b_out + ch));
        };
        const int mw = m0 + warp - 4;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            p0[k] = p1[k] = so[k] = bo[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            fetch(mw + 4 * k, k);
        }
        bool ok = true;
        const int part = 31 - __clz(TT / kXoGroups);   // a group's tokens: 2^part
        for (int mb = mw; mb < m1 && ok; mb += 4 * kAhead) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int m = mb + 4 * k;
                if (m >= m1) break;
                const int slot = (m - m0) % kXoAcc;
                ok = wait_bar_warp(&sh.acc_empty[slot], (uint32_t)((m - m0) / kXoAcc & 1) ^ 1u, limit, &sh.abort, a.ctl,
                                   kWaitEmpty);
                if (!ok) break;
                const int n = (int)(sh.ent[m] >> 16 & 255u) + 1;
                XoMeta& mt = sh.meta[slot];
                reinterpret_cast<float4*>(mt.so)[lane] = so[k];
                if (biased) reinterpret_cast<float4*>(mt.bo)[lane] = bo[k];
                const int r0 = __float_as_int(p0[k].x) & (TT - 1), r1 = __float_as_int(p1[k].x) & (TT - 1);
                const int g0 = lane < n ? r0 >> part : kXoGroups, g1 = lane + 32 < n ? r1 >> part : kXoGroups;
                int from = 0;   // columns before group g
#pragma unroll
                for (int g = 0; g < kXoGroups; ++g) {
                    const int cn = __popc(__ballot_sync(0xffffffffu, g0 == g)) + __popc(__ballot_sync(0xffffffffu, g1 == g));
                    if (g0 == g) {
                        mt.col[g][lane - from] = make_uint2((uint32_t)r0 * 512u, __float_as_uint(p0[k].y));
                        mt.gate[g][lane - from] = p0[k].z;
                    }
                    if (g1 == g) {
                        mt.col[g][lane + 32 - from] = make_uint2((uint32_t)r1 * 512u, __float_as_uint(p1[k].y));
                        mt.gate[g][lane + 32 - from] = p1[k].z;
                    }
                    if (lane < 8) {
                        mt.col[g][cn + lane] = make_uint2((uint32_t)TT * 512u, 0u);
                        mt.gate[g][cn + lane] = 0.f;
                    }
                    if (lane == g) mt.span[g] = make_int2(from, cn);
                    from += cn;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.acc_full[slot]);
                fetch(m + 4 * kAhead, k);
            }
        }
        __syncwarp();
    } else if (warp >= 8) {
        // A warp group owns its part of the tile's tokens (a thread one channel of them), so no
        // sum is touched by two warps and the groups need not meet.
        const int q = warp & 3, group = (warp - 8) >> 2, ch = q * 32 + lane;
        const bool biased = a.b_out != nullptr;
        int buf = 0;
        uint32_t bph = 0;
        const uint32_t my = smem_u32(acc) + (uint32_t)ch * 4u;
        uint32_t got = 0;
        for (int m = m0; m < m1; ++m) {
            if (!wait_tested(got, &sh.acc_full[buf], bph, limit, &sh.abort, a.ctl, kWaitAccFull)) break;
            tc_fence_after();
            const int nbuf = buf + 1 == kXoAcc ? 0 : buf + 1;
            const uint32_t nbph = nbuf == 0 ? bph ^ 1u : bph;
            got = mbar_test_wait(&sh.acc_full[nbuf], nbph);
            const int2 span = sh.meta[buf].span[group];
            const uint2* col = sh.meta[buf].col[group];
            const float* gate = sh.meta[buf].gate[group];
            const float so = sh.meta[buf].so[ch], bo = biased ? sh.meta[buf].bo[ch] : 0.f;
            const uint32_t tacc = tmem + (uint32_t)(buf * kXoNB + span.x) + ((uint32_t)(q * 32) << 16);
#pragma unroll 1
            for (int c = 0; c < span.y; c += 8) xo_add(tacc + (uint32_t)c, col + c, gate + c, my, so, bo, biased);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.acc_empty[buf]);
            buf = nbuf;
            bph = nbph;
        }
    }
    // y: the blocks of the cluster add their rows in rank order, each its share of the tokens
    if (S > 1) cluster_barrier_sync();
    else __syncthreads();
    if (!sh.refused && sh.abort == 0) {
        // (a thread four channels of a row)
        const int ra = (int)(((float)(TT * rank) + 0.25f) * per_rank);
        const int rb = min((int)(((float)(TT * (rank + 1)) + 0.25f) * per_rank), a.T - t0);
#pragma unroll 1
        for (int i = ra * 32 + (int)threadIdx.x; i < rb * 32; i += kXoThreads) {
            const float* p = acc + i * 4;
            float4 f = *reinterpret_cast<const float4*>(p);
            if (S > 1) {
                float4 u[8];   // all ranks' rows in flight at once
                const uint32_t off = smem_u32(p);
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    u[r] = r < S ? ld_shared_cluster_f4(mapa_shared(off, (uint32_t)r)) : make_float4(0.f, 0.f, 0.f, 0.f);
                f = u[0];
#pragma unroll
                for (int r = 1; r < 8; ++r) {
                    f.x += u[r].x;
                    f.y += u[r].y;
                    f.z += u[r].z;
                    f.w += u[r].w;
                }
            }
            const __nv_bfloat162 b0 = __floats2bfloat162_rn(f.x, f.y), b1 = __floats2bfloat162_rn(f.z, f.w);
            *reinterpret_cast<uint2*>(a.y + (size_t)(t0 + (i >> 5)) * a.d_h + slab * 128 + (i & 31) * 4) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
        }
    }
    if (S > 1) cluster_barrier_sync_relaxed();   // no block leaves while its rows may be read
    tc_fence_before();
    __syncthreads();
    if (warp == 2) tmem_dealloc(tmem, kXoTmem);
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
    static SmemOptIn opt_in;
    cudaError_t e = opt_in(kern);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[2];
    cudaLaunchConfig_t cfg = x8_config(grid, XiCfg<MT>::kThreads, smem, s, at, a.CS);
    return cudaLaunchKernelEx(&cfg, kern, maps[0], maps[1], a);
}

}  // namespace

cudaError_t launch_int8_prepare(const __nv_bfloat16* x, const float* gates, int T, int d_h, int E, const X8Bufs& w,
                                Ctl* ctl, cudaStream_t s) {
    const QuantPlan p = quantize_plan(T, d_h, 2);
    const int per = kQThreads >> p.lgW;
    cudaLaunchAttribute at[2];
    cudaLaunchConfig_t cfg = x8_config(E + (T + per - 1) / per, kQThreads, 0, s, at, 1);
    if (p.C == 0) return cudaLaunchKernelEx(&cfg, int8_prepare_kernel<0>, x, gates, T, d_h, E, p.lgW, w, ctl);
    if (p.C == 2) return cudaLaunchKernelEx(&cfg, int8_prepare_kernel<2>, x, gates, T, d_h, E, p.lgW, w, ctl);
    if (p.C == 4) return cudaLaunchKernelEx(&cfg, int8_prepare_kernel<4>, x, gates, T, d_h, E, p.lgW, w, ctl);
    return cudaLaunchKernelEx(&cfg, int8_prepare_kernel<8>, x, gates, T, d_h, E, p.lgW, w, ctl);
}

// Tokens per tile and blocks per cluster.  A tile of all an expert's tokens reads its
// weight once, so N grows with T, up to what two accumulators of all d_e rows leave of
// TMEM (2 * d_e / 128 * N <= 512 columns).  Where
// the tiles may be fewer than the SMs, clusters let several blocks share a tile.
cudaError_t launch_int8_experts_in(X8In a, const CUtensorMap* maps, int sms, cudaStream_t s) {
    const int MT = a.d_e / 128, stage = MT * kXTile + (128 << a.lgN);
    a.stages = kXRing / stage < kXMaxStages ? kXRing / stage : kXMaxStages;
    const size_t smem = 1024 + (size_t)a.stages * stage + sizeof(XiShared);
    const int fit = a.CS > 1 ? int8_cluster_capacity()[a.CS] * a.CS : sms;
    const int grid = fit > 0 ? fit : sms / a.CS * a.CS;
    switch (MT) {
        case 1: return launch_in<1>(a, maps, grid, smem, s);
        case 2: return launch_in<2>(a, maps, grid, smem, s);
        case 3: return launch_in<3>(a, maps, grid, smem, s);
        default: return launch_in<4>(a, maps, grid, smem, s);
    }
}

cudaError_t launch_int8_experts_out(X8Out a, const CUtensorMap* maps, cudaStream_t s) {
    const int stage = kXTile + (128 << a.lgNB);
    const int room = (kMaxSmem - 1024 - (int)sizeof(XoShared) - (a.TT + 1) * 512) / stage;
    a.stages = room < kXoMaxStages ? room : kXoMaxStages;
    const size_t smem = 1024 + (size_t)a.stages * stage + (size_t)(a.TT + 1) * 512 + sizeof(XoShared);
    auto kern = int8_experts_out_kernel;
    static SmemOptIn opt_in;
    cudaError_t e = opt_in(kern);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[2];
    cudaLaunchConfig_t cfg = x8_config(a.slabs * a.S, kXoThreads, smem, s, at, a.S);
    cfg.gridDim.y = (unsigned)((a.T + a.TT - 1) / a.TT);
    return cudaLaunchKernelEx(&cfg, kern, maps[0], maps[1], maps[2], maps[3], a);
}

}  // namespace bffn
