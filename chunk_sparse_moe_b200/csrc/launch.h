// launch.h -- host-side launchers of the BlockFFN kernels (internal to the
// library; the public interface is include/blockffn.h).
#pragma once
#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace bffn {

// bf16 matrix [rows, cols] as a 3-D TMA tensor {64, row, column block}; a box
// {64, box_rows, nkb} lands as nkb consecutive [box_rows x 128 B] 128-byte-
// swizzled tiles (defined in abi.cu)
bool make_map_kblocks(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint32_t box_rows,
                      uint32_t nkb);

cudaError_t launch_route(const void* x, const void* W_r, const float* b_r, const float* gamma,
                         float eps, int T, int d_h, int E, bool bf16, float* gates,
                         cudaStream_t s);

// ctl: nothing is written after an error recorded there (nullptr: no such call before it)
cudaError_t launch_residual_layernorm(const void* y, const void* x, const float* ln_gamma, const float* ln_beta,
                                      float eps, int T, int d_h, bool bf16, void* out, cudaStream_t s,
                                      const Ctl* ctl = nullptr);

cudaError_t launch_chunk_union(const float* gates, int T, int E, int n, int32_t* counts,
                               int32_t* idx, uint32_t* tmask, cudaStream_t s);

// compute_union: tables from the gates; otherwise the caller's tables are checked
// (a mismatch records an error in ctl and the forward computes nothing)
cudaError_t launch_chunk_union_plan(const float* gates, int T, int E, int n, int32_t* counts,
                                    int32_t* idx, uint32_t* tmask, bool compute_union, Ctl* ctl,
                                    int32_t* offsets, int32_t* pair_ce, void* y, int d_h,
                                    int y_elem_bytes, cudaStream_t s);

// group tables of the multi-chunk forward (see union.cu)
cudaError_t launch_group_plan(const float* gates, int T, int E, int n, int32_t* counts, int32_t* idx,
                              uint32_t* tmask, bool compute_union, Ctl* ctl, int NG, int NGr,
                              int32_t* gcounts, int32_t* goffsets, int32_t* gpair, __nv_bfloat16* y,
                              int d_h, cudaStream_t s);

// b_in [E, d_e] and b_out [E, d_h] fp32 expert biases, or nullptr
cudaError_t launch_forward_f32(const float* x, const float* gates, const float* W_in,
                               const float* W_out, const float* b_in, const float* b_out,
                               const int32_t* counts, const int32_t* offsets,
                               const int32_t* pair_ce, const uint32_t* tmask, const Ctl* ctl,
                               float* hbuf, int T, int d_h, int E, int d_e, int n, float* y,
                               int num_sms, cudaStream_t s);

// ybias[t, :] = sum over the union of t's chunk (ascending) of the gate-masked
// fc2 biases, bit_t ? g[t,e] b_out[e,:] : 0, fp32 [T, d_h] (expert_bias.cu)
cudaError_t launch_expert_bias_sum(const float* gates, const int32_t* counts, const int32_t* idx,
                                   const uint32_t* tmask, const Ctl* ctl, const float* b_out, int T,
                                   int d_h, int E, int n, float* ybias, cudaStream_t s);

// Arguments of the multi-chunk group forward (forward_group.cu).
struct GrArgs {
    const float* gates;       // [T, E]
    const uint32_t* tmask;    // [C, E] chunk token masks
    const int32_t* gcounts;   // [NGr] size of each group's expert set
    const int32_t* goffsets;  // [NGr + 1]
    const int32_t* gpair;     // [P] (group << 8) | expert, by group, experts ascending
    __nv_bfloat16* hbuf;      // [P][N][d_e] gated activations h'
    float* partB;             // [grid][2][N*128] split-expert partial sums (expert-out)
    uint32_t* readyA;         // [2][cnt_a_len] expert-in units whose h' is written
    uint32_t* cntB;           // [2][cnt_b_len] blocks that published an expert-out partial
    long long cnt_a_len;      // NGr*E*MT
    long long cnt_b_len;      // NGr*RT
    Ctl* ctl;
    __nv_bfloat16* y;         // [T, d_h]
    const float* b_in;        // [E, d_e] fc1 biases, or nullptr
    const float* ybias;       // [T, d_h] per-token fc2 bias sums (expert_bias.cu), or nullptr
    int T, d_h, E, d_e, n;
    int N;     // tokens per MMA: 128 or 256
    int NT;    // tokens per group: (N / n) * n
    int NGr;   // groups
    int KB, MT, RT, KBe;
    int skip_flag_unit;       // test support: unit whose h' is never announced ready (-1: off)
    unsigned long long wait_ns;
    unsigned long long shape_key;
    unsigned long long* trace;   // optional [grid][64] globaltimer stamps (nullptr: off)
};
// maps: x [T, d_h] (box {64, N}), W_in [E*d_e, d_h] and W_out [E*d_h, d_e] (box
// {64, 128}), h' [P*N, d_e] (box {64, N}): 2-D, bf16, 128-byte swizzle; the
// expert-out partial tiles as fp32 lines of 512 floats (box {128, N/4}, no swizzle)
cudaError_t launch_forward_group(const GrArgs& a, const CUtensorMap* maps, int grid, cudaStream_t s);

// Arguments of the single-chunk forward (see forward_decode.cu): expert-in
// units are (union expert, 128-row tile of W_in) split along K over a pair of
// blocks (a cluster of 2); expert-out row tiles are split over blocks and
// reduced in two passes.
struct DcArgs {
    const float* gates;       // [T, E], T <= n
    // the caller's union tables of the chunk (counts [1], idx [E], tmask [E]), or
    // all nullptr: the kernel forms the union from the gates
    const int32_t* counts_in;
    const int32_t* idx_in;
    const uint32_t* tmask_in;
    __nv_bfloat16* y;         // [T, d_h]
    __nv_bfloat16* hbuf;      // [E slots][N][d_e] gated activations h'
    uint32_t* readyA;         // [2][E] halves of an expert slot written, by launch parity
    Ctl* ctl;
    const float* b_in;        // [E, d_e] fc1 biases, or nullptr
    const float* b_out;       // [E, d_h] fc2 biases, or nullptr
    int T, d_h, E, d_e, n, N;
    int KB;    // d_h / 64
    int RT;    // d_h / 128
    int skip_unit;            // test support: expert-in half never counted in (-1: off)
    unsigned long long wait_ns;
    unsigned long long* trace;   // optional [grid][64] globaltimer stamps
    unsigned long long shape_key;   // the workspace layout this launch expects (Ctl::shape_key)
};
// maps: x [T, d_h] (box N rows), W_in [E*d_e, d_h] and W_out [E*d_h, d_e] (box 128
// rows), h' [E*N, d_e] (box N rows): 3-D {64, rows, column block} boxes of two
// 64-wide column blocks, 128-byte swizzle; y [T, d_h] (box 32 wide x N rows, no
// swizzle, for stores)
cudaError_t launch_forward_decode(const DcArgs& a, const CUtensorMap* maps, int grid, cudaStream_t s);
size_t forward_decode_smem_bytes();
// clusters of 4 blocks that can be resident at once (the launch uses 4 x this
// many blocks), -1 on error
int decode_max_clusters();

// top-k routing from logits and its gradient (route_topk.cu); bias and gates may be
// nullptr
cudaError_t launch_route_topk(const void* logits, bool bf16, const float* bias, int T, int E, int k, bool sigmoid,
                              int n_group, int topk_group, bool renorm, float scale, float* gates, int32_t* ids,
                              float* weights, cudaStream_t s);
cudaError_t launch_route_topk_backward(const void* logits, bool bf16, const int32_t* ids, const float* d_weights, int T,
                                       int E, int k, bool sigmoid, bool renorm, float scale, void* d_logits,
                                       cudaStream_t s);

// rows of K values rounded to 8 bits, one scale per row (int8_linear.cu); ctl: the control
// block of the workspace that q and scale are in, or nullptr
cudaError_t launch_quantize_rows(const void* v, bool bf16, int rows, int K, int8_t* q, float* scale, Ctl* ctl,
                                 cudaStream_t s);

// A kernel's permission to use 227 KB of shared memory, asked for once per device (one
// static object for each kernel).
class SmemOptIn {
  public:
    template <typename K>
    cudaError_t operator()(K kern) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const unsigned long long bit = 1ull << (dev & 63);
        if (done_.load(std::memory_order_relaxed) & bit) return cudaSuccess;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e == cudaSuccess) done_.fetch_or(bit, std::memory_order_relaxed);
        return e;
    }

  private:
    std::atomic<unsigned long long> done_{0};
};

// Arguments of the 8-bit integer product (int8_linear.cu).
struct IlArgs {
    const float* sx;          // [T] token scales
    const float* sw;          // [O] channel scales
    const float* bias;        // [O] or nullptr
    void* y;                  // [T, O]
    Ctl* ctl;
    int T, O;
    int KP;                   // 128-byte blocks of K in a pipeline stage (1 or 2)
    int KB;                   // stages that K takes
    int N, S;                 // tokens per tile, blocks per tile (K split)
    bool pair;                // pairs of blocks, tiles of 256 x 256 (cta_group::2)
    int tiles_o, tiles_t;
    int stages;               // set by the launcher
    int kb_lo[9];             // first K block of each of the S blocks (set by the launcher)
    unsigned long long wait_ns;
};
const int* int8_cluster_capacity();   // [9], by blocks per cluster
void int8_linear_plan(int T, int K, int O, int sms, int* N, int* S, bool* pair);
// maps: W [O, K] (box {128, 128}) and q [T, K] (box {128, N}; pair: {128, 128}), bytes, 128-byte swizzle;
// KP = 2: as blocks of 128 columns, boxes of two
cudaError_t launch_int8_linear(IlArgs a, const CUtensorMap* maps, bool bf16_out, int sms, cudaStream_t s);

// Scratch of the 8-bit expert sum (forward_int8.cu), for a slice of up to Tcap tokens.
struct X8Bufs {
    int8_t* xq;               // [Tcap, d_h] the tokens in 8 bits
    float* sx;                // [Tcap] their scales
    int32_t* counts;          // [E] tokens of each expert
    int32_t* list;            // [E, Tcap] the tokens of each expert, ascending
    int32_t* tpos;            // [E, C32 + 1] how many of them come before token 32 c (last: all)
    float4* pair;             // [E, Tcap] of each listed token: its index (bits), gate * scale of h, gate, 0
    int8_t* hq;               // [E * Tcap, d_e] h of each listed token in 8 bits
    int Tcap;
    int C32;                  // ceil(T / 32) of the slice
};
cudaError_t launch_int8_prepare(const __nv_bfloat16* x, const float* gates, int T, int d_h, int E, const X8Bufs& w,
                                Ctl* ctl, cudaStream_t s);

struct X8In {
    X8Bufs w;
    const float* gates;       // [T, E]
    const float* s_in;        // [E, d_e]
    const float* b_in;        // [E, d_e] or nullptr
    Ctl* ctl;
    int T, E, d_e;
    int KB;                   // d_h / 128
    int lgN;                  // 2^lgN tokens per tile, at most
    int CS;                   // blocks per cluster
    int stages;               // set by the launcher
    unsigned long long wait_ns;
};
// maps: W_in [E * d_e, d_h] (box {128, 128}) and xq [T, d_h] (box {128, 2^lgN}, used when T <= 2^lgN)
cudaError_t launch_int8_experts_in(X8In a, const CUtensorMap* maps, int sms, cudaStream_t s);

struct X8Out {
    X8Bufs w;
    const float* s_out;       // [E, d_h]
    const float* b_out;       // [E, d_h] or nullptr
    __nv_bfloat16* y;         // [T, d_h]
    Ctl* ctl;
    int T, E, d_h;
    int KBe;                  // d_e / 128
    int slabs;                // d_h / 128
    int TT;                   // tokens per tile (a multiple of 32)
    int lgNB;                 // 2^lgNB pairs multiplied at a time, at most (16, 32 or 64)
    int S;                    // blocks per cluster
    int stages;               // set by the launcher
    unsigned long long wait_ns;
};
// maps: W_out [E * d_h, d_e] (box {128, 128}) and hq [E * Tcap, d_e] (boxes {128, 16 | 32 | 64})
cudaError_t launch_int8_experts_out(X8Out a, const CUtensorMap* maps, cudaStream_t s);

}  // namespace bffn
