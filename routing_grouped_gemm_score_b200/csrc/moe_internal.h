// moe_internal.h -- launchers shared between the kernel files and the C ABI.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/moe_b200.h"

namespace moe {

using bf16 = __nv_bfloat16;

// Whether the kernels that this host thread launches for its current call are
// chained (programmatic dependent launch). Chaining hides each kernel's launch
// and prologue behind the end of the kernel before it, which pays in calls of
// a few rows, where those fixed costs are most of the time (measured on B200:
// a one-token layer forward 60 -> 49 us). In large calls it cost 2.5-4 %, so
// the entry points turn it on by the call's size (ChainScope, kChainMaxRows).
bool& chained_launches();   // thread-local, moe_api.cu
constexpr int64_t kChainMaxRows = 4096;
struct ChainScope {
    bool prev;
    explicit ChainScope(bool on) : prev(chained_launches()) { chained_launches() = on; }
    ~ChainScope() { chained_launches() = prev; }
};

// Launches a kernel of a layer call, chained when chained_launches() says so:
// it may then be scheduled before the previous kernel in the stream has
// finished, and it calls pdl_wait() (moe_common.cuh) before it touches data
// that other kernels write or read (without a chain pdl_wait returns at once).
template <class... KArgs, class... Args>
cudaError_t launch_chained(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                           Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = chained_launches() ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<Args&&>(args)...);
}

// Allows a kernel `bytes` of dynamic shared memory, once per device (the setting
// belongs to the current device); a failure is tried again on the next call.
struct PerDeviceFlag {
    std::atomic<bool> done[64] = {};
};
template <class K>
cudaError_t allow_smem(K kern, size_t bytes, PerDeviceFlag& flag) {
    int device = 0;
    const cudaError_t got = cudaGetDevice(&device);
    if (got != cudaSuccess) return got;
    const bool known = device >= 0 && device < 64;
    if (known && flag.done[device].load(std::memory_order_acquire)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && known) flag.done[device].store(true, std::memory_order_release);
    return e;
}

// Values in the 8-bit row format and their scale bytes (rows8.cuh, rows8.cu).
// Rows of parts * cols columns (parts 1 or 2, each with its own blocks); scales
// [rows][parts * S], or [parts * S][rows] when block_major, S = ceil(cols / 32).
struct Rows8 {
    uint8_t* q = nullptr;
    uint8_t* scale = nullptr;
};

// Tokens handled by one block of the router / rank kernels (a power of two,
// 8..64). Ranks inside an expert block are counted per such token block, then
// offset by a scan. Small batches use small token blocks so that every SM gets
// work; large ones use 64 to keep the per-block counts ([E][blocks]) small.
constexpr int kMaxTokensPerRouteBlock = 64;

inline int route_tokens_per_block(int64_t T) {
    if (T <= 8192) return 8;
    if (T <= 32768) return 16;
    if (T <= 131072) return 32;
    return 64;
}

inline int64_t route_blocks(int64_t T) {
    const int tpb = route_tokens_per_block(T);
    return (T + tpb - 1) / tpb;
}

// Scratch of the routing path, carved from the caller's workspace.
struct RouteScratch {
    int32_t* block_base;  // [E][nb]: per-(expert, token block) counts, then exclusive prefix
    int32_t* local_rank;  // [T][k]: rank of the assignment inside its token block
    unsigned* ticket;     // last-block-done counter of the scan kernel
};
size_t route_scratch_bytes(int64_t T, int E, int k);
RouteScratch carve_route_scratch(void* base, int64_t T, int E, int k);

// With counts and offsets given and a single token block (T <= 8 tokens), the
// router also writes the counts and offsets and sets *scanned; otherwise
// launch_expert_scan must follow. Whichever writes the offsets also sets
// zero[0 .. n_zero) to 0 (the fused expert MLP's schedule counters; NULL: none).
// When the router writes them, x, x_perm, sorted_token, row_of and permuted
// are given and the permuted rows take at most 64 KB, it also does the permute
// (x [T][H] into x_perm [T k][H]) and sets *permuted; otherwise
// launch_permute must follow.
cudaError_t launch_router_topk(const float* logits, int64_t T, int E, int k,
                               const moe_router_opts& opts, int32_t* topk_idx, float* topk_prob,
                               uint8_t* routing_map, const RouteScratch& rs, cudaStream_t st,
                               unsigned* err, int32_t* counts = nullptr, int32_t* offsets = nullptr,
                               bool* scanned = nullptr, int32_t* zero = nullptr, int n_zero = 0,
                               const bf16* x = nullptr, int H = 0, bf16* x_perm = nullptr,
                               int32_t* sorted_token = nullptr, int32_t* row_of = nullptr, bool* permuted = nullptr);
cudaError_t launch_router_backward(const float* logits, int64_t T, int E, int k, const moe_router_opts& opts,
                                   const int32_t* topk_idx, const float* dprob, float* dlogits,
                                   cudaStream_t st, unsigned* err);
cudaError_t launch_expert_bias_update(const int32_t* counts, int E, float coeff, float* bias, cudaStream_t st);

// Auxiliary load-balancing loss (aux_loss.cu).
size_t aux_loss_workspace_bytes(int64_t T, int E);
cudaError_t launch_aux_loss(const float* logits, int64_t T, int E, int k, int score_fn, const int32_t* counts,
                            float coeff, float* loss, float* scores, void* ws, cudaStream_t st);
cudaError_t launch_aux_loss_backward(const float* logits, int64_t T, int E, int k, int score_fn,
                                     const int32_t* counts, float coeff, const float* grad_loss, float* dlogits,
                                     int accumulate, cudaStream_t st);
cudaError_t launch_rank_from_indices(const int32_t* topk_idx, int64_t T, int E, int k,
                                     const RouteScratch& rs, cudaStream_t st, unsigned* err);
// Turns block counts into exclusive prefixes; writes counts/offsets if given,
// and then sets zero[0 .. n_zero) to 0 (NULL: none).
cudaError_t launch_expert_scan(int64_t T, int E, const RouteScratch& rs, int32_t* counts,
                               int32_t* offsets, cudaStream_t st, int32_t* zero = nullptr, int n_zero = 0);
// Padded dispatch (Token permutation, Padding and alignment).
cudaError_t launch_pad_offsets(const int32_t* offsets, int E, int align, int32_t* padded_offsets, cudaStream_t st);
cudaError_t launch_pad_fill(const int32_t* offsets, const int32_t* padded_offsets, int E, int H, bf16* x_perm,
                            int32_t* sorted_token, float* prob_perm, cudaStream_t st);
cudaError_t launch_prob_perm(const float* topk_prob, const int32_t* row_of, int64_t n, float* prob_perm,
                             cudaStream_t st);
// row_bound: rows of x_perm and sorted_token (<= 0: T*k, the unpadded dispatch)
// x8: with x_perm, x also goes there in 8 bits, by token (one part, scales by row)
cudaError_t launch_permute(const bf16* x, int64_t T, int H, const int32_t* topk_idx, int k,
                           const int32_t* offsets, int E, const RouteScratch& rs, bf16* x_perm,
                           int32_t* sorted_token, int32_t* row_of, cudaStream_t st, unsigned* err,
                           int64_t row_bound = 0, const Rows8& x8 = Rows8());

// The fixed scratch array behind moe_router_topk_noalloc (routing.cu).
size_t router_noalloc_capacity();
cudaError_t router_noalloc_scratch(void** ptr);

cudaError_t launch_combine(const bf16* y_perm, const int32_t* row_of, const float* probs,
                           int64_t T, int k, int H, int64_t A, const bf16* shared, bf16* out,
                           cudaStream_t st, unsigned* err);
cudaError_t launch_combine_backward(const bf16* dout, const bf16* y_perm, const int32_t* row_of,
                                    const float* probs, int64_t T, int k, int H, int64_t A,
                                    bf16* dy_perm, float* dprob, cudaStream_t st, unsigned* err);
// dy[r] = dout[sorted_token[r]] for r < offsets[E] (-1: a zero row).
cudaError_t launch_gather_rows(const bf16* dout, const int32_t* sorted_token, int64_t T, const int32_t* offsets,
                               int E, int64_t A, int H, bf16* dy, cudaStream_t st, unsigned* err);
// dprob[i] = sum_{q < nq} row_dot[row_of[i] * nq + q], q ascending.
cudaError_t launch_row_dot_sum(const float* row_dot, int nq, const int32_t* row_of, int64_t n, int64_t A,
                               float* dprob, cudaStream_t st, unsigned* err);

cudaError_t launch_quantize_rows(const bf16* x, int64_t rows, int cols, int parts, int block_major, uint8_t* q,
                                 uint8_t* scale, cudaStream_t st);
cudaError_t launch_dequantize_rows(const uint8_t* q, const uint8_t* scale, int64_t rows, int cols, int parts,
                                   int block_major, bf16* x, cudaStream_t st);
// The dispatches of the 8-bit checkpoint's backward, into row blocks padded with
// zero rows to multiples of 16: pad_offsets [E + 1] and pad_row [T][k] (written by
// the first) hold the blocks and each assignment's row. rows has A + 15 min(E, A)
// rows (pad16_rows).
constexpr int64_t pad16_rows(int64_t A, int E) { return A + 15 * (A < E ? A : (int64_t)E); }
// rows[pad_row[t, j]] = src[t], prob_row[row] = prob[t, j] (0 in a zero row), and
// row_from[row] = t k + j, not written in rows that no assignment has
cudaError_t launch_spread_rows(const bf16* src, const int32_t* row_of, const int32_t* offsets, const float* prob,
                               int64_t T, int k, int E, int H, bf16* rows, float* prob_row, int32_t* pad_offsets,
                               int32_t* pad_row, int32_t* row_from, cudaStream_t st, unsigned* err);
// What is left to do by token between the gate_up dgrad and its weight's gradient,
// with pad_row given: dx[t] = sum_j rows[pad_row[t, j]] (each row's dx), then those
// rows become x[t], read back from x8 (the padding zeros); and dprob[t, j] = the sum
// of row_dot [row][nq] over the row.
cudaError_t launch_finish_rows(const Rows8& x8, const int32_t* offsets, int64_t T, int k, int E, int H, bf16* rows,
                               const int32_t* pad_row, const float* row_dot, int nq, bf16* dx, float* dprob,
                               cudaStream_t st);

// RMSNorm with the residual's addition, and its backward (rmsnorm.cu).
constexpr int kRmsnormMaxH = 16384;
cudaError_t launch_rmsnorm(const bf16* x, const bf16* residual, const bf16* weight, int64_t T, int H, float eps,
                           bf16* sum, bf16* y, uint8_t* y_q, uint8_t* y_scale, float* rstd, cudaStream_t st);
size_t rmsnorm_backward_workspace_bytes(int64_t T, int H);
cudaError_t launch_rmsnorm_backward(const bf16* dy, const bf16* s, const bf16* weight, const float* rstd,
                                    const bf16* dsum, int64_t T, int H, bf16* dx, float* dweight, float* partial,
                                    cudaStream_t st, unsigned* err);

// ---------------------------------------------------------------- GEMMs
// Grouped GEMMs on tcgen05. Each returns cudaErrorInvalidValue if a tensor
// map cannot be encoded (bad alignment or extent).
// gate_up + SwiGLU: h[r] = silu(x[r] Wg[e]) * (x[r] Wu[e]); optionally gu[r] = [g | u]
// in bf16 (gu_save) or, from the fp32 accumulators, in 8 bits (gu8: two parts of I
// columns, block-major scales; gu_save is then not written).
// offsets NULL: one group of `rows` rows using the weights of group 0.
// max_group_rows: an upper bound on the rows of any group (0: rows), which
// lets small batches take narrower swap-AB tiles (a layer call passes T: a
// token is routed to an expert at most once).
cudaError_t gemm_gate_up_swiglu(const bf16* x, int64_t rows, const int32_t* offsets, int E, int H,
                                int I, const bf16* w_gate_up, bf16* h, bf16* gu_save,
                                cudaStream_t st, unsigned* err, const float* row_scale = nullptr,
                                int64_t max_group_rows = 0, const Rows8& gu8 = Rows8());
// gate_up + SwiGLU with A row r gathered from x: row sorted_token[r] (-1: a
// zero row) of x [T][H], so no permuted copy of x is needed. Single-CTA tiles
// only; H a multiple of 8 and x 16-byte aligned.
cudaError_t gemm_gate_up_swiglu_gather(const bf16* x, int64_t T, const int32_t* sorted_token, int64_t rows,
                                       const int32_t* offsets, int E, int H, int I, const bf16* w_gate_up, bf16* h,
                                       bf16* gu_save, cudaStream_t st, unsigned* err,
                                       const float* row_scale = nullptr, const Rows8& gu8 = Rows8());
// The expert MLP of a small batch in one launch (gemm_swap_mlp_kernel):
// h = SwiGLU(x W_gate_up) (and gu = [g | u] if gu_save), then y = h W_down,
// on swap-AB tiles. Every expert must hold at most max_group_rows <= 64 rows
// (a layer call passes T). sched: E + 1 int32 that are zero when the launch
// starts (the router or the scan zeroes them). use_fused_mlp says whether a
// call of this many rows, groups and columns of h takes it.
bool use_fused_mlp(int64_t rows, int groups, int64_t max_group_rows, int I);
cudaError_t gemm_expert_mlp_fused(const bf16* x, int64_t rows, const int32_t* offsets, int E, int H, int I,
                                  const bf16* w_gate_up, const bf16* w_down, bf16* h, bf16* gu_save, bf16* y,
                                  int32_t* sched, int64_t max_group_rows, cudaStream_t st, unsigned* err,
                                  const Rows8& gu8 = Rows8());
// Whether the forward gate_up GEMM runs on single-CTA 128-row tiles (not CTA
// pairs, not swap-AB tiles) for this many rows and groups.
bool grouped_gemm_single_tiles(int64_t rows, int groups);
// Whether a group-M GEMM of this many rows and groups runs on CTA-pair tiles.
bool grouped_gemm_pair_tiles(int64_t rows, int groups);
// The shared expert's down GEMM with the token combine folded into its
// epilogue: out[t] = bf16(h[t] Wd + sum_j probs[t,j] y_perm[row_of[t,j]]), the
// sum in fp32 after the product, j ascending. CTA-pair tiles only
// (cudaErrorNotSupported when grouped_gemm_pair_tiles(T, 1) is false).
cudaError_t gemm_down_combine(const bf16* h, int64_t T, int H, int I, const bf16* w_down, const bf16* y_perm,
                              int64_t y_rows, const int32_t* row_of, const float* probs, int k, bf16* out,
                              cudaStream_t st, unsigned* err);
// down: y[r] = h[r] Wd[e]
cudaError_t gemm_down(const bf16* h, int64_t rows, const int32_t* offsets, int E, int H, int I,
                      const bf16* w_down, bf16* y, cudaStream_t st, unsigned* err, int64_t max_group_rows = 0);
// dgrad of down with SwiGLU backward: dh = dy Wd[e]^T, then dgu = [dg | du].
// ScaledSwiGLU (row_dot non-NULL): the forward's h[r] was scaled by
// row_scale[r], so [dg | du] is taken from row_scale[r] * dh, and
// row_dot [rows][ceil(I/64)] gets each 64-column group's sum of
// dh * silu(g) * u (the routing weight's gradient, in parts).
cudaError_t gemm_down_dgrad_swiglu(const bf16* dy, int64_t rows, const int32_t* offsets, int E,
                                   int H, int I, const bf16* w_down, const bf16* gu, bf16* dgu,
                                   cudaStream_t st, unsigned* err, const float* row_scale = nullptr,
                                   float* row_dot = nullptr);
// dgrad of down with the SwiGLU backward from an 8-bit [g | u] (gu8 as above): as
// gemm_down_dgrad_swiglu with row_scale and row_dot, and h[r] = row_scale[r] *
// silu(g) * u, recomputed, for the down weight's gradient. The row blocks of dy and
// of the outputs (offsets) may be padded; gu8's rows are those of gu8_offsets,
// gu8_rows of them, and the rows past them in a block get zeros. So does a row r that no
// assignment has, pad_row[row_from[r]] != r (see launch_spread_rows): it is recorded
// as kErrDeviceCheck, and its dy, which holds anything, is set to zeros as well.
cudaError_t gemm_down_dgrad_swiglu8(bf16* dy, int64_t rows, const int32_t* offsets, int E, int H, int I,
                                    const bf16* w_down, const Rows8& gu8, int64_t gu8_rows, const int32_t* gu8_offsets,
                                    const int32_t* row_from, const int32_t* pad_row, const float* row_scale, bf16* dgu,
                                    bf16* h, float* row_dot, cudaStream_t st, unsigned* err);
// dgrad of gate_up: dx_perm = dgu Wgu[e]^T
cudaError_t gemm_gate_up_dgrad(const bf16* dgu, int64_t rows, const int32_t* offsets, int E, int H,
                               int I, const bf16* w_gate_up, bf16* dx_perm, cudaStream_t st,
                               unsigned* err);
// wgrad: dW[e] = X_e^T D_e over the rows of group e (ragged reduction);
// X [rows, M], D [rows, N], dW [E, M, N]. Empty groups get dW[e] = 0.
// blocks16: every block is a multiple of 16 rows (zero rows at its end), which
// lets it run on CTA pairs.
cudaError_t gemm_wgrad(const bf16* X, const bf16* D, int64_t rows, const int32_t* offsets, int E,
                       int M, int N, bf16* dW, cudaStream_t st, unsigned* err, bool blocks16 = false);

int sm_count();

// Kernel variants forced by moe_testing_set_kernels (MOE_TESTING_AUTO: the
// library's own choice by shape).
struct KernelOverride {
    int gemm_tiles = MOE_TESTING_AUTO;
    int router = MOE_TESTING_AUTO;
    int permute = MOE_TESTING_AUTO;
    int fold_permute = 0;
};
const KernelOverride& kernel_override();

}  // namespace moe
