// rows8.cu -- rows in the 8-bit format of rows8.cuh: to it from bf16 and back,
// and the two dispatches of the 8-bit checkpoint's backward, which write each
// routed row's output gradient and its x, read back from the token's 8-bit row,
// into expert blocks padded to whole K steps of 16 rows.
//
// All of them are bound by HBM bandwidth. A warp owns a unit of up to 1024
// consecutive columns of one row (32 lanes x 4 chunks of 8 columns), its loads
// issued together; four adjacent lanes hold one 32-column block, so a block's
// scale takes two shuffles.
#include "moe_internal.h"
#include "rows8.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxExperts = 256;
constexpr int kChunks = 4;                   // 8-column chunks of a lane in one unit
constexpr int kUnitChunks = 32 * kChunks;    // chunks of a unit (blocks of four chunks, padded)
constexpr int kSpreadChunks = 2;             // the same for the dispatches
constexpr int kSpreadUnit = 32 * kSpreadChunks;

// Quotient and remainder of a unit index by the units of a row.
__device__ __forceinline__ void split_unit(int64_t u, int per_row, int64_t& row, int& part) {
    if (u <= 0xFFFFFFFFll) {
        const uint32_t q = (uint32_t)u / (uint32_t)per_row;
        row = q;
        part = (int)((uint32_t)u - q * (uint32_t)per_row);
    } else {
        row = u / per_row;
        part = (int)(u - row * per_row);
    }
}

// A row of parts * cols columns has parts * S blocks, S = ceil(cols / 32), each
// of four 8-column chunks (those past a part's end are absent). Chunk c of the
// row: its block, and its column in the row, or -1 where it is absent.
__device__ __forceinline__ int chunk_col(int c, int parts, int cols, int S) {
    const int block = c >> 2;
    const int part = block >= S ? 1 : 0;     // parts is 1 or 2
    const int col = (block - part * S) * kRows8Block + (c & 3) * 8;
    return (part < parts && col < cols) ? part * cols + col : -1;
}

// Scale of block b of row r: [rows][parts * S], or [parts * S][rows].
__device__ __forceinline__ int64_t scale_at(int64_t r, int b, int64_t rows, int blocks, int block_major) {
    return block_major ? (int64_t)b * rows + r : r * blocks + b;
}

__global__ void __launch_bounds__(kThreads)
    quantize_rows_kernel(const bf16* __restrict__ x, int64_t rows, int cols, int parts, int block_major,
                         uint8_t* __restrict__ q, uint8_t* __restrict__ scale) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int S = rows8_blocks(cols), blocks = parts * S, width = parts * cols;
    const int per_row = (4 * blocks + kUnitChunks - 1) / kUnitChunks;
    const int64_t units = rows * per_row, nwarps = ((int64_t)gridDim.x * kThreads) >> 5;
    for (int64_t u = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; u < units; u += nwarps) {
        int64_t r;
        int part;
        split_unit(u, per_row, r, part);
        uint4 in[kChunks];
        int col[kChunks];
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            col[i] = chunk_col(part * kUnitChunks + 32 * i + lane, parts, cols, S);
            in[i] = make_uint4(0, 0, 0, 0);
            if (col[i] >= 0) in[i] = __ldg(reinterpret_cast<const uint4*>(x + r * width + col[i]));
        }
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int c = part * kUnitChunks + 32 * i + lane;
            const uint32_t w[4] = {in[i].x, in[i].y, in[i].z, in[i].w};
            float v[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = unpack_bf16x2(w[j]);
                v[2 * j] = f.x;
                v[2 * j + 1] = f.y;
            }
            uint2 packed;
            const uint32_t byte = rows8_quantize_quad(v, packed);
            if (col[i] < 0) continue;   // after the shuffles
            *reinterpret_cast<uint2*>(q + r * width + col[i]) = packed;
            if ((c & 3) == 0) scale[scale_at(r, c >> 2, rows, blocks, block_major)] = (uint8_t)byte;
        }
    }
}

__global__ void __launch_bounds__(kThreads)
    dequantize_rows_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ scale, int64_t rows, int cols,
                           int parts, int block_major, bf16* __restrict__ x) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int S = rows8_blocks(cols), blocks = parts * S, width = parts * cols;
    const int per_row = (4 * blocks + kUnitChunks - 1) / kUnitChunks;
    const int64_t units = rows * per_row, nwarps = ((int64_t)gridDim.x * kThreads) >> 5;
    for (int64_t u = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; u < units; u += nwarps) {
        int64_t r;
        int part;
        split_unit(u, per_row, r, part);
        uint2 in[kChunks];
        uint32_t byte[kChunks];
        int col[kChunks];
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int c = part * kUnitChunks + 32 * i + lane;
            col[i] = chunk_col(c, parts, cols, S);
            if (col[i] < 0) continue;
            in[i] = __ldg(reinterpret_cast<const uint2*>(q + r * width + col[i]));
            byte[i] = __ldg(scale + scale_at(r, c >> 2, rows, blocks, block_major));
        }
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            if (col[i] >= 0) *reinterpret_cast<uint4*>(x + r * width + col[i]) = rows8_dequantize8(in[i], byte[i]);
    }
}

// The row blocks of the backward are padded with zero rows to multiples of 16, a
// K step of the weight gradients: block e starts at pad[e] = sum over e' < e of
// the counts rounded up. Both in shared memory; called by the whole block.
struct PadBlocks {
    int off[kMaxExperts + 1], pad[kMaxExperts + 1];
    int warp_sum[kThreads / 32];
};
static_assert(kThreads >= kMaxExperts, "one thread per expert");

__device__ __forceinline__ void pad_blocks(PadBlocks& b, const int32_t* __restrict__ offsets, int E, int64_t A) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = threadIdx.x;
    for (int i = threadIdx.x; i <= E; i += kThreads) b.off[i] = (int)min(max((int64_t)__ldg(offsets + i), (int64_t)0), A);
    __syncthreads();
    int sum = e < E ? (max(b.off[e + 1] - b.off[e], 0) + 15) / 16 * 16 : 0;   // inclusive prefix
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += v;
    }
    if (lane == 31) b.warp_sum[warp] = sum;
    __syncthreads();
    for (int w = 0; w < warp; ++w) sum += b.warp_sum[w];
    if (e < E) b.pad[e + 1] = sum;
    if (e == 0) b.pad[0] = 0;
    __syncthreads();
}

// Zero rows at the blocks' ends, a warp per row: rows (and prob_row, if given).
__device__ __forceinline__ void zero_pad_rows(const int* off, const int* pad, int E, int chunks, int64_t bound,
                                              uint4* rows, float* prob_row) {
    const int lane = threadIdx.x & 31;
    const int64_t nwarps = ((int64_t)gridDim.x * kThreads) >> 5;
    for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; i < 16 * (int64_t)E; i += nwarps) {
        const int e = (int)(i >> 4);
        const int64_t r = (int64_t)pad[e] + max(off[e + 1] - off[e], 0) + (i & 15);
        if (r >= pad[e + 1] || r >= bound) continue;
        for (int c = lane; c < chunks; c += 32) rows[r * chunks + c] = make_uint4(0, 0, 0, 0);
        if (prob_row != nullptr && lane == 0) prob_row[r] = 0.0f;
    }
}

// One token's row to the k rows that its assignments hold: bf16 as it is (Q8
// false) or read back from 8 bits (Q8 true). Each token's row is read once. A
// warp owns a unit of one token's row (512 columns: with 1024, 8192 rows of 5120
// from 8 bits took 34 us against 27); lane j holds the row of assignment j.
// Q8 false finds the padded rows: the expert of row_of[t, j] by bisection of the
// blocks' offsets, then its place in the padded block. The unit of a token's
// first columns writes pad_row and prob_row, and the first block pad_offsets. A
// row outside its range is recorded and skipped (pad_row -1).
template <bool Q8>
__global__ void __launch_bounds__(kThreads)
    spread_rows_kernel(const void* __restrict__ src, const uint8_t* __restrict__ scale,
                       const int32_t* __restrict__ row_of, const int32_t* __restrict__ offsets,
                       const float* __restrict__ prob, int64_t T, int k, int E, int H, bf16* __restrict__ rows,
                       float* __restrict__ prob_row, int32_t* pad_offsets, int32_t* pad_row, unsigned* err) {
    __shared__ PadBlocks b;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int chunks = H / 8, S = rows8_blocks(H);
    const int per_row = (chunks + kSpreadUnit - 1) / kSpreadUnit;
    const int64_t A = T * k, bound = pad16_rows(A, E);
    const int64_t units = T * per_row, nwarps = ((int64_t)gridDim.x * kThreads) >> 5;
    pad_blocks(b, offsets, E, A);
    if (!Q8 && blockIdx.x == 0)
        for (int i = threadIdx.x; i <= E; i += kThreads) pad_offsets[i] = b.pad[i];
    for (int64_t u = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; u < units; u += nwarps) {
        int64_t t;
        int part;
        split_unit(u, per_row, t, part);
        int32_t mine = -1;
        if (lane < k) {
            if (Q8) {
                mine = __ldg(pad_row + t * k + lane);
            } else {
                const int32_t row = __ldg(row_of + t * k + lane);
                if (row >= 0 && row < A) {
                    int lo = 0, hi = E - 1;   // last expert whose block starts at or before the row
                    while (lo < hi) {
                        const int mid = (lo + hi + 1) >> 1;
                        if (b.off[mid] <= row) lo = mid;
                        else hi = mid - 1;
                    }
                    const int64_t r = (int64_t)b.pad[lo] + (row - b.off[lo]);
                    if (row >= b.off[lo] && row < b.off[lo + 1] && r < bound) mine = (int32_t)r;
                }
                if (mine < 0) raise_error(err, kErrDeviceCheck);
                if (part == 0) {
                    pad_row[t * k + lane] = mine;
                    if (mine >= 0) prob_row[mine] = __ldg(prob + t * k + lane);
                }
            }
        }
        uint4 v[kSpreadChunks];
#pragma unroll
        for (int i = 0; i < kSpreadChunks; ++i) {
            const int c = part * kSpreadUnit + 32 * i + lane;
            if (c >= chunks) continue;
            if (Q8) {
                const uint8_t* qs = static_cast<const uint8_t*>(src) + t * H;
                v[i] = rows8_dequantize8(__ldg(reinterpret_cast<const uint2*>(qs) + c), __ldg(scale + t * S + (c >> 2)));
            } else {
                v[i] = __ldg(reinterpret_cast<const uint4*>(src) + t * chunks + c);
            }
        }
        for (int j = 0; j < k; ++j) {
            const int64_t r = __shfl_sync(0xFFFFFFFFu, mine, j);
            if (r < 0) continue;
            uint4* dst = reinterpret_cast<uint4*>(rows) + r * chunks;
#pragma unroll
            for (int i = 0; i < kSpreadChunks; ++i) {
                const int c = part * kSpreadUnit + 32 * i + lane;
                if (c < chunks) dst[c] = v[i];
            }
        }
    }
    zero_pad_rows(b.off, b.pad, E, chunks, bound, reinterpret_cast<uint4*>(rows), Q8 ? nullptr : prob_row);
}

// Blocks for a warp-per-unit kernel: enough warps for every unit, at most `cap`
// (each warp then loops).
unsigned unit_blocks(int64_t units, int64_t cap) {
    const int64_t need = (units + kThreads / 32 - 1) / (kThreads / 32);
    return (unsigned)(need < cap ? need : cap);
}

// What stays resident, 8 blocks of 256 threads an SM; or a block for every eight
// units. Rows of 5120 and [g | u] rows of 28672 columns (16384 and 8192 rows): to 8
// bits 49 and 131 us resident, 52 and 150 with a block each; back 41 and 133
// against 37 and 108.
int64_t resident_blocks() { return (int64_t)sm_count() * 8; }
constexpr int64_t kEveryBlock = (int64_t)1 << 30;

int64_t format_units(int64_t rows, int cols, int parts) {
    return rows * ((4 * parts * rows8_blocks(cols) + kUnitChunks - 1) / kUnitChunks);
}

}  // namespace

cudaError_t launch_quantize_rows(const bf16* x, int64_t rows, int cols, int parts, int block_major, uint8_t* q,
                                 uint8_t* scale, cudaStream_t st) {
    if (rows == 0) return cudaSuccess;
    return launch_chained(quantize_rows_kernel, dim3(unit_blocks(format_units(rows, cols, parts), resident_blocks())),
                          dim3(kThreads), 0, st, x, rows, cols, parts, block_major, q, scale);
}

cudaError_t launch_dequantize_rows(const uint8_t* q, const uint8_t* scale, int64_t rows, int cols, int parts,
                                   int block_major, bf16* x, cudaStream_t st) {
    if (rows == 0) return cudaSuccess;
    return launch_chained(dequantize_rows_kernel, dim3(unit_blocks(format_units(rows, cols, parts), kEveryBlock)),
                          dim3(kThreads), 0, st, q, scale, rows, cols, parts, block_major, x);
}

cudaError_t launch_spread_rows(const bf16* src, const int32_t* row_of, const int32_t* offsets, const float* prob,
                               int64_t T, int k, int E, int H, bf16* rows, float* prob_row, int32_t* pad_offsets,
                               int32_t* pad_row, cudaStream_t st, unsigned* err) {
    if (T == 0) return cudaSuccess;
    const int64_t units = T * ((H / 8 + kSpreadUnit - 1) / kSpreadUnit);
    return launch_chained(spread_rows_kernel<false>, dim3(unit_blocks(units, resident_blocks())), dim3(kThreads), 0, st,
                          static_cast<const void*>(src), static_cast<const uint8_t*>(nullptr), row_of, offsets, prob,
                          T, k, E, H, rows, prob_row, pad_offsets, pad_row, err);
}

cudaError_t launch_spread_rows8(const uint8_t* q, const uint8_t* scale, const int32_t* offsets, int64_t T, int k,
                                int E, int H, bf16* rows, const int32_t* pad_offsets, const int32_t* pad_row,
                                cudaStream_t st) {
    if (T == 0) return cudaSuccess;
    const int64_t units = T * ((H / 8 + kSpreadUnit - 1) / kSpreadUnit);
    return launch_chained(spread_rows_kernel<true>, dim3(unit_blocks(units, resident_blocks())), dim3(kThreads), 0, st,
                          static_cast<const void*>(q), scale, static_cast<const int32_t*>(nullptr), offsets,
                          static_cast<const float*>(nullptr), T, k, E, H, rows, static_cast<float*>(nullptr),
                          const_cast<int32_t*>(pad_offsets), const_cast<int32_t*>(pad_row),
                          static_cast<unsigned*>(nullptr));
}

}  // namespace moe
