// rows8.cu -- rows in the 8-bit format of rows8.cuh: to it from bf16 and back,
// and the two dispatches of the 8-bit checkpoint's backward, which write each
// routed row's output gradient and its x, read back from the token's 8-bit row.
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
constexpr int kChunks = 4;                   // 8-column chunks of a lane in one unit
constexpr int kUnitChunks = 32 * kChunks;    // chunks of a unit (blocks of four chunks, padded)

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

// One token's row to the k rows that its assignments hold: rows[row_of[t, j]] =
// the token's row, bf16 as it is (Q8 false) or read back from 8 bits (Q8 true).
// Each token's row is read once. A warp owns a unit of one token's row; its
// lanes hold the token's rows (lane j: row_of[t, j]). With prob given, the unit
// of a token's first columns also writes prob_row[row] = prob[t, j]. A row
// outside [0, A) is recorded and skipped.
template <bool Q8>
__global__ void __launch_bounds__(kThreads)
    spread_rows_kernel(const void* __restrict__ src, const uint8_t* __restrict__ scale,
                       const int32_t* __restrict__ row_of, const float* __restrict__ prob, int64_t T, int k, int H,
                       int64_t A, bf16* __restrict__ rows, float* __restrict__ prob_row, unsigned* err) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int chunks = H / 8, S = rows8_blocks(H);
    const int per_row = (chunks + kUnitChunks - 1) / kUnitChunks;
    const int64_t units = T * per_row, nwarps = ((int64_t)gridDim.x * kThreads) >> 5;
    for (int64_t u = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; u < units; u += nwarps) {
        int64_t t;
        int part;
        split_unit(u, per_row, t, part);
        int32_t mine = -1;
        if (lane < k) {
            mine = __ldg(row_of + t * k + lane);
            if (mine < 0 || mine >= A) {
                raise_error(err, kErrDeviceCheck);
                mine = -1;
            }
            if (prob_row != nullptr && part == 0 && mine >= 0) prob_row[mine] = __ldg(prob + t * k + lane);
        }
        uint4 v[kChunks];
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int c = part * kUnitChunks + 32 * i + lane;
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
            for (int i = 0; i < kChunks; ++i) {
                const int c = part * kUnitChunks + 32 * i + lane;
                if (c < chunks) dst[c] = v[i];
            }
        }
    }
}

// Blocks for a warp-per-unit kernel: enough warps for every unit, at most what
// stays resident (8 blocks of 256 threads an SM).
unsigned unit_blocks(int64_t units) {
    const int64_t cap = (int64_t)sm_count() * 8;
    const int64_t need = (units + kThreads / 32 - 1) / (kThreads / 32);
    return (unsigned)(need < cap ? need : cap);
}

int64_t format_units(int64_t rows, int cols, int parts) {
    return rows * ((4 * parts * rows8_blocks(cols) + kUnitChunks - 1) / kUnitChunks);
}

}  // namespace

cudaError_t launch_quantize_rows(const bf16* x, int64_t rows, int cols, int parts, int block_major, uint8_t* q,
                                 uint8_t* scale, cudaStream_t st) {
    if (rows == 0) return cudaSuccess;
    return launch_chained(quantize_rows_kernel, dim3(unit_blocks(format_units(rows, cols, parts))), dim3(kThreads), 0,
                          st, x, rows, cols, parts, block_major, q, scale);
}

cudaError_t launch_dequantize_rows(const uint8_t* q, const uint8_t* scale, int64_t rows, int cols, int parts,
                                   int block_major, bf16* x, cudaStream_t st) {
    if (rows == 0) return cudaSuccess;
    return launch_chained(dequantize_rows_kernel, dim3(unit_blocks(format_units(rows, cols, parts))), dim3(kThreads),
                          0, st, q, scale, rows, cols, parts, block_major, x);
}

cudaError_t launch_spread_rows(const bf16* src, const int32_t* row_of, const float* prob, int64_t T, int k, int H,
                               int64_t A, bf16* rows, float* prob_row, cudaStream_t st, unsigned* err) {
    if (T == 0) return cudaSuccess;
    const int64_t units = T * ((H / 8 + kUnitChunks - 1) / kUnitChunks);
    return launch_chained(spread_rows_kernel<false>, dim3(unit_blocks(units)), dim3(kThreads), 0, st,
                          static_cast<const void*>(src), static_cast<const uint8_t*>(nullptr), row_of, prob, T, k, H,
                          A, rows, prob_row, err);
}

cudaError_t launch_spread_rows8(const uint8_t* q, const uint8_t* scale, const int32_t* row_of, int64_t T, int k,
                                int H, int64_t A, bf16* rows, cudaStream_t st, unsigned* err) {
    if (T == 0) return cudaSuccess;
    const int64_t units = T * ((H / 8 + kUnitChunks - 1) / kUnitChunks);
    return launch_chained(spread_rows_kernel<true>, dim3(unit_blocks(units)), dim3(kThreads), 0, st,
                          static_cast<const void*>(q), scale, row_of, static_cast<const float*>(nullptr), T, k, H, A,
                          rows, static_cast<float*>(nullptr), err);
}

}  // namespace moe
