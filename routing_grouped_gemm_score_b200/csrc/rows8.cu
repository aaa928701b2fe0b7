// rows8.cu -- rows in the 8-bit format of rows8.cuh: to it from bf16 and back,
// and the two steps by token of the 8-bit checkpoint's backward: each routed row's
// output gradient into expert blocks padded to whole K steps of 16 rows, and, once
// those rows hold dx, their sum by token and x in their place.
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
__device__ __forceinline__ void zero_pad_rows(const PadBlocks& b, int E, int chunks, int64_t bound, uint4* rows,
                                              float* prob_row) {
    const int lane = threadIdx.x & 31;
    const int64_t nwarps = ((int64_t)gridDim.x * kThreads) >> 5;
    for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; i < 16 * (int64_t)E; i += nwarps) {
        const int e = (int)(i >> 4);
        const int64_t r = (int64_t)b.pad[e] + max(b.off[e + 1] - b.off[e], 0) + (i & 15);
        if (r < 0 || r >= b.pad[e + 1] || r >= bound) continue;   // < 0: offsets whose sum passed 2^31
        for (int c = lane; c < chunks; c += 32) rows[r * chunks + c] = make_uint4(0, 0, 0, 0);
        if (prob_row != nullptr && lane == 0) prob_row[r] = 0.0f;
    }
}

// One token's row to the k padded rows of its assignments. Each token's row is
// read once. A warp owns a unit of one token's row (512 columns); lane j finds the
// row of assignment j: the expert of row_of[t, j] by bisection of the blocks' offsets,
// then its place in the padded block. The unit of a token's first columns writes
// pad_row, prob_row and row_from, and the first block pad_offsets. A row outside its
// range is recorded and skipped (pad_row -1). A row of a block that no assignment has
// keeps what the memory held: the down dgrad finds those rows, by a row_from whose
// pad_row is another, and clears them. 4096 tokens of 2048 columns, k = 8: 30 us
// (134 MB written), 8192 of 5120, k = 1: 32 us (84 MB read, 84 written).
__global__ void __launch_bounds__(kThreads)
    spread_rows_kernel(const uint4* __restrict__ src, const int32_t* __restrict__ row_of,
                       const int32_t* __restrict__ offsets, const float* __restrict__ prob, int64_t T, int k, int E,
                       int H, uint4* __restrict__ rows, float* __restrict__ prob_row,
                       int32_t* __restrict__ pad_offsets, int32_t* __restrict__ pad_row,
                       int32_t* __restrict__ row_from, unsigned* err) {
    __shared__ PadBlocks b;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int chunks = H / 8;
    const int per_row = (chunks + kSpreadUnit - 1) / kSpreadUnit;
    const int64_t A = T * k, bound = pad16_rows(A, E);
    const int64_t units = T * per_row, nwarps = ((int64_t)gridDim.x * kThreads) >> 5;
    pad_blocks(b, offsets, E, A);
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i <= E; i += kThreads) pad_offsets[i] = b.pad[i];
    for (int64_t u = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; u < units; u += nwarps) {
        int64_t t;
        int part;
        split_unit(u, per_row, t, part);
        int32_t mine = -1;
        if (lane < k) {
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
                if (mine >= 0) {
                    prob_row[mine] = __ldg(prob + t * k + lane);
                    row_from[mine] = (int32_t)(t * k + lane);
                }
            }
        }
        uint4 v[kSpreadChunks];
#pragma unroll
        for (int i = 0; i < kSpreadChunks; ++i) {
            const int c = part * kSpreadUnit + 32 * i + lane;
            if (c < chunks) v[i] = __ldg(src + t * chunks + c);
        }
        for (int j = 0; j < k; ++j) {
            const int64_t r = __shfl_sync(0xFFFFFFFFu, mine, j);
            if (r < 0) continue;
#pragma unroll
            for (int i = 0; i < kSpreadChunks; ++i) {
                const int c = part * kSpreadUnit + 32 * i + lane;
                if (c < chunks) rows[r * chunks + c] = v[i];
            }
        }
    }
    zero_pad_rows(b, E, chunks, bound, rows, prob_row);
}

// The last step by token (launch_finish_rows), one pass over its rows: they are
// read as dx, summed (j ascending, fp32), and written as x. A warp owns a unit of
// one token's row, so no other thread reads or writes what it does; the k loads
// of a column chunk are issued together. The unit of a token's first columns also
// sums its routing weights' gradients: the 32 / KB lanes of an assignment take
// every so many-th partial, a butterfly adds theirs, a fixed order.
// In one launch for k = 8 (4096 x 2048) 54 us, for k = 1 (8192 x 5120) 50; as three (the
// token sum, the weights' sums, x by row) 27 + 4 + 26 and 30 + 5 + 27.
template <int KB, int CH>
__global__ void __launch_bounds__(kThreads, KB > 8 ? 2 : 4)
    finish_rows_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ scale,
                       const int32_t* __restrict__ offsets, int64_t T, int k, int E, int H, uint4* rows,
                       const int32_t* __restrict__ pad_row, const float* __restrict__ row_dot, int nq,
                       uint4* __restrict__ dx, float* __restrict__ dprob) {
    constexpr unsigned kFull = 0xFFFFFFFFu;
    __shared__ PadBlocks b;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int chunks = H / 8, S = rows8_blocks(H);
    const int per_row = (chunks + (32 * CH) - 1) / (32 * CH);
    const int64_t A = T * k, bound = pad16_rows(A, E);
    const int64_t units = T * per_row, nwarps = ((int64_t)gridDim.x * kThreads) >> 5;
    pad_blocks(b, offsets, E, A);
    for (int64_t u = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; u < units; u += nwarps) {
        int64_t t;
        int part;
        split_unit(u, per_row, t, part);
        const int32_t mine = lane < k ? __ldg(pad_row + t * k + lane) : -1;   // -1: recorded by spread_rows_kernel
        int32_t r[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) r[j] = __shfl_sync(kFull, mine, j);   // -1 from k on
        // all loads of the unit before the first store: the rows are read and written
        uint4 v[CH][KB];
        uint2 xq[CH];
        uint32_t xb[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = part * (32 * CH) + 32 * i + lane;
            if (c >= chunks) continue;
#pragma unroll
            for (int j = 0; j < KB; ++j)
                if (r[j] >= 0) v[i][j] = rows[(int64_t)r[j] * chunks + c];
            xq[i] = __ldg(reinterpret_cast<const uint2*>(q + t * H) + c);
            xb[i] = __ldg(scale + t * S + (c >> 2));
        }
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = part * (32 * CH) + 32 * i + lane;
            if (c >= chunks) continue;
            float acc[8];
#pragma unroll
            for (int n = 0; n < 8; ++n) acc[n] = 0.0f;
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                if (r[j] < 0) continue;
                const uint32_t w[4] = {v[i][j].x, v[i][j].y, v[i][j].z, v[i][j].w};
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float2 f = unpack_bf16x2(w[n]);
                    acc[2 * n] += f.x;
                    acc[2 * n + 1] += f.y;
                }
            }
            dx[t * chunks + c] = make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                                            pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7]));
            const uint4 xv = rows8_dequantize8(xq[i], xb[i]);
#pragma unroll
            for (int j = 0; j < KB; ++j)
                if (r[j] >= 0) rows[(int64_t)r[j] * chunks + c] = xv;
        }
        if (part == 0) {
            constexpr int G = 32 / KB;   // lanes of an assignment
            const int j = lane / G;
            const int64_t row = __shfl_sync(kFull, mine, j);
            float sum = 0.0f;
            if (row >= 0) {
#pragma unroll 4
                for (int p = lane % G; p < nq; p += G) sum += __ldg(row_dot + row * nq + p);
            }
#pragma unroll
            for (int o = G / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
            if (lane % G == 0 && j < k) dprob[t * k + j] = sum;
        }
    }
    zero_pad_rows(b, E, chunks, bound, rows, nullptr);
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
                               int32_t* pad_row, int32_t* row_from, cudaStream_t st, unsigned* err) {
    if (T == 0) return cudaSuccess;
    const int64_t units = T * ((H / 8 + kSpreadUnit - 1) / kSpreadUnit);
    return launch_chained(spread_rows_kernel, dim3(unit_blocks(units, resident_blocks())), dim3(kThreads), 0, st,
                          reinterpret_cast<const uint4*>(src), row_of, offsets, prob, T, k, E, H,
                          reinterpret_cast<uint4*>(rows), prob_row, pad_offsets, pad_row, row_from, err);
}

cudaError_t launch_finish_rows(const Rows8& x8, const int32_t* offsets, int64_t T, int k, int E, int H, bf16* rows,
                               const int32_t* pad_row, const float* row_dot, int nq, bf16* dx, float* dprob,
                               cudaStream_t st) {
    if (T == 0) return cudaSuccess;
    const int unit = k <= 2 ? 64 : 32;   // chunks of a warp's unit
    const int64_t units = T * ((H / 8 + unit - 1) / unit);
    auto kern = k <= 2 ? finish_rows_kernel<2, 2>
              : k <= 4 ? finish_rows_kernel<4, 1> : k <= 8 ? finish_rows_kernel<8, 1> : finish_rows_kernel<16, 1>;
    return launch_chained(kern, dim3(unit_blocks(units, resident_blocks() / 2)), dim3(kThreads), 0, st,
                          static_cast<const uint8_t*>(x8.q), static_cast<const uint8_t*>(x8.scale), offsets, T, k, E,
                          H, reinterpret_cast<uint4*>(rows), pad_row, row_dot, nq, reinterpret_cast<uint4*>(dx), dprob);
}

}  // namespace moe
