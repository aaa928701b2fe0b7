// rmsnorm.cu -- RMSNorm in front of the MoE layer, with the residual's
// addition and an 8-bit output (rows8.cuh), and its backward.
//
// Forward, per row of H columns:
//   s = bf16(x + r)  (s = x without a residual; the stored sum is what is normalised, so
//                     the backward, which reads it, differentiates what was computed)
//   rstd = (sum_i s_i^2 / H + eps)^(-1/2)
//   y_i = (s_i rstd) w_i, stored in bf16 and, from the same fp32 value, in 8 bits
// Backward, with xhat = s rstd:
//   dx_i = rstd (w_i dy_i - xhat_i c) (+ dsum_i),  c = sum_j w_j dy_j xhat_j / H
//   dw_i = sum_t dy_{t,i} xhat_{t,i}
// Sums run in fp32 in a fixed order. Both are bound by HBM bandwidth: the row
// stays in registers between its one read and its one write.
#include "moe_internal.h"
#include "rows8.cuh"

namespace moe {

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kMaxWarps = 16;      // of a block that owns one row
constexpr int kWarpRows = 4;       // rows of a block whose warps own one row each

__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack_bf16x2(u[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// One row per block (WARP false; blockDim.x threads hold CH 8-column chunks
// each) or per warp (WARP true). The pointers may alias as documented (sum with
// x or residual): a row's elements are read before they are written, by the
// same thread, so no pointer is marked restrict or read through the
// non-coherent path.
template <int CH, bool WARP>
__global__ void __launch_bounds__(32 * kMaxWarps)
    rmsnorm_kernel(const uint4* x, const uint4* residual, const uint4* weight, int64_t T, int H, float eps,
                               uint4* sum, uint4* y, uint8_t* y_q, uint8_t* y_scale, float* rstd_out) {
    __shared__ float red[kMaxWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int width = WARP ? 32 : (int)blockDim.x;
    const int me = WARP ? lane : (int)threadIdx.x;
    const int64_t t = WARP ? (int64_t)blockIdx.x * kWarpRows + warp : (int64_t)blockIdx.x;
    if (t >= T) return;   // WARP: whole warps
    const int chunks = H / 8;
    uint4 xv[CH], rv[CH], wv[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = me + i * width;
        xv[i] = rv[i] = wv[i] = make_uint4(0, 0, 0, 0);
        if (c >= chunks) continue;
        xv[i] = x[t * chunks + c];
        if (residual) rv[i] = residual[t * chunks + c];
        wv[i] = weight[c];
    }
    float v[CH][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        unpack8(xv[i], v[i]);
        if (residual) {
            float r[8];
            unpack8(rv[i], r);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] += r[j];
            const uint4 s = pack8(v[i]);
            const int c = me + i * width;
            if (sum && c < chunks) sum[t * chunks + c] = s;
            unpack8(s, v[i]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += v[i][j] * v[i][j];
    }
    ss = warp_sum(ss);
    if (!WARP) {
        if (lane == 0) red[warp] = ss;
        __syncthreads();
        ss = 0.0f;
        for (int i = 0; i < (int)(blockDim.x >> 5); ++i) ss += red[i];
    }
    const float rstd = 1.0f / sqrtf(ss / (float)H + eps);
    if (rstd_out && me == 0) rstd_out[t] = rstd;
    const int S = rows8_blocks(H);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = me + i * width;
        float w[8];
        unpack8(wv[i], w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * w[j];
        if (y && c < chunks) y[t * chunks + c] = pack8(v[i]);
        if (y_q) {
            if (c >= chunks) {   // absent columns do not count towards a block's scale (0 * rstd may be NaN)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
            }
            uint2 q;
            const uint32_t byte = rows8_quantize_quad(v[i], q);
            if (c < chunks) {
                *reinterpret_cast<uint2*>(y_q + t * H + 8 * c) = q;
                if ((c & 3) == 0) y_scale[t * S + (c >> 2)] = (uint8_t)byte;
            }
        }
    }
}

template <int CH>
struct BwdRows {
    static constexpr int value = CH == 1 ? 4 : CH == 2 ? 2 : 1;   // rows of one block step
};

// A block owns whole rows, R of them a step (one barrier for R sums), and keeps
// its threads' columns of dweight in registers over all of its rows; partial
// [gridDim.x][H] gets them at the end. dx may be dy or dsum itself.
template <int CH>
__global__ void __launch_bounds__(32 * kMaxWarps)
    rmsnorm_backward_kernel(const uint4* dy, const uint4* s, const uint4* __restrict__ weight,
                                        const float* __restrict__ rstd, const uint4* dsum, int64_t T, int H,
                                        uint4* dx, float* __restrict__ partial) {
    constexpr int R = BwdRows<CH>::value;
    __shared__ float red[2][R][kMaxWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int width = blockDim.x, chunks = H / 8;
    const float inv_h = 1.0f / (float)H;
    uint4 wv[CH];
    float dw[CH][8];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = threadIdx.x + i * width;
        wv[i] = c < chunks ? weight[c] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
    }
    int turn = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * R; t0 < T; t0 += (int64_t)gridDim.x * R, turn ^= 1) {
        uint4 g[R][CH], v[R][CH], d[R][CH];
        float rs[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t t = t0 + r;
            rs[r] = t < T ? rstd[t] : 0.0f;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int c = threadIdx.x + i * width;
                g[r][i] = v[r][i] = d[r][i] = make_uint4(0, 0, 0, 0);
                if (t >= T || c >= chunks) continue;
                g[r][i] = dy[t * chunks + c];
                v[r][i] = s[t * chunks + c];
                if (dsum) d[r][i] = dsum[t * chunks + c];
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                float gf[8], vf[8], wf[8];
                unpack8(g[r][i], gf);
                unpack8(v[r][i], vf);
                unpack8(wv[i], wf);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float xhat = vf[j] * rs[r];
                    dw[i][j] += gf[j] * xhat;
                    dot += gf[j] * wf[j] * xhat;
                }
            }
            dot = warp_sum(dot);
            if (lane == 0) red[turn][r][warp] = dot;
        }
        __syncthreads();   // red[turn] is written again two steps on, after the next step's barrier
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t t = t0 + r;
            float c0 = 0.0f;
            for (int w = 0; w < warps; ++w) c0 += red[turn][r][w];
            c0 *= inv_h;
            if (t >= T) continue;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int c = threadIdx.x + i * width;
                if (c >= chunks) continue;
                float gf[8], vf[8], wf[8], df[8], o[8];
                unpack8(g[r][i], gf);
                unpack8(v[r][i], vf);
                unpack8(wv[i], wf);
                unpack8(d[r][i], df);
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = rs[r] * (gf[j] * wf[j] - vf[j] * rs[r] * c0) + df[j];
                dx[t * chunks + c] = pack8(o);
            }
        }
    }
    if (partial) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int c = threadIdx.x + i * width;
            if (c >= chunks) continue;
            float4* out = reinterpret_cast<float4*>(partial + (int64_t)blockIdx.x * H + 8 * c);
            out[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
            out[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
        }
    }
}

// dweight[i] = sum_b partial[b][i]: a block owns 32 columns, its 32 warps every
// 32nd partial row each, then the warps' sums in warp order.
__global__ void __launch_bounds__(1024)
    rmsnorm_dweight_kernel(const float* __restrict__ partial, int blocks, int H, float* __restrict__ dweight) {
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (col < H) {
#pragma unroll 4
        for (int b = warp; b < blocks; b += 32) v += partial[(int64_t)b * H + col];
    }
    red[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && col < H) {
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < 32; ++w) v += red[w][lane];
        dweight[col] = v;
    }
}

// Threads of a block that owns a row with CH chunks a thread.
int row_threads(int H, int ch) {
    const int need = (H / 8 + ch - 1) / ch;
    return (need + 31) / 32 * 32;
}

int bwd_chunks(int H) { return H <= 4096 ? 1 : H <= 8192 ? 2 : 4; }

int64_t bwd_blocks(int64_t T, int H, int sms) {
    const int ch = bwd_chunks(H);
    const int rows = ch == 1 ? 4 : ch == 2 ? 2 : 1;
    const int64_t need = (T + rows - 1) / rows;
    const int64_t cap = 2 * (int64_t)sms;
    return need < cap ? need : cap;
}

constexpr int kMaxSms = 256;   // bounds the workspace whatever the GPU

}  // namespace

cudaError_t launch_rmsnorm(const bf16* x, const bf16* residual, const bf16* weight, int64_t T, int H, float eps,
                           bf16* sum, bf16* y, uint8_t* y_q, uint8_t* y_scale, float* rstd, cudaStream_t st) {
    if (T == 0) return cudaSuccess;
    const int chunks = H / 8;
    auto go = [&](auto kern, dim3 grid, int threads) {
        kern<<<grid, threads, 0, st>>>(reinterpret_cast<const uint4*>(x), reinterpret_cast<const uint4*>(residual),
                                       reinterpret_cast<const uint4*>(weight), T, H, eps,
                                       reinterpret_cast<uint4*>(sum), reinterpret_cast<uint4*>(y), y_q, y_scale, rstd);
    };
    const dim3 rows((unsigned)T);
    if (chunks <= 512) go(rmsnorm_kernel<1, false>, rows, row_threads(H, 1));
    else if (chunks <= 1024) go(rmsnorm_kernel<2, false>, rows, row_threads(H, 2));
    else go(rmsnorm_kernel<4, false>, rows, row_threads(H, 4));
    return cudaGetLastError();
}

size_t rmsnorm_backward_workspace_bytes(int64_t T, int H) {
    return (size_t)bwd_blocks(T, H, kMaxSms) * (size_t)H * sizeof(float);
}

cudaError_t launch_rmsnorm_backward(const bf16* dy, const bf16* s, const bf16* weight, const float* rstd,
                                    const bf16* dsum, int64_t T, int H, bf16* dx, float* dweight, float* partial,
                                    cudaStream_t st) {
    if (T == 0) return dweight ? cudaMemsetAsync(dweight, 0, sizeof(float) * (size_t)H, st) : cudaSuccess;
    const int sms = sm_count() < kMaxSms ? sm_count() : kMaxSms;
    const int64_t blocks = bwd_blocks(T, H, sms);
    const int ch = bwd_chunks(H);
    auto go = [&](auto kern) {
        kern<<<(unsigned)blocks, row_threads(H, ch), 0, st>>>(
            reinterpret_cast<const uint4*>(dy), reinterpret_cast<const uint4*>(s),
            reinterpret_cast<const uint4*>(weight), rstd, reinterpret_cast<const uint4*>(dsum), T, H,
            reinterpret_cast<uint4*>(dx), dweight ? partial : nullptr);
    };
    if (ch == 1) go(rmsnorm_backward_kernel<1>);
    else if (ch == 2) go(rmsnorm_backward_kernel<2>);
    else go(rmsnorm_backward_kernel<4>);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && dweight) {
        rmsnorm_dweight_kernel<<<(unsigned)((H + 31) / 32), 1024, 0, st>>>(partial, (int)blocks, H, dweight);
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace moe
