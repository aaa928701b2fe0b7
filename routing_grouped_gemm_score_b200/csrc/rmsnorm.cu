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
// Sums run in fp32 in a fixed order. Both are bound by HBM bandwidth: a row is
// read once, stays in registers (forward) or in shared memory (backward) until its
// sum is known, and is written once. Measured: 16384 rows of 5120 with a residual
// and both outputs 122 us (6.2 TB/s), their backward for 8192 rows 59 + 5 us for
// dweight (5.7 TB/s); one row of 2048 2.1-2.3 us.
#include "moe_internal.h"
#include "rows8.cuh"

namespace moe {

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kMaxWarps = 16;      // of a block that owns one row
constexpr float kSmallestMean = 0x1p-100f;   // of squares that are summed without scaling
constexpr size_t kBwdSmem = 200 * 1024;   // an SM's shared memory for the backward's rings
// Backward threads an SM: 1024 and 1536 measured alike at 5120 columns (59 us for
// 8192 rows), and at 2048 (4096 rows) 14.2 + 3.5 against 13.8 + 4.5 us, since more
// blocks leave more partial sums; 512 takes 17.4 and 98 us.
constexpr int kBwdThreads = 1024;
constexpr int kMaxStages = 8;      // row slots of a backward block's ring

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

// Threads for a row of that many chunks with ch of them each, whole warps.
__host__ __device__ constexpr int row_sums(int chunks, int ch) { return ((chunks + ch - 1) / ch + 31) / 32 * 32; }

// The rest of the order of a row's sum of squares (rmsnorm_kernel), from each thread's or
// the chunks' sums; the same in every thread.
template <int CH, int OC>
__device__ __forceinline__ float row_sum(float ss, const float* chunk_sum, float* red, int chunks) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, me = (int)threadIdx.x;
    const int sums = CH < OC ? row_sums(chunks, OC) : (int)blockDim.x;   // W
    if constexpr (CH < OC) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < OC; ++i)
            if (me < sums && me + i * sums < chunks) ss += chunk_sum[me + i * sums];
    }
    ss = warp_sum(ss);
    if (lane == 0) red[warp] = ss;
    __syncthreads();
    ss = 0.0f;
    for (int i = 0; i < (sums >> 5); ++i) ss += red[i];
    return ss;
}

// The rest of a row whose squares are past fp32's range, or so small that their roundings
// count (at a mean of 2^-100 a square is off by 2^-50 of it at most): summed again, scaled
// by up0 up1, the power of two that takes the larger of the row's magnitude and eps^1/2 to
// [1, 2). A row with an infinity, or of zeros with eps = 0, stays as it is. The pointers
// are the row's; its s (or x and residual) is read again, a chunk at a time, and a path of
// its own keeps the usual one as it is: as a detour before the outputs, from registers,
// it took 20 more of them, and the norm of 16384 rows of 5120 144 us (124 with the
// registers capped) instead of 122.
template <int CH, int OC>
__device__ __noinline__ void scaled_row(const uint4* s, const uint4* residual, const uint4* weight, int H, float eps,
                                        uint4* y, uint8_t* y_q, uint8_t* y_scale, float* rstd_out, float* chunk_sum,
                                        float* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int width = (int)blockDim.x, me = (int)threadIdx.x, chunks = H / 8;
    const auto s_chunk = [&](int c, float (&f)[8]) {   // zeros past the row
        const uint4 none = make_uint4(0, 0, 0, 0);
        unpack8(c < chunks ? s[c] : none, f);
        if (residual) {
            float r[8];
            unpack8(c < chunks ? residual[c] : none, r);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] += r[j];
            unpack8(pack8(f), f);
        }
    };
    float a = 0.0f, f[8];
#pragma unroll 1
    for (int i = 0; i < CH; ++i) {
        s_chunk(me + i * width, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(f[j]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(kFull, a, o));
    __syncthreads();   // every warp is done with red
    if (lane == 0) red[warp] = a;
    __syncthreads();
    for (int i = 0; i < (width >> 5); ++i) a = fmaxf(a, red[i]);
    a = fmaxf(a, sqrtf(eps));
    __syncthreads();
    float up0 = 1.0f, up1 = 1.0f;
    if (a > 0.0f && a < INFINITY) {
        const int k = -ilogbf(a);   // in [-127, 149]: in two factors that fp32 holds
        up0 = __uint_as_float((uint32_t)(127 + k / 2) << 23);
        up1 = __uint_as_float((uint32_t)(127 + k - k / 2) << 23);
    }
    float ss = 0.0f;
#pragma unroll 1
    for (int i = 0; i < CH; ++i) {
        s_chunk(me + i * width, f);
        float part = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            f[j] = f[j] * up0 * up1;
            part += f[j] * f[j];
        }
        if constexpr (CH < OC) chunk_sum[me + i * width] = part;
        else ss += part;
    }
    const float mean = row_sum<CH, OC>(ss, chunk_sum, red, chunks) / (float)H + eps * up0 * up1 * up0 * up1;
    const float rs = 1.0f / sqrtf(mean) * up1;   // rstd = rs up0
    if (rstd_out && me == 0) *rstd_out = rs * up0;
#pragma unroll 1
    for (int i = 0; i < CH; ++i) {
        const int c = me + i * width;
        s_chunk(c, f);
        if (c < chunks) {
            float w[8];
            unpack8(weight[c], w);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = f[j] * up0 * rs * w[j];
            if (y) y[c] = pack8(f);
        }
        if (y_q) {
            uint2 q;
            const uint32_t byte = rows8_quantize_quad(f, q);
            if (c < chunks) {
                *reinterpret_cast<uint2*>(y_q + 8 * c) = q;
                if ((c & 3) == 0) y_scale[c >> 2] = (uint8_t)byte;
            }
        }
    }
}

// Forward. One row per block, whose threads hold CH 8-column chunks each. The squares
// are added in one order for a given H, so that a row's results do not depend on T, by
// which CH is chosen: the eight of a chunk; W apart, the OC chunks of one of W sums; 32
// of those by a butterfly; then the warps'. OC and W are the CH and the threads of the
// kernel for many rows, which adds them in registers; the one for few rows (CH < OC)
// hands its chunks' sums over in shared memory. (32 chunks by a butterfly each, then
// these: one order as well, but 127 us instead of 122 for 16384 rows of 5120.) The
// pointers may alias as documented (sum with x or residual, y with x): a row's
// elements are read before they are written, by the same thread, so no pointer is
// marked restrict or read through the non-coherent path.
template <int CH, int OC>
__global__ void __launch_bounds__(32 * kMaxWarps)
    rmsnorm_kernel(const uint4* x, const uint4* residual, const uint4* weight, int H, float eps, uint4* sum, uint4* y,
                   uint8_t* y_q, uint8_t* y_scale, float* rstd_out) {
    static_assert(CH <= OC, "the order is the kernel's for many rows, whose threads hold more chunks");
    __shared__ float red[kMaxWarps];
    __shared__ float chunk_sum[CH < OC ? 32 * kMaxWarps * CH : 1];
    const int width = (int)blockDim.x, me = (int)threadIdx.x;
    const int64_t t = blockIdx.x;
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
        float part = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) part += v[i][j] * v[i][j];
        if constexpr (CH < OC) chunk_sum[me + i * width] = part;   // absent chunks: 0
        else ss += part;
    }
    const float mean = row_sum<CH, OC>(ss, chunk_sum, red, chunks) / (float)H + eps;
    if (mean < kSmallestMean || mean == INFINITY) {   // the same in every thread
        scaled_row<CH, OC>((sum ? sum : x) + t * chunks, residual && !sum ? residual + t * chunks : nullptr, weight, H,
                           eps, y ? y + t * chunks : nullptr, y_q ? y_q + t * H : nullptr,
                           y_q ? y_scale + t * rows8_blocks(H) : nullptr, rstd_out ? rstd_out + t : nullptr,
                           chunk_sum, red);
        return;
    }
    const float rstd = 1.0f / sqrtf(mean);
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

// Rows that a block of the backward reduces together: their sums share one
// barrier, which pays where a row is short.
template <int CH>
struct BwdRows {
    static constexpr int value = CH == 1 ? 2 : 1;
};

// Backward. A block owns groups of R whole rows (blockIdx.x, + gridDim.x, ...)
// and keeps its threads' columns of dweight in registers over all of them;
// partial [gridDim.x][H] gets them at the end. The rows of dy, s and dsum come as
// bulk asynchronous copies into a ring of `stages` slots in shared memory, one
// group each, so that loads are in flight while a group is reduced and written,
// whatever the block's registers hold. A group's slot is read twice, before and
// after the barrier of its reduction; the next group's barrier says that every
// thread is done with it, and it is filled again. dx may be dy or dsum itself: a
// row is written after its own copy has landed, by the block that alone reads it.
// Every wait is bounded; on a timeout the block records it and leaves.
template <int CH>
__global__ void __launch_bounds__(32 * kMaxWarps)
    rmsnorm_backward_kernel(const bf16* dy, const bf16* s, const uint4* __restrict__ weight,
                            const float* __restrict__ rstd, const bf16* dsum, int64_t T, int H, uint4* dx,
                            float* __restrict__ partial, int stages, unsigned* err) {
    constexpr int R = BwdRows<CH>::value;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ uint64_t full[kMaxStages];
    __shared__ float red[2][R][kMaxWarps];
    __shared__ int gave_up;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int width = blockDim.x, chunks = H / 8;
    const float inv_h = 1.0f / (float)H;
    const uint32_t row_bytes = 2u * (uint32_t)H, slot_bytes = (dsum ? 3u : 2u) * R * row_bytes;
    const int64_t groups = (T + R - 1) / R;
    int fills = 0;   // thread 0: slots filled so far; fill j used slot j % stages
    auto fill = [&](int64_t group, int slot) {
        ++fills;
        uint8_t* to = ring + slot * slot_bytes;
        const int64_t at = group * R * H;
        const uint32_t bytes = row_bytes * (uint32_t)min((int64_t)R, T - group * R);
        mbar_arrive_expect_tx(&full[slot], (dsum ? 3u : 2u) * bytes);
        bulk_load(&full[slot], to, dy + at, bytes);
        bulk_load(&full[slot], to + R * row_bytes, s + at, bytes);
        if (dsum) bulk_load(&full[slot], to + 2 * R * row_bytes, dsum + at, bytes);
    };
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
        gave_up = 0;
        fence_mbar_init();
        fence_proxy_async_smem();
        for (int64_t g = blockIdx.x; g < groups && fills < stages; g += gridDim.x) fill(g, fills);   // every slot
    }
    uint4 wv[CH];
    float dw[CH][8];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int c = threadIdx.x + i * width;
        wv[i] = c < chunks ? weight[c] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
    }
    float rs_next[R];
    auto load_rstd = [&](int64_t group) {
#pragma unroll
        for (int r = 0; r < R; ++r) rs_next[r] = group * R + r < T ? rstd[group * R + r] : 0.0f;
    };
    load_rstd(blockIdx.x);
    __syncthreads();   // the barriers are initialised
    int slot = 0, prev = 0, turn = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int64_t g = blockIdx.x; g < groups; g += gridDim.x) {
        float rs[R], dot[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            rs[r] = rs_next[r];
            dot[r] = 0.0f;
        }
        load_rstd(g + gridDim.x);
        ok = mbar_wait(&full[slot], phase, &gave_up, err);
        const int rows = (int)min((int64_t)R, T - g * R);
        const uint4* g_rows = reinterpret_cast<const uint4*>(ring + slot * slot_bytes);
        const uint4* s_rows = g_rows + R * chunks;
        if (ok) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (r >= rows) break;
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    const int c = threadIdx.x + i * width;
                    if (c >= chunks) continue;
                    float gf[8], vf[8], wf[8];
                    unpack8(g_rows[r * chunks + c], gf);
                    unpack8(s_rows[r * chunks + c], vf);
                    unpack8(wv[i], wf);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float xhat = vf[j] * rs[r];
                        dw[i][j] += gf[j] * xhat;
                        dot[r] += gf[j] * wf[j] * xhat;
                    }
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            dot[r] = warp_sum(dot[r]);
            if (lane == 0) red[turn][r][warp] = dot[r];   // read until the next barrier, written again after it
        }
        if (__syncthreads_or(!ok)) break;   // after a timeout every thread leaves
        if (threadIdx.x == 0 && g != blockIdx.x) {   // the group before is done with: its slot takes the next one to come
            const int64_t next = g + (int64_t)(stages - 1) * gridDim.x;
            if (next < groups) fill(next, prev);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r >= rows) break;
            float c0 = 0.0f;
            for (int w = 0; w < warps; ++w) c0 += red[turn][r][w];
            c0 *= inv_h;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const int c = threadIdx.x + i * width;
                if (c >= chunks) continue;
                float gf[8], vf[8], wf[8], o[8];
                unpack8(g_rows[r * chunks + c], gf);
                unpack8(s_rows[r * chunks + c], vf);
                unpack8(wv[i], wf);
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = rs[r] * (gf[j] * wf[j] - vf[j] * rs[r] * c0);
                if (dsum) {
                    float df[8];
                    unpack8(s_rows[(R + r) * chunks + c], df);
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] += df[j];
                }
                dx[(g * R + r) * chunks + c] = pack8(o);
            }
        }
        turn ^= 1;
        prev = slot;
        if (++slot == stages) {
            slot = 0;
            phase ^= 1u;
        }
    }
    if (!ok && threadIdx.x == 0) {   // copies still in flight land before the block's shared memory is given up
        for (int i = 0; i < stages; ++i)
            if (fills > i) mbar_wait_bounded(&full[i], (uint32_t)((fills - 1 - i) / stages) & 1u, err);
    }
    pdl_launch_dependents();   // rmsnorm_dweight_kernel may be scheduled; it waits for this kernel's end
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
    pdl_wait();
    __shared__ float red[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (col < H) {
#pragma unroll 8
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
int row_threads(int H, int ch) { return row_sums(H / 8, ch); }

int bwd_chunks(int H) { return H <= 4096 ? 1 : H <= 8192 ? 2 : 4; }

int bwd_rows(int H) { return bwd_chunks(H) == 1 ? BwdRows<1>::value : 1; }

// Blocks an SM and slots a block of the backward: about kBwdThreads threads an SM,
// as many slots as fit beside each other (at least two, so that a copy is always
// in flight).
struct BwdShape {
    int per_sm, stages;
    size_t smem;
};

BwdShape bwd_shape(int H, bool has_dsum) {
    const size_t slot = (has_dsum ? 3 : 2) * 2 * (size_t)H * bwd_rows(H);
    BwdShape b;
    b.per_sm = kBwdThreads / row_threads(H, bwd_chunks(H));
    if (b.per_sm > 8) b.per_sm = 8;
    if (b.per_sm < 1) b.per_sm = 1;
    while (b.per_sm > 1 && kBwdSmem / b.per_sm < 2 * slot) --b.per_sm;
    b.stages = (int)(kBwdSmem / b.per_sm / slot);
    if (b.stages > kMaxStages) b.stages = kMaxStages;
    b.smem = b.stages * slot;
    return b;
}

int64_t bwd_blocks(int64_t T, int H, int per_sm, int sms) {
    const int64_t cap = (int64_t)per_sm * sms, groups = (T + bwd_rows(H) - 1) / bwd_rows(H);
    return groups < cap ? groups : cap;
}

constexpr int kMaxSms = 256;   // bounds the workspace whatever the GPU

template <int CH>
cudaError_t launch_bwd(const bf16* dy, const bf16* s, const bf16* weight, const float* rstd, const bf16* dsum, int64_t T,
                       int H, bf16* dx, float* partial, int64_t blocks, const BwdShape& b, cudaStream_t st,
                       unsigned* err) {
    auto kern = rmsnorm_backward_kernel<CH>;
    static PerDeviceFlag configured;
    if (const cudaError_t e = allow_smem(kern, kBwdSmem, configured); e != cudaSuccess) return e;
    kern<<<(unsigned)blocks, row_threads(H, CH), b.smem, st>>>(dy, s, reinterpret_cast<const uint4*>(weight), rstd, dsum,
                                                               T, H, reinterpret_cast<uint4*>(dx), partial, b.stages, err);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rmsnorm(const bf16* x, const bf16* residual, const bf16* weight, int64_t T, int H, float eps,
                           bf16* sum, bf16* y, uint8_t* y_q, uint8_t* y_scale, float* rstd, cudaStream_t st) {
    if (T == 0) return cudaSuccess;
    const int chunks = H / 8;
    auto go = [&](auto kern, dim3 grid, int threads) {
        kern<<<grid, threads, 0, st>>>(reinterpret_cast<const uint4*>(x), reinterpret_cast<const uint4*>(residual),
                                       reinterpret_cast<const uint4*>(weight), H, eps,
                                       reinterpret_cast<uint4*>(sum), reinterpret_cast<uint4*>(y), y_q, y_scale, rstd);
    };
    const dim3 rows((unsigned)T);
    // More columns a thread keep more loads in flight an SM: 16384 rows of 5120 take
    // 133, 127 and 122 us with 1, 2 and 4 chunks a thread, 4096 rows of 2048 14.3,
    // 13.4 and 13.3. With fewer rows than SMs only the latency of one row counts
    // (2.2, 2.4 and 3.2 us): as many threads as a block may have.
    const bool few = T < sm_count();
    if (chunks <= 128) go(rmsnorm_kernel<1, 1>, rows, row_threads(H, 1));
    else if (chunks <= 512 && few) go(rmsnorm_kernel<1, 2>, rows, row_threads(H, 1));
    else if (chunks <= 512) go(rmsnorm_kernel<2, 2>, rows, row_threads(H, 2));
    else if (chunks <= 1024 && few) go(rmsnorm_kernel<2, 4>, rows, row_threads(H, 2));
    else go(rmsnorm_kernel<4, 4>, rows, row_threads(H, 4));
    return cudaGetLastError();
}

size_t rmsnorm_backward_workspace_bytes(int64_t T, int H) {
    const int a = bwd_shape(H, true).per_sm, b = bwd_shape(H, false).per_sm;
    return (size_t)bwd_blocks(T, H, a > b ? a : b, kMaxSms) * (size_t)H * sizeof(float);
}

cudaError_t launch_rmsnorm_backward(const bf16* dy, const bf16* s, const bf16* weight, const float* rstd,
                                    const bf16* dsum, int64_t T, int H, bf16* dx, float* dweight, float* partial,
                                    cudaStream_t st, unsigned* err) {
    if (T == 0) return dweight ? cudaMemsetAsync(dweight, 0, sizeof(float) * (size_t)H, st) : cudaSuccess;
    const BwdShape b = bwd_shape(H, dsum != nullptr);
    const int64_t blocks = bwd_blocks(T, H, b.per_sm, sm_count() < kMaxSms ? sm_count() : kMaxSms);
    if (!dweight) partial = nullptr;
    const int ch = bwd_chunks(H);
    cudaError_t e = ch == 1   ? launch_bwd<1>(dy, s, weight, rstd, dsum, T, H, dx, partial, blocks, b, st, err)
                    : ch == 2 ? launch_bwd<2>(dy, s, weight, rstd, dsum, T, H, dx, partial, blocks, b, st, err)
                              : launch_bwd<4>(dy, s, weight, rstd, dsum, T, H, dx, partial, blocks, b, st, err);
    if (e == cudaSuccess && dweight) {
        const ChainScope chain(true);   // its launch and prologue overlap the last blocks' rows
        e = launch_chained(rmsnorm_dweight_kernel, dim3((unsigned)((H + 31) / 32)), dim3(1024), 0, st,
                           static_cast<const float*>(partial), (int)blocks, H, dweight);
    }
    return e;
}

}  // namespace moe
