// Root-mean-square norm with the residual's addition, S = X + R (rounded to bf16, the
// residual stream as it is kept), y = S rstd g with rstd = 1 / sqrt(mean(S^2) + eps), as
// bf16 or as int8 with a scale a row; and its gradients: with a = dY g and n = S rstd,
// dX = dS + rstd (a - n mean(a n)) and dg = sum over rows of dY n.
//
// y is made of S as it is stored, not of the unrounded sum, so that the backward pass,
// which reads S, differentiates what was computed.  rstd is not kept: a row of S is read
// whole either way, and its sum of squares costs nothing beside that.
//
// A block takes a row at a time and keeps it in registers between the sum and the
// outputs, so every operand is read once.  All operands have the same pitch and
// 16-byte-aligned bases, so a row starts at the same place of a 16-byte vector in each:
// a thread takes whole aligned vectors (eight elements of the flat matrix), masked at
// the row's two ends, whatever the width.
#include <cuda_runtime.h>

#include "op_gemm.cuh"
#include "op_host.h"

namespace pg {

constexpr int kNormMaxD = 32768;

// One row as a block of threads holds it: vector v covers the elements 8 v - shift ..
// 8 v - shift + 7 of the row.
struct RowSpan {
    long long first;  // flat index of vector 0's first element (a multiple of 8)
    int shift, vecs, D;
    __device__ __forceinline__ RowSpan(long long row, int D_) : D(D_) {
        const long long at = row * D_;
        shift = static_cast<int>(at & 7);
        first = at - shift;
        vecs = (D_ + shift + 7) >> 3;
    }
    __device__ __forceinline__ int col(int v) const { return 8 * v - shift; }
    __device__ __forceinline__ bool whole(int v) const {
        return col(v) >= 0 && col(v) + 8 <= D;
    }
};

__device__ __forceinline__ void unpack8(const uint4 &x, float (&f)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                      pack_bf16(f[6], f[7]));
}

// Vector v of a row, zeros where the row is not.
__device__ __forceinline__ uint4 row_load(const uint16_t *p, const RowSpan &r, int v) {
    const uint16_t *at = p + r.first + 8ll * v;
    if (r.whole(v)) return *reinterpret_cast<const uint4 *>(at);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = r.col(v) + i;
        if (c >= 0 && c < r.D) w[i / 2] |= static_cast<uint32_t>(at[i]) << (i % 2 * 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void row_store(uint16_t *p, const RowSpan &r, int v, const uint4 &x) {
    uint16_t *at = p + r.first + 8ll * v;
    if (r.whole(v)) {
        *reinterpret_cast<uint4 *>(at) = x;
        return;
    }
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = r.col(v) + i;
        if (c >= 0 && c < r.D) at[i] = static_cast<uint16_t>(w[i / 2] >> (i % 2 * 16));
    }
}

// The gains of vector v's columns (ones without gains; anything where the row is not).
__device__ __forceinline__ void gain_load(const uint16_t *g, const RowSpan &r, int v,
                                          float (&f)[8]) {
    if (g == nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 1.0f;
    } else if (r.shift == 0 && r.whole(v)) {
        unpack8(__ldg(reinterpret_cast<const uint4 *>(g) + v), f);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = r.col(v) + i;
            f[i] = c >= 0 && c < r.D
                       ? __uint_as_float(static_cast<uint32_t>(__ldg(g + c)) << 16)
                       : 0.0f;
        }
    }
}

struct Add {
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct Larger {  // a NaN stays one
    __device__ __forceinline__ float operator()(float a, float b) const {
        return a > b || a != a ? a : b;
    }
};

// op over the block's threads, in an order that does not depend on timing; the same in
// every thread.  `part` (32 floats) may be used again after the block's next barrier.
template <int THREADS, class Op>
__device__ __forceinline__ float block_reduce(float x, float *part, Op op) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x = op(x, __shfl_xor_sync(0xffffffffu, x, d));
    if constexpr (THREADS > 32) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
        __syncthreads();
        constexpr int W = THREADS / 32;
        x = part[(threadIdx.x & 31) % W];
#pragma unroll
        for (int d = W / 2; d > 0; d >>= 1) x = op(x, __shfl_xor_sync(0xffffffffu, x, d));
    }
    return x;
}

struct NormParams {
    int T, D;
    float eps;
    const uint16_t *x, *r, *gain;
    uint16_t *s, *y;
    int8_t *q;
    float *scale;
    // backward
    const uint16_t *dy, *ds;
    uint16_t *dx;
    float *dgain;  // [blocks][D] partial sums, or nullptr
};

template <int THREADS, int V, bool I8>
__global__ void __launch_bounds__(THREADS) rmsnorm_kernel(const NormParams p) {
    __shared__ float part[2][32];
    grid_dependency_wait();
    grid_launch_dependents();
    int turn = 0;
    for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
        const RowSpan row(t, p.D);
        float f[V][8];
        float sum = 0.0f;
        uint4 a[V], b[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = threadIdx.x + i * THREADS;
            a[i] = b[i] = make_uint4(0u, 0u, 0u, 0u);
            if (v < row.vecs) {
                a[i] = row_load(p.x, row, v);
                if (p.r) b[i] = row_load(p.r, row, v);
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = threadIdx.x + i * THREADS;
            if (p.r) {
                float fa[8], fb[8];
                unpack8(a[i], fa);
                unpack8(b[i], fb);
#pragma unroll
                for (int j = 0; j < 8; ++j) fa[j] += fb[j];
                a[i] = pack8(fa);  // S as it is stored
            }
            if (p.s && v < row.vecs) row_store(p.s, row, v, a[i]);
            unpack8(a[i], f[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(f[i][j], f[i][j], sum);
        }
        sum = block_reduce<THREADS>(sum, part[turn], Add{});
        turn ^= 1;
        const float rstd = 1.0f / sqrtf(sum / static_cast<float>(p.D) + p.eps);
        float most = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = threadIdx.x + i * THREADS;
            if (v >= row.vecs) break;
            float g[8];
            gain_load(p.gain, row, v, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                f[i][j] = f[i][j] * rstd * g[j];
                if (I8) {
                    const int c = row.col(v) + j;
                    if (c >= 0 && c < p.D) most = Larger{}(fabsf(f[i][j]), most);
                }
            }
            if constexpr (!I8) row_store(p.y, row, v, pack8(f[i]));
        }
        if constexpr (I8) {
            most = block_reduce<THREADS>(most, part[turn], Larger{});
            turn ^= 1;
            const bool fine = most < __int_as_float(0x7f800000);
            if (threadIdx.x == 0)
                p.scale[t] = fine ? most / 127.0f : __int_as_float(0x7fc00000);
            // far below 1 everything is scaled up first, so that the reciprocal is finite
            const float up = most < 8.6736174e-19f ? 1.1529215e18f : 1.0f;  // 2^-60, 2^60
            const float inv = fine && most > 0.0f ? 127.0f / (most * up) : 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int v = threadIdx.x + i * THREADS;
                if (v >= row.vecs) break;
                uint32_t w[2] = {0u, 0u};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int q = fine ? __float2int_rn(f[i][j] * up * inv) : 0;
                    w[j / 4] |= (static_cast<uint32_t>(q) & 0xffu) << (j % 4 * 8);
                }
                int8_t *at = p.q + row.first + 8ll * v;
                if (row.whole(v)) {
                    *reinterpret_cast<uint2 *>(at) = make_uint2(w[0], w[1]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int c = row.col(v) + j;
                        if (c >= 0 && c < p.D)
                            at[j] = static_cast<int8_t>(w[j / 4] >> (j % 4 * 8));
                    }
                }
            }
        }
    }
}

// The gains' gradient: each block adds its rows' dY n in shared memory, column c at
// (c % 8) * pitch + c / 8, so that a warp's eight elements a lane fall on different
// banks, and leaves the sums for norm_join_kernel.
template <int THREADS, int V>
__global__ void __launch_bounds__(THREADS) rmsnorm_backward_kernel(const NormParams p) {
    extern __shared__ float sums[];
    __shared__ float part[2][2][32];
    const int pitch = (p.D + 7) / 8;
    if (p.dgain)
        for (int i = threadIdx.x; i < 8 * pitch; i += THREADS) sums[i] = 0.0f;
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();
    int turn = 0;
    for (int t = blockIdx.x; t < p.T; t += gridDim.x) {
        const RowSpan row(t, p.D);
        uint4 s[V], dy[V], ds[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = threadIdx.x + i * THREADS;
            s[i] = dy[i] = ds[i] = make_uint4(0u, 0u, 0u, 0u);
            if (v < row.vecs) {
                s[i] = row_load(p.x, row, v);
                dy[i] = row_load(p.dy, row, v);
                if (p.ds) ds[i] = row_load(p.ds, row, v);
            }
        }
        float sum = 0.0f, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = threadIdx.x + i * THREADS;
            if (v >= row.vecs) break;
            float fs[8], fd[8], g[8];
            unpack8(s[i], fs);
            unpack8(dy[i], fd);
            gain_load(p.gain, row, v, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sum = fmaf(fs[j], fs[j], sum);
                dot = fmaf(fd[j] * g[j], fs[j], dot);
            }
        }
        sum = block_reduce<THREADS>(sum, part[turn][0], Add{});
        dot = block_reduce<THREADS>(dot, part[turn][1], Add{});
        turn ^= 1;
        const float rstd = 1.0f / sqrtf(sum / static_cast<float>(p.D) + p.eps);
        const float m = dot * rstd / static_cast<float>(p.D);  // mean(a n)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = threadIdx.x + i * THREADS;
            if (v >= row.vecs) break;
            float fs[8], fd[8], g[8], o[8];
            unpack8(s[i], fs);
            unpack8(dy[i], fd);
            gain_load(p.gain, row, v, g);
            unpack8(ds[i], o);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float n = fs[j] * rstd;
                o[j] += rstd * fmaf(-n, m, fd[j] * g[j]);
                const int c = row.col(v) + j;
                if (p.dgain && c >= 0 && c < p.D) {
                    float *at = sums + (c & 7) * pitch + (c >> 3);
                    *at = fmaf(fd[j], n, *at);
                }
            }
            if (p.dx) row_store(p.dx, row, v, pack8(o));
        }
        // (with rows that start anywhere in a vector, the next row's columns are other
        // threads': its two block_reduce barriers stand between)
        if (THREADS == 32) __syncwarp();
    }
    if (p.dgain) {
        __syncthreads();
        float *out = p.dgain + static_cast<long long>(blockIdx.x) * p.D;
        for (int c = threadIdx.x; c < p.D; c += THREADS) out[c] = sums[(c & 7) * pitch + (c >> 3)];
    }
}

// dgain = sum of the blocks' sums, in order: eight warps take every eighth block's, 32
// columns a block.
__global__ void __launch_bounds__(256)
    norm_join_kernel(const float *part, int blocks, int D, uint16_t *out) {
    grid_dependency_wait();
    grid_launch_dependents();
    __shared__ float s[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float t = 0.0f;
    if (c < D) {
#pragma unroll 8
        for (int b = w; b < blocks; b += 8) t += part[static_cast<long long>(b) * D + c];
    }
    s[w][lane] = t;
    __syncthreads();
    if (w == 0 && c < D) {
#pragma unroll
        for (int i = 1; i < 8; ++i) t += s[i][lane];
        out[c] = static_cast<uint16_t>(pack_bf16(t, 0.0f) & 0xffffu);
    }
}

// f(threads, vectors a thread) as integral constants for rows of D: two vectors a thread
// where rows are many, one where the row's own latency counts.
template <class F>
static pgemm_status with_row(int D, bool few, F &&f) {
    const int vecs = D % 8 == 0 ? D / 8 : (D + 14) / 8;
    using std::integral_constant;
    auto pick = [&](auto threads) {
        constexpr int N = decltype(threads)::value;
        return vecs <= N ? f(threads, integral_constant<int, 1>{})
                         : f(threads, integral_constant<int, 2>{});
    };
    const int per = few ? 1 : 2;
    if (vecs <= 32 * per) return pick(integral_constant<int, 32>{});
    if (vecs <= 64 * per) return pick(integral_constant<int, 64>{});
    if (vecs <= 128 * per) return pick(integral_constant<int, 128>{});
    if (vecs <= 256 * per) return pick(integral_constant<int, 256>{});
    if (vecs <= 512 * per) return pick(integral_constant<int, 512>{});
    if (vecs <= 2048) return pick(integral_constant<int, 1024>{});
    return f(integral_constant<int, 1024>{}, integral_constant<int, 5>{});
}

static pgemm_status norm_check(int T, int D) {
    if (T < 0 || D < 0) return PGEMM_ERR_INVALID_VALUE;
    return D > kNormMaxD ? PGEMM_ERR_TOO_LARGE : PGEMM_OK;
}

static pgemm_status norm_forward(bool i8, int T, int D, const uint16_t *X, const uint16_t *R,
                                 const uint16_t *gain, float eps, uint16_t *S, void *out,
                                 float *scale, cudaStream_t s) {
    pgemm_status st = norm_check(T, D);
    if (st != PGEMM_OK) return st;
    if (!(eps >= 0.0f)) return PGEMM_ERR_INVALID_VALUE;
    if (T == 0 || D == 0) return PGEMM_OK;
    if (!X || !out || (i8 && !scale)) return PGEMM_ERR_INVALID_VALUE;
    if (!op_aligned16(X) || !op_aligned16(R) || !op_aligned16(gain) || !op_aligned16(S) ||
        !op_aligned16(out) || !op_aligned16(scale))
        return PGEMM_ERR_MISALIGNED;
    OpDevice dev;
    if ((st = op_device(&dev)) != PGEMM_OK) return st;
    NormParams p{};
    p.T = T;
    p.D = D;
    p.eps = eps;
    p.x = X;
    p.r = R;
    p.gain = gain;
    p.s = S;
    p.y = i8 ? nullptr : static_cast<uint16_t *>(out);
    p.q = i8 ? static_cast<int8_t *>(out) : nullptr;
    p.scale = scale;
    return with_row(D, T < 2 * dev.sm_count, [&](auto threads, auto v) {
        constexpr int N = decltype(threads)::value, V = decltype(v)::value;
        const long long most = dev.sm_count * (N >= 2048 / 32 ? 2048ll / N : 32ll);
        const dim3 grid(static_cast<unsigned>(T < most ? T : most));
        return i8 ? launch_small(rmsnorm_kernel<N, V, true>, grid, dim3(N), s, p)
                  : launch_small(rmsnorm_kernel<N, V, false>, grid, dim3(N), s, p);
    });
}

static pgemm_status norm_backward(int T, int D, const uint16_t *S, const uint16_t *gain, float eps,
                                  const uint16_t *dY, const uint16_t *dS, uint16_t *dX,
                                  uint16_t *dgain, cudaStream_t s) {
    pgemm_status st = norm_check(T, D);
    if (st != PGEMM_OK) return st;
    if (!(eps >= 0.0f)) return PGEMM_ERR_INVALID_VALUE;
    if (D == 0 || (!dgain && (T == 0 || !dX))) return PGEMM_OK;
    if (T > 0 && (!S || !dY)) return PGEMM_ERR_INVALID_VALUE;
    if (!op_aligned16(S) || !op_aligned16(gain) || !op_aligned16(dY) || !op_aligned16(dS) ||
        !op_aligned16(dX) || !op_aligned16(dgain))
        return PGEMM_ERR_MISALIGNED;
    OpDevice dev;
    if ((st = op_device(&dev)) != PGEMM_OK) return st;
    if (T == 0)
        return cudaMemsetAsync(dgain, 0, static_cast<size_t>(D) * 2, s) == cudaSuccess
                   ? PGEMM_OK
                   : PGEMM_ERR_CUDA;
    NormParams p{};
    p.T = T;
    p.D = D;
    p.eps = eps;
    p.x = S;
    p.gain = gain;
    p.dy = dY;
    p.ds = dS;
    p.dx = dX;
    return with_row(D, true, [&](auto threads, auto v) -> pgemm_status {
        constexpr int N = decltype(threads)::value, V = decltype(v)::value;
        // blocks of an SM: what threads and shared memory allow, eight at most, since
        // each leaves a row of sums behind
        const int smem = dgain ? (D + 7) / 8 * 32 : 0;
        int per_sm = 2048 / N < 8 ? 2048 / N : 8;
        while (per_sm > 1 && per_sm * (smem + 2048) > kSmemPerSm) --per_sm;
        const int most = dev.sm_count * per_sm;
        const int blocks = T < most ? T : most;
        static const KernelInfo info = [] {
            KernelInfo k;
            k.threads = N;
            k.smem_bytes = kNormMaxD * 4;
            k.func = reinterpret_cast<const void *>(rmsnorm_backward_kernel<N, V>);
            return k;
        }();
        pgemm_status e = op_kernel_setup(dev, info, nullptr);
        if (e != PGEMM_OK) return e;
        OpArena arena(dev, s);
        const long long at = arena.add(dgain ? 4ll * blocks * D : 0);
        if ((e = arena.alloc()) != PGEMM_OK) return e;
        NormParams q = p;
        q.dgain = dgain ? arena.at<float>(at) : nullptr;
        e = launch_small_smem(rmsnorm_backward_kernel<N, V>, dim3(blocks), dim3(N), smem, s, q);
        if (e != PGEMM_OK || !dgain) return e;
        return launch_small(norm_join_kernel, dim3(op_blocks(D, 32)), dim3(256), s,
                            static_cast<const float *>(q.dgain), blocks, D, dgain);
    });
}

}  // namespace pg

extern "C" {

pgemm_status rmsnorm_bf16(int T, int D, const uint16_t *X, const uint16_t *R, const uint16_t *gain,
                          float eps, uint16_t *S, uint16_t *Y, pgemm_stream_t stream) {
    return pg::op_guard([&] {
        return pg::norm_forward(false, T, D, X, R, gain, eps, S, Y, nullptr, stream);
    });
}

pgemm_status rmsnorm_i8(int T, int D, const uint16_t *X, const uint16_t *R, const uint16_t *gain,
                        float eps, uint16_t *S, int8_t *Q, float *scale, pgemm_stream_t stream) {
    return pg::op_guard(
        [&] { return pg::norm_forward(true, T, D, X, R, gain, eps, S, Q, scale, stream); });
}

pgemm_status rmsnorm_bf16_backward(int T, int D, const uint16_t *S, const uint16_t *gain,
                                   float eps, const uint16_t *dY, const uint16_t *dS, uint16_t *dX,
                                   uint16_t *dgain, pgemm_stream_t stream) {
    return pg::op_guard(
        [&] { return pg::norm_backward(T, D, S, gain, eps, dY, dS, dX, dgain, stream); });
}

}  // extern "C"
