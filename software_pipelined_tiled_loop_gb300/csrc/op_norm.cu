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
// outputs, so every operand is read once; the next row's operands travel meanwhile where
// registers hold them (up to 512 threads; backward, up to two vectors a thread).  All
// operands have the same pitch and 16-byte-aligned bases, so a row starts at the same place
// of a 16-byte vector in each: a thread takes whole aligned vectors (eight elements of the
// flat matrix), masked at the row's two ends, whatever the width.  Bound by HBM: 8192 x 4096
// with a residual 42 us (6.4 TB/s), as int8 40 (5.9), backward 49 (5.5; the gains' gradient
// and its join 5 of them); 4097 x 5120 27.5, 27.8 and 46.5, 4097 x 5121 33, 37.3 and 50.5,
// 2048 x 16384 45, 48.5 and 73.  Backward, wider rows than 4096 leave an SM one block or two
// with too little on the way.  Above 20480 values registers spill, backward most (1024 x 32768
// 55, 62 and 207).  One row of 4096 1.8 us from a graph.
#include <cuda_runtime.h>

#include "op_gemm.cuh"
#include "op_host.h"
#include "op_rows.cuh"

namespace pg {

constexpr int kNormMaxD = 32768;

// The gains of vector v's columns (ones without gains; anything where the row is not).
__device__ __forceinline__ uint4 gain_load(const uint16_t *g, const RowSpan &r, int v) {
    if (g == nullptr) return make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    const int c0 = r.col(v);
    if (r.whole(v) && c0 / 8 * 8 + 16 <= r.D) {
        const uint4 *at = reinterpret_cast<const uint4 *>(g) + c0 / 8;
        shift16(__ldg(at), __ldg(at + 1), static_cast<uint32_t>(c0 & 7) * 2u, w);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c0 + i >= 0 && c0 + i < r.D)
                w[i / 2] |= static_cast<uint32_t>(__ldg(g + c0 + i)) << (i % 2 * 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The sums of N values over the block's threads, in an order that does not depend on timing,
// and the largest `most`; the same in every thread.  `part` may be used again after the
// block's next barrier.
template <int N, bool MOST>
__device__ __forceinline__ void block_reduce(float (&x)[N], uint32_t &most,
                                             uint32_t (*part)[32]) {
    auto lanes = [&] {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) x[i] += __shfl_xor_sync(0xffffffffu, x[i], d);
        if constexpr (MOST) most = __reduce_max_sync(0xffffffffu, most);
    };
    lanes();
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warps > 1) {
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) part[i][warp] = __float_as_uint(x[i]);
            if constexpr (MOST) part[N][warp] = most;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = lane < warps ? __uint_as_float(part[i][lane]) : 0.0f;
        if constexpr (MOST) most = lane < warps ? part[N][lane] : 0u;
        lanes();
    }
}

// A magnitude as bits: ordered as the numbers are, infinity behind them, NaN behind that.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Four integers of at most 127, rounded to nearest with ties to even by adding 1.5 * 2^23,
// below which a float's last place is one.
__device__ __forceinline__ uint32_t round4_i8(const float *x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(x[i] + 12582912.0f);
    return __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
}

// With an eps of less than 2^-100 a row's squares may all have left fp32's range and its norm
// be finite.  Such calls have kernels of their own (ENDS): where mean(S^2) + eps lies outside
// 2^-100 .. infinity they go through the row again as S by, with eps by^2: by = 2^76 below
// (values under 2^-42, squares from 2^-114 to 2^84), 2^-72 above (squares up to 2^112; what
// that takes below bf16's range is 2^-110 of the norm's ones).  They take 5 % more time
// (8192 x 4096 backward 52.8 us for 49.4), which is why not all calls do.
constexpr float kEndsBelow = 7.8886091e-31f;
__device__ __forceinline__ bool var_fits(float var) {
    return var >= kEndsBelow && var < __int_as_float(0x7f800000);
}
__device__ __forceinline__ float var_shift(float var) {
    return var < 1.0f ? 7.5557864e22f : 2.1175824e-22f;
}
// Eight values of S, times by.
__device__ __forceinline__ void shift8(uint4 &s, float by) {
    float f[8];
    unpack8(s, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= by;
    s = pack8(f);
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
    int early;     // op_begin_early
};

// The gains of a thread's vectors.  A block's rows are a multiple of eight apart (norm_grid),
// so all of them start at the same place of a vector, and a thread has the same columns in
// each.
template <int V>
__device__ __forceinline__ void gains_load(const NormParams &p, const RowSpan &row,
                                           uint4 (&gains)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < row.vecs) gains[i] = gain_load(p.gain, row, v);
    }
}

// V vectors a thread, up to MOST threads; ALIGNED: D is a multiple of 8.  (Held to 64
// registers where rows are aligned and not wide: int8 8192 x 4096 39.9 us against 48.7; of
// other rows 4097 x 5121 would take 48.6 against 37.1, so those are left to the compiler.)
template <int V, int MOST, bool ALIGNED, bool I8, bool ENDS>
__global__ void __launch_bounds__(MOST, ALIGNED && V <= 2 ? 2 : 0)
    rmsnorm_kernel(const NormParams p) {
    __shared__ uint32_t part[2][2][32];
    constexpr bool AHEAD = MOST <= 512;  // (more leave no registers for the next row)
    op_begin_early(p.early);
    int turn = 0;
    uint4 a[V], b[V], gains[V];
    gains_load(p, RowSpan(ALIGNED ? 0 : blockIdx.x, p.T, p.D), gains);
    auto fetch = [&](unsigned t) {
        const RowSpan row(t, p.T, p.D);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = threadIdx.x + i * blockDim.x;
            a[i] = b[i] = make_uint4(0u, 0u, 0u, 0u);
            if (v < row.vecs) {
                a[i] = row_load(p.x, row, v);
                if (p.r) b[i] = row_load(p.r, row, v);
            }
        }
    };
    const unsigned T = p.T;  // (unsigned: a step behind the last row may pass 2^31)
    unsigned t = blockIdx.x;
    if (AHEAD && t < T) fetch(t);
    for (; t < T; t += gridDim.x) {
        if (!AHEAD) fetch(t);
        const RowSpan row(t, p.T, p.D);
        uint4 s[V];
        float sum[1] = {0.0f};  // of squares
        uint32_t most = 0u;     // int8: the largest |S gain|
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = threadIdx.x + i * blockDim.x;
            if (!ALIGNED && v < row.vecs) {
                row_mask(a[i], row, v);
                row_mask(b[i], row, v);
            }
            float f[8];
            unpack8(a[i], f);
            s[i] = a[i];
            if (p.r) {
                float g[8];
                unpack8(b[i], g);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] += g[j];
                s[i] = pack8(f);  // S as it is stored
                unpack8(s[i], f);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[0] = fmaf(f[j], f[j], sum[0]);
            if constexpr (I8) {
                if (v < row.vecs) {
                    float g[8];
                    unpack8(gains[i], g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) most = max(most, magnitude(f[j] * g[j]));
                }
            }
            if (p.s && v < row.vecs) row_store(p.s, row, v, s[i]);
        }
        // (S may be X or R: a row's stores touch no other row)
        if (AHEAD && t + gridDim.x < T) fetch(t + gridDim.x);
        block_reduce<1, I8>(sum, most, part[turn]);
        turn ^= 1;
        float var = sum[0] / static_cast<float>(p.D) + p.eps;
        bool fits = true;
        if constexpr (ENDS) {
            fits = var_fits(var);
            if (!fits) {
                const float by = var_shift(var);
                sum[0] = 0.0f;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    shift8(s[i], by);
                    float f[8];
                    unpack8(s[i], f);
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[0] = fmaf(f[j], f[j], sum[0]);
                }
                uint32_t none = 0u;
                block_reduce<1, false>(sum, none, part[turn]);
                turn ^= 1;
                var = sum[0] / static_cast<float>(p.D) + p.eps * by * by;
            }
        }
        const float rstd = 1.0f / sqrtf(var);  // (ENDS: of S by)
        auto value = [&](int i, float (&y)[8]) {
            float g[8];
            unpack8(gains[i], g);
            unpack8(s[i], y);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = y[j] * rstd * g[j];
        };
        if constexpr (!I8) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int v = threadIdx.x + i * blockDim.x;
                if (v >= row.vecs) break;
                float y[8];
                value(i, y);
                row_store(p.y, row, v, pack8(y));
            }
        } else {
            // y = (S gain) rstd here, so that the largest |y| is the largest |S gain| times
            // rstd, with no second sum over the block, and Q = (S gain) (127 / the largest).
            // Where those come near the ends of the range the y are looked through instead,
            // and far below 1 scaled up first, so that the reciprocal is finite.
            const float product = __uint_as_float(most);
            float top = product * rstd, by = 1.0f, inv = 0.0f;
            const bool near = fits && product > 7.8886091e-31f && product < 1.2676506e30f &&  // 2^+-100
                              rstd > 0.0f && top < __int_as_float(0x7f800000);
            if (near) {
                inv = 127.0f / product;
            } else {
                most = 0u;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int v = threadIdx.x + i * blockDim.x;
                    if (v >= row.vecs) break;
                    float y[8];
                    value(i, y);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int c = row.col(v) + j;
                        if (ALIGNED || (c >= 0 && c < p.D)) most = max(most, magnitude(y[j]));
                    }
                }
                float none[1] = {0.0f};
                block_reduce<1, true>(none, most, part[turn]);
                turn ^= 1;
                top = __uint_as_float(most);
                by = top < 8.6736174e-19f ? 1.1529215e18f : 1.0f;  // 2^-60, 2^60
                if (top > 0.0f && top < __int_as_float(0x7f800000)) inv = 127.0f / (top * by);
            }
            if (threadIdx.x == 0)
                p.scale[t] = top < __int_as_float(0x7f800000) ? top / 127.0f
                                                              : __int_as_float(0x7fc00000);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int v = threadIdx.x + i * blockDim.x;
                if (v >= row.vecs) break;
                float y[8];
                if (near) {
                    float g[8];
                    unpack8(gains[i], g);
                    unpack8(s[i], y);
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] = y[j] * g[j] * inv;
                } else {
                    value(i, y);
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] = inv > 0.0f ? y[j] * by * inv : 0.0f;
                }
                const uint32_t w[2] = {round4_i8(y), round4_i8(y + 4)};
                int8_t *at = p.q + row.first + 8ll * v;
                if (ALIGNED || row.whole(v)) {
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

// The gains' gradient: each block leaves the sums of its rows' dY n for norm_join_kernel.  A
// thread keeps its columns' in its registers, or where a row is so wide that it has more
// than two vectors, in places of its own in shared memory.
enum class GainSum { NONE, REGISTERS, SHARED };

template <int V, int MOST, bool ALIGNED, GainSum SUM, bool ENDS>
__global__ void __launch_bounds__(MOST) rmsnorm_backward_kernel(const NormParams p) {
    extern __shared__ float4 sums[];  // [V][2][threads]
    __shared__ uint32_t part[2][2][32];
    constexpr bool AHEAD = V <= 2 && MOST <= 512;  // (else no registers for the next row)
    constexpr int OWN = SUM == GainSum::REGISTERS ? V : 1;
    float own[OWN][8];
#pragma unroll
    for (int i = 0; i < OWN; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) own[i][j] = 0.0f;
    auto place = [&](int i, int h) -> float4 & {
        return sums[(2 * i + h) * blockDim.x + threadIdx.x];
    };
    if constexpr (SUM == GainSum::SHARED) {
#pragma unroll
        for (int i = 0; i < V; ++i)
            place(i, 0) = place(i, 1) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    op_begin_early(p.early);
    int turn = 0;
    uint4 s[V], dy[V], ds[V], gains[V];
    gains_load(p, RowSpan(ALIGNED ? 0 : blockIdx.x, p.T, p.D), gains);
    auto fetch = [&](unsigned t, uint4 (&s)[V], uint4 (&dy)[V], uint4 (&ds)[V]) {
        const RowSpan row(t, p.T, p.D);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = threadIdx.x + i * blockDim.x;
            s[i] = dy[i] = ds[i] = make_uint4(0u, 0u, 0u, 0u);
            if (v < row.vecs) {
                s[i] = row_load(p.x, row, v);
                dy[i] = row_load(p.dy, row, v);
                if (p.ds) ds[i] = row_load(p.ds, row, v);
            }
        }
    };
    const unsigned T = p.T;
    unsigned t = blockIdx.x;
    if (t < T) fetch(t, s, dy, ds);
    for (; t < T; t += gridDim.x) {
        const RowSpan row(t, p.T, p.D);
        float both[2] = {0.0f, 0.0f};
        auto sum_up = [&] {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int v = threadIdx.x + i * blockDim.x;
                if (v >= row.vecs) break;
                if (!ALIGNED) {
                    row_mask(s[i], row, v);
                    row_mask(dy[i], row, v);
                }
                float fs[8], fd[8], g[8];
                unpack8(s[i], fs);
                unpack8(dy[i], fd);
                unpack8(gains[i], g);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    both[0] = fmaf(fs[j], fs[j], both[0]);
                    both[1] = fmaf(fd[j] * g[j], fs[j], both[1]);
                }
            }
        };
        sum_up();
        const unsigned after = t + gridDim.x;
        uint4 s1[V], dy1[V], ds1[V];
        if (AHEAD && after < T) fetch(after, s1, dy1, ds1);
        uint32_t none = 0u;
        block_reduce<2, false>(both, none, part[turn]);
        turn ^= 1;
        float var = both[0] / static_cast<float>(p.D) + p.eps, by = 1.0f;
        if constexpr (ENDS) {
            if (!var_fits(var)) {
                by = var_shift(var);
#pragma unroll
                for (int i = 0; i < V; ++i) shift8(s[i], by);
                both[0] = both[1] = 0.0f;
                sum_up();
                block_reduce<2, false>(both, none, part[turn]);
                turn ^= 1;
                var = both[0] / static_cast<float>(p.D) + p.eps * by * by;
            }
        }
        const float rstd = 1.0f / sqrtf(var);  // (ENDS: of S by)
        const float m = both[1] * rstd / static_cast<float>(p.D);  // mean(a n)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = threadIdx.x + i * blockDim.x;
            if (v >= row.vecs) break;
            float fs[8], fd[8], g[8], o[8];
            unpack8(s[i], fs);
            unpack8(dy[i], fd);
            unpack8(gains[i], g);
            unpack8(ds[i], o);
            float more[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float n = fs[j] * rstd;
                const float d = fmaf(-n, m, fd[j] * g[j]);
                o[j] += rstd * (ENDS ? by * d : d);
                if constexpr (SUM == GainSum::REGISTERS)
                    own[i][j] = fmaf(fd[j], n, own[i][j]);
                else
                    more[j] = fd[j] * n;
            }
            if constexpr (SUM == GainSum::SHARED) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float4 at = place(i, h);
                    at.x += more[4 * h];
                    at.y += more[4 * h + 1];
                    at.z += more[4 * h + 2];
                    at.w += more[4 * h + 3];
                    place(i, h) = at;
                }
            }
            if (p.dx) row_store(p.dx, row, v, pack8(o));
        }
        if (AHEAD) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                s[i] = s1[i];
                dy[i] = dy1[i];
                ds[i] = ds1[i];
            }
        } else if (after < T) {
            fetch(after, s, dy, ds);
        }
    }
    if constexpr (SUM != GainSum::NONE) {
        float *out = p.dgain + static_cast<long long>(blockIdx.x) * p.D;
        const RowSpan row(blockIdx.x, p.T, p.D);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = threadIdx.x + i * blockDim.x;
            if (v >= row.vecs) break;
            float4 x[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (SUM == GainSum::SHARED)
                    x[h] = place(i, h);
                else
                    x[h] = make_float4(own[i][4 * h], own[i][4 * h + 1], own[i][4 * h + 2],
                                       own[i][4 * h + 3]);
            }
            const int c = row.col(v);
            if constexpr (ALIGNED) {
                *reinterpret_cast<float4 *>(out + c) = x[0];
                *reinterpret_cast<float4 *>(out + c + 4) = x[1];
            } else {
                const float f[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j >= 0 && c + j < p.D) out[c + j] = f[j];
            }
        }
    }
}

// dgain = sum of the blocks' sums, in order: a warp takes every 32nd block's, 32 columns a
// block.
__global__ void __launch_bounds__(1024)
    norm_join_kernel(const float *part, int blocks, int D, uint16_t *out) {
    grid_dependency_wait();
    grid_launch_dependents();
    __shared__ float s[32][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float t = 0.0f;
    if (c < D) {
#pragma unroll 8
        for (int b = w; b < blocks; b += 32) t += part[static_cast<long long>(b) * D + c];
    }
    s[w][lane] = t;
    __syncthreads();
    if (w == 0 && c < D) {
#pragma unroll
        for (int i = 1; i < 32; ++i) t += s[i][lane];
        out[c] = static_cast<uint16_t>(pack_bf16(t, 0.0f) & 0xffffu);
    }
}

// f(vectors a thread, threads at most, whether rows start on vectors) as constants, and
// threads.  Two vectors a thread or one (`one`: up to 512): forward, two are quicker with rows
// for every SM (8192 x 4096 41.7 us against 48.9, 1500 x 4096 6.8 against 7.7) and one where a
// row's own latency counts (1 x 4096 1.8 against 2.0); backward, whose thread holds three
// operands and the next row's, one is (8192 x 4096 48.9 against 53.2, 400 x 4096 7.4 against
// 9.0).  Wider rows, backward: two again, without the next row, while their sums fit the
// registers (2730 x 12288 63 us, 2048 x 16384 72; with five 103 and 93).
template <bool BACKWARD, class F>
static pgemm_status with_row(int D, bool one, F &&f) {
    const int vecs = D % 8 == 0 ? D / 8 : (D + 14) / 8;
    using std::integral_constant;
    auto pick = [&](auto v, auto most) {
        const int threads = op_blocks(op_blocks(vecs, decltype(v)::value), 32) * 32;
        return D % 8 == 0 ? f(v, most, std::true_type{}, threads)
                          : f(v, most, std::false_type{}, threads);
    };
    const integral_constant<int, 512> few;
    if (vecs <= (one ? 512 : 32)) return pick(integral_constant<int, 1>{}, few);
    if (vecs <= 1024) return pick(integral_constant<int, 2>{}, few);
    if constexpr (BACKWARD) {
        if (vecs <= 1536) return pick(integral_constant<int, 2>{}, integral_constant<int, 768>{});
        if (vecs <= 2048) return pick(integral_constant<int, 2>{}, integral_constant<int, 1024>{});
    }
    if (vecs <= 2560) return pick(integral_constant<int, 5>{}, few);
    return pick(integral_constant<int, 5>{}, integral_constant<int, 832>{});
}

// Blocks for T rows, some `most` at most: a multiple of eight where one has more than a row.
static unsigned norm_grid(int T, long long most) {
    return static_cast<unsigned>(T <= most ? T : most < 8 ? 8 : most / 8 * 8);
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
    const bool one = T < 2 * dev.sm_count;
    return with_row<false>(D, one, [&](auto v, auto limit, auto aligned, int threads) {
        constexpr int V = decltype(v)::value, MOST = decltype(limit)::value;
        constexpr bool A = decltype(aligned)::value;
        const long long most = dev.sm_count * (threads >= 64 ? 2048ll / threads : 32ll);
        const dim3 grid(norm_grid(T, most));
        p.early = op_early(dev, grid.x);
        if (eps < kEndsBelow)
            return launch_small(i8 ? rmsnorm_kernel<V, MOST, A, true, true>
                                   : rmsnorm_kernel<V, MOST, A, false, true>,
                                grid, dim3(threads), s, p);
        return launch_small(i8 ? rmsnorm_kernel<V, MOST, A, true, false>
                               : rmsnorm_kernel<V, MOST, A, false, false>,
                            grid, dim3(threads), s, p);
    });
}

template <int V, int MOST, bool ALIGNED, GainSum SUM, bool ENDS>
static pgemm_status norm_backward_launch(const OpDevice &dev, dim3 grid, int threads, int smem,
                                         cudaStream_t s, const NormParams &p) {
    constexpr auto kernel = rmsnorm_backward_kernel<V, MOST, ALIGNED, SUM, ENDS>;
    if constexpr (SUM == GainSum::SHARED) {
        static const KernelInfo info = [] {
            KernelInfo k;
            k.threads = 32;
            k.smem_bytes = 32 * V * MOST;
            k.func = reinterpret_cast<const void *>(
                rmsnorm_backward_kernel<V, MOST, ALIGNED, SUM, ENDS>);
            return k;
        }();
        const pgemm_status st = op_kernel_setup(dev, info, nullptr);
        if (st != PGEMM_OK) return st;
    }
    return launch_small_smem(kernel, grid, dim3(threads), smem, s, p);
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
    return with_row<true>(D, true, [&](auto v, auto limit, auto aligned,
                                       int threads) -> pgemm_status {
        constexpr int V = decltype(v)::value, MOST = decltype(limit)::value;
        constexpr bool A = decltype(aligned)::value;
        constexpr GainSum SUM = V <= 2 ? GainSum::REGISTERS : GainSum::SHARED;
        // blocks of an SM: what registers and shared memory allow, eight at most, since
        // each leaves a row of sums behind
        const int smem = dgain && SUM == GainSum::SHARED ? 32 * V * threads : 0;
        int per_sm = threads <= 128 ? 8 : 1024 / threads;
        while (per_sm > 1 && per_sm * (smem + 2048) > kSmemPerSm) --per_sm;
        const int blocks = norm_grid(T, static_cast<long long>(dev.sm_count) * per_sm);
        p.early = op_early(dev, blocks);
        OpArena arena(dev, s);
        const long long at = arena.add(dgain ? 4ll * blocks * D : 0);
        pgemm_status e = arena.alloc();
        if (e != PGEMM_OK) return e;
        p.dgain = dgain ? arena.at<float>(at) : nullptr;
        const dim3 grid(blocks);
        const bool ends = eps < kEndsBelow;
        if (!dgain)
            return ends ? norm_backward_launch<V, MOST, A, GainSum::NONE, true>(dev, grid, threads,
                                                                                0, s, p)
                        : norm_backward_launch<V, MOST, A, GainSum::NONE, false>(dev, grid, threads,
                                                                                 0, s, p);
        e = ends ? norm_backward_launch<V, MOST, A, SUM, true>(dev, grid, threads, smem, s, p)
                 : norm_backward_launch<V, MOST, A, SUM, false>(dev, grid, threads, smem, s, p);
        if (e != PGEMM_OK) return e;
        return launch_small(norm_join_kernel, dim3(op_blocks(D, 32)), dim3(1024), s,
                            static_cast<const float *>(p.dgain), blocks, D, dgain);
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
