// The generic product of the operators (forms NN, NT and TN, bf16 output with
// an optional bias, activation and residual), its split along K, and the
// elementwise gradient pass in front of the gradient products.
#include <cuda_runtime.h>

#include "op_act.cuh"
#include "op_gemm.cuh"
#include "op_host.h"

namespace pg {

// ------------------------------------------------------------- epilogue ---
// out = round(act(acc + bias) + residual) to bf16, once, from fp32; or, for a
// product split along K, the accumulator itself as one of the parts.
// FULL = false: no bias, activation, residual or kept pre-activation (the
// gradient products), so that their kernels carry none of it.
template <bool FULL>
struct EpiOut {
    const uint16_t *bias, *residual;
    float *preact, *parts;
    const float *scale;     // one device value that multiplies acc, or nullptr
    uint16_t *out[2];
    long long ldo;          // row length of out, residual and preact
    long long parts_rows;
    int parts_segments;
    int act;
    int tma_out, tma_preact;
    int plain;  // no bias, activation, residual or kept pre-activation

    template <class Cfg, class Acc>
    __device__ __forceinline__ bool run(EpiCtx<Cfg::NBUF> &c, const OpMaps &maps, const OpArgs &,
                                        const OpUnit &w, Acc &acc, uint32_t e) const {
        int col0, cols;
        epi_cols<Cfg>(w, e, col0, cols);
        const int nf = w.n0 + col0;
        const bool have = acc.have();
        const CUtensorMap *map = tma_out ? &maps.c[w.seg] : nullptr;
        uint16_t *o = out[w.seg];
        const int row0 = static_cast<int>(
            (static_cast<long long>(w.part) * parts_segments + w.seg) * parts_rows + c.m0);
        auto put_part = [&](int n, const uint32_t *v) {
            put_words16(c, &maps.c[0], nullptr, 0, row0, n, v);
            put_words16(c, &maps.c[0], nullptr, 0, row0, n + 16, v + 16);
        };
        // the residual's next columns travel while the products finish, and then
        // while the present ones are worked on
        RowsIn res{residual, ldo};
        const bool have_r = FULL && residual != nullptr && parts == nullptr;
        // 32 columns from nf + cc: v holds the accumulator's
        auto finish = [&](int cc, uint32_t *v) {
            const int n = nf + cc;
            uint32_t p[16];
            if (scale != nullptr) {
                const float f = *scale;
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * f);
            }
            if constexpr (FULL) {
                if (bias != nullptr) {
                    float b[32];
                    get_vec32(bias, c.N, n, b);
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[j] = __float_as_uint(__uint_as_float(v[j]) + b[j]);
                }
                if (preact != nullptr) {
                    const CUtensorMap *mz = tma_preact ? &maps.c[2] : nullptr;
                    put_words16(c, mz, preact, ldo, c.m0, n, v);
                    put_words16(c, mz, preact, ldo, c.m0, n + 16, v + 16);
                }
                auto activate = [&](auto A) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[j] = __float_as_uint(
                            act_value<decltype(A)::value>(__uint_as_float(v[j])));
                };
                if constexpr (Cfg::ROUND > 0)
                    activate(std::integral_constant<int, PGEMM_ACT_RELU>{});
                else if (act != PGEMM_ACT_NONE)
                    with_act(act, activate);
                if (have_r) {
                    uint32_t r[16];
                    res.take(c, r);
                    if (cc + 32 < cols) res.load(c, n + 32);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        v[2 * j] = __float_as_uint(__uint_as_float(v[2 * j]) + bf16_lo(r[j]));
                        v[2 * j + 1] =
                            __float_as_uint(__uint_as_float(v[2 * j + 1]) + bf16_hi(r[j]));
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < 16; ++j)
                p[j] = pack_bf16(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
            put_rows32(c, map, o, ldo, n, p);
        };
        if constexpr (Cfg::ROUND > 0) {
            float f[Cfg::EPI_COLS];
            if (!acc_sum_unit<Cfg>(acc, col0, cols, f)) return false;
            if (have_r) res.load(c, nf);  // (the sums fill the registers until here)
#pragma unroll
            for (int b = 0; b < Cfg::EPI_COLS / 32; ++b) {
                if (32 * b >= cols) break;
                uint32_t v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(f[32 * b + j]);
                if (parts != nullptr)
                    put_part(nf + 32 * b, v);
                else
                    finish(32 * b, v);
            }
            return true;
        }
        if (plain && parts == nullptr && map != nullptr && have && cols == Cfg::EPI_COLS) {
            // nothing but rounding: read the whole accumulator at once, hand it
            // back, and stage as much as fits in one go
            if (!acc.wait()) return false;
            const uint32_t t_row = acc.row() + col0;
            constexpr int C = Cfg::EPI_COLS / 32, B = C < Cfg::NBUF ? C : Cfg::NBUF;
            uint32_t v[32 * C];
#pragma unroll
            for (int b = 0; b < C; ++b)
                tmem_ld_32x32b_x32(t_row + 32 * b, *reinterpret_cast<uint32_t(*)[32]>(v + 32 * b));
            tmem_ld_wait();
            acc.release();
            if (scale != nullptr) {
                const float f = *scale;
#pragma unroll
                for (int j = 0; j < 16 * C; ++j)
                    v[j] = pack_bf16(__uint_as_float(v[2 * j]) * f,
                                     __uint_as_float(v[2 * j + 1]) * f);
            } else {
#pragma unroll
                for (int j = 0; j < 16 * C; ++j)
                    v[j] = pack_bf16(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
            }
#pragma unroll
            for (int b = 0; b < C; b += B)
                put_rows32_batch<B>(c, map, nf + 32 * b, v + 16 * b);
            return true;
        }
        if (have_r) res.load(c, nf);
        if (!acc.wait()) return false;
        const uint32_t t_row = acc.row() + col0;
#pragma unroll 1
        for (int cc = 0; cc < cols; cc += 32) {
            uint32_t v[32];
            acc_cols32(t_row + cc, have, v);
            if (cc + 32 >= cols) acc.release();
            if (parts != nullptr)
                put_part(nf + cc, v);
            else
                finish(cc, v);
        }
        return true;
    }
};

// --------------------------------------------------------------- choice ---
// Time of a product, from graphs of calls on warm operands (us, 19 shapes from
// 135 x 256 x 208 to 2560 x 1384 x 3432, within 10 %): a launch and its first
// tile's pipeline and epilogue, then for every wave its 64-wide K steps, and an
// epilogue between waves that the next tile does not hide.  A CTA pair's tiles
// (256 x 256) go faster a product but cost more to start than 128 x 128 tiles on
// single CTAs; its leftover tiles run as half-width units where those fit.
// Parts along K shorten the waves and add the join: its launch, and parts * M * N
// fp32 values written and read.
struct WaveCost {
    double fixed, step, half_step;
};
constexpr WaveCost kPairCost{5.0, 0.32, 0.25}, kOneCost{3.4, 0.29, 0.29};
constexpr double kWaveGapUs = 0.8, kJoinUs = 4.0, kJoinUsPerMB = 0.25;

static double wave_us(bool pair, long long tiles, int sm_count, long long steps) {
    const WaveCost &c = pair ? kPairCost : kOneCost;
    const long long slots = pair ? sm_count / 2 : sm_count;
    const long long whole = tiles / slots, left = tiles % slots;
    double us = c.fixed + static_cast<double>(whole) * static_cast<double>(steps) * c.step;
    if (left > 0)
        us += static_cast<double>(steps) * (pair && 2 * left <= slots ? c.half_step : c.step);
    return us + kWaveGapUs * static_cast<double>(whole + (left > 0) - 1);
}

static OpPlan plan_product(int sm_count, long long M, long long N, long long K, int segments,
                           bool split, double *best_time = nullptr) {
    const long long steps = (K + 63) / 64;
    OpPlan best{false, 1};
    double best_us = 1e30;
    for (int pair = 0; pair < 2; ++pair) {
        const long long b = pair ? 256 : 128;
        const long long tiles = ((M + b - 1) / b) * ((N + b - 1) / b) * segments;
        for (const int parts : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
            if (parts > 1 && (!split || steps / parts < 8)) break;
            double us = wave_us(pair != 0, tiles * parts, sm_count, (steps + parts - 1) / parts);
            if (parts > 1)
                us += kJoinUs + kJoinUsPerMB * 4e-6 * parts * static_cast<double>(M) *
                                    static_cast<double>(N) * segments;
            if (us < best_us * 0.999) {
                best_us = us;
                best = OpPlan{pair != 0, parts};
            }
        }
    }
    if (best_time != nullptr) *best_time = best_us;
    return best;
}

double op_product_us(const OpDevice &dev, long long M, long long N, long long K) {
    double us = 0.0;
    plan_product(dev.sm_count, M, N, K, 1, true, &us);
    return us;
}
double op_gated_us(const OpDevice &dev, long long M, long long F, long long K) {
    const long long steps = (K + 63) / 64;
    const double pair = wave_us(true, ((M + 255) / 256) * ((F + 127) / 128), dev.sm_count, steps);
    const double one = wave_us(false, ((M + 127) / 128) * ((F + 63) / 64), dev.sm_count, steps);
    return pair < one ? pair : one;
}

bool op_use_pair(const OpDevice &dev, long long M, long long N, long long K, long long pair_n,
                 long long one_n) {
    const long long steps = (K + 63) / 64;
    const long long tp = ((M + 255) / 256) * ((N + pair_n - 1) / pair_n);
    const long long t1 = ((M + 127) / 128) * ((N + one_n - 1) / one_n);
    return wave_us(true, tp, dev.sm_count, steps) <= wave_us(false, t1, dev.sm_count, steps);
}

int op_product_parts(const OpDevice &dev, int M, int N, int K, int segments) {
    return plan_product(dev.sm_count, M, N, K, segments, true).parts;
}
long long op_parts_ld(int N) { return op_round_up(N, 64); }
long long op_parts_rows(int M) { return op_round_up(M, 32); }

// ----------------------------------------------------------------- launch ---
template <class Cfg, bool FULL>
static pgemm_status launch_form(const OpDevice &dev, const OpProduct &p, float *parts_area,
                                int parts, cudaStream_t s) {
    constexpr int TM = Cfg::BM * Cfg::CG, TN = Cfg::TILE_N;
    OpMaps maps{};
    for (int j = 0; j < 2; ++j) {
        const OpMat &a = p.A[p.k_segments == 2 ? j : 0];
        const OpMat &b = p.B[(p.k_segments == 2 || p.n_segments == 2) ? j : 0];
        pgemm_status st;
        if (p.K > 0) {
            st = Cfg::A_MN ? op_encode(&maps.a[j], a.p, p.M, p.K, a.ld, 64)
                           : op_encode(&maps.a[j], a.p, p.K, p.M, a.ld, 128);
            if (st == PGEMM_OK)
                st = Cfg::B_K ? op_encode(&maps.b[j], b.p, p.K, p.N, b.ld, 64)
                              : op_encode(&maps.b[j], b.p, p.N, p.K, b.ld, 64);
            if (st != PGEMM_OK) return st;
        }
    }
    EpiOut<FULL> e{};
    e.act = p.epi.act;
    e.scale = p.epi.scale;
    e.bias = p.epi.bias;
    e.residual = p.epi.residual;
    e.preact = p.epi.preact;
    e.out[0] = p.out[0];
    e.out[1] = p.out[1];
    e.ldo = p.N;
    e.parts = parts_area;
    e.plain = !e.bias && !e.residual && !e.preact && e.act == PGEMM_ACT_NONE;
    if (parts_area != nullptr) {
        if (op_parts_ld(p.N) > 0x7fffffffll) return PGEMM_ERR_INVALID_VALUE;
        e.parts_rows = op_parts_rows(p.M);
        e.parts_segments = p.n_segments;
        const pgemm_status st =
            op_encode_out(&maps.c[0], OpElem::F32, parts_area, op_parts_ld(p.N),
                          e.parts_rows * parts * p.n_segments, op_parts_ld(p.N));
        if (st != PGEMM_OK) return st;
    } else {
        e.tma_out = p.N % 8 == 0;
        for (int j = 0; e.tma_out && j < p.n_segments; ++j) {
            const pgemm_status st =
                op_encode_out(&maps.c[j], OpElem::BF16, p.out[j], p.N, p.M, p.N);
            if (st != PGEMM_OK) return st;
        }
        e.tma_preact = e.preact != nullptr && p.N % 4 == 0;
        if (e.tma_preact) {
            const pgemm_status st =
                op_encode_out(&maps.c[2], OpElem::F32, e.preact, p.N, p.M, p.N);
            if (st != PGEMM_OK) return st;
        }
    }
    OpArgs a{};
    a.M = p.M;
    // the parts' padding columns are written too, so that the join reads whole vectors
    a.N = parts_area != nullptr ? static_cast<int>(op_parts_ld(p.N)) : p.N;
    a.K = p.K;
    a.m_tiles = op_blocks(p.M, TM);
    a.n_seg = op_blocks(p.N, TN);
    a.n_tiles = a.n_seg * p.n_segments;
    a.k_seg = op_blocks(p.K, Cfg::SBK);
    a.k_tiles = a.k_seg * p.k_segments;
    a.parts = parts;
    a.overlap = p.overlap ? 1 : 0;
    return op_launch<Cfg, EpiOut<FULL>>(dev, maps, a, e, s);
}

template <bool A_MN, bool B_K>
using PairCfg = OpCfg<256, 3, 2, 2, A_MN, B_K>;
// Short K: a unit's epilogue takes longer than its products, so the ring gives
// up a sixth for staging buffers that hold a warp's whole output (four instead
// of two).  8192 x 8192 outputs, us with this and with three 128-column stages:
// K = 64 35.2 against 43.5, K = 256 41.7 against 50.9, K = 512 57.0 against
// 55.8, K = 2048 (4096 x 4096) 46.4 against 42.0.
constexpr int kShortK = 384;
template <bool A_MN, bool B_K>
using ShortCfg = OpCfg<256, 5, 1, 2, A_MN, B_K, false, 0, 4>;
template <bool A_MN, bool B_K>
using OneCfg = OpCfg<128, 6, 1, 1, A_MN, B_K>;
using SignPairCfg = OpCfg<256, 3, 2, 2, false, false, false, SignPair::value>;
using SignOneCfg = OpCfg<128, 6, 1, 1, false, false, false, SignOne::value>;

template <bool FULL, bool A_MN, bool B_K>
static pgemm_status launch_size(const OpDevice &dev, const OpProduct &p, float *area,
                                cudaStream_t s) {
    const OpPlan &plan = p.plan;
    if constexpr (FULL) {
        if (p.epi.preact && op_sign_rounds(p.epi.act, p.K))
            return plan.pair ? launch_form<SignPairCfg, FULL>(dev, p, area, plan.parts, s)
                             : launch_form<SignOneCfg, FULL>(dev, p, area, plan.parts, s);
    }
    if (plan.pair && static_cast<long long>(p.K) * p.k_segments <= kShortK)
        return launch_form<ShortCfg<A_MN, B_K>, FULL>(dev, p, area, plan.parts, s);
    return plan.pair ? launch_form<PairCfg<A_MN, B_K>, FULL>(dev, p, area, plan.parts, s)
                     : launch_form<OneCfg<A_MN, B_K>, FULL>(dev, p, area, plan.parts, s);
}

void op_product_plan(const OpDevice &dev, OpProduct &p, OpArena &arena) {
    p.plan = plan_product(dev.sm_count, p.M, p.N, static_cast<long long>(p.K) * p.k_segments,
                          p.n_segments, true);
    if (p.plan.parts > 1 && p.parts_area == nullptr && p.M > 0 && p.N > 0)
        p.area_at = arena.add(op_parts_ld(p.N) * op_parts_rows(p.M) * 4 * p.plan.parts *
                              p.n_segments);
}

pgemm_status op_product(const OpDevice &dev, const OpProduct &p, const OpArena &arena,
                        cudaStream_t s) {
    if (p.M <= 0 || p.N <= 0) return PGEMM_OK;
    float *area = p.parts_area ? p.parts_area : p.area_at >= 0 ? arena.at<float>(p.area_at) : nullptr;
    switch (p.form) {
        case OpForm::NN: return launch_size<true, false, false>(dev, p, area, s);
        case OpForm::NT: return launch_size<false, false, true>(dev, p, area, s);
        case OpForm::TN: return launch_size<false, true, false>(dev, p, area, s);
    }
    return PGEMM_ERR_INVALID_VALUE;
}

pgemm_status op_product_join(const OpDevice &dev, const OpProduct &p, const OpArena &arena,
                             cudaStream_t s) {
    if (p.area_at < 0) return PGEMM_OK;
    return op_join_parts(dev, arena.at<float>(p.area_at), p.plan.parts, p.n_segments, p.M, p.N,
                         p.out, p.epi, s);
}

// ------------------------------------------------------------------- join ---
// Memory-bound: reads parts * M * N fp32 values once, writes M * N bf16 (two
// parts of 4096 x 4096: 34 us, 4.9 TB/s; 54 us with one place a thread).  A
// thread owns four columns of a row, so loads are 16 bytes and the parts are
// added in order (the result does not depend on timing).  Eight loads travel at
// a time: of eight parts, or with few parts two each of four places.
struct JoinParams {
    const float *area;
    long long ld, rows;
    int parts, segments, M, N;
    uint16_t *out[2];
    OpEpilogue e;
};

template <int PLACES>
__global__ void __launch_bounds__(256) join_parts_kernel(const JoinParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int AHEAD = 8 / PLACES;
    const unsigned quads = (static_cast<unsigned>(p.N) + 3) / 4;
    const long long total = static_cast<long long>(p.M) * quads * p.segments;
    const long long step = p.segments * p.rows * p.ld;
    for (long long i0 = blockIdx.x * (256ll * PLACES) + threadIdx.x; i0 < total;
         i0 += gridDim.x * (256ll * PLACES)) {
        const float *src[PLACES];
        long long at[PLACES];
        int n[PLACES], seg[PLACES];
        float v[PLACES][4];
#pragma unroll
        for (int u = 0; u < PLACES; ++u) {
            const long long i = i0 + 256 * u < total ? i0 + 256 * u : i0;
            // segment * M + row (a 32-bit division where it fits)
            const long long sm = total <= 0xffffffffll
                                     ? static_cast<unsigned>(i) / quads
                                     : i / static_cast<long long>(quads);
            n[u] = static_cast<int>(i - sm * quads) * 4;
            seg[u] = sm >= p.M ? 1 : 0;
            const long long m = sm - (seg[u] ? p.M : 0);
            src[u] = p.area + (seg[u] * p.rows + m) * p.ld + n[u];
            at[u] = m * p.N + n[u];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[u][j] = 0.0f;
        }
        for (int k = 0; k < p.parts; k += AHEAD) {
            float4 x[PLACES][AHEAD];
#pragma unroll
            for (int u = 0; u < PLACES; ++u)
#pragma unroll
                for (int j = 0; j < AHEAD; ++j)
                    x[u][j] = k + j < p.parts
                                  ? __ldcs(reinterpret_cast<const float4 *>(src[u] + (k + j) * step))
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int u = 0; u < PLACES; ++u)
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) {
                    v[u][0] += x[u][j].x;
                    v[u][1] += x[u][j].y;
                    v[u][2] += x[u][j].z;
                    v[u][3] += x[u][j].w;
                }
        }
#pragma unroll
        for (int u = 0; u < PLACES; ++u) {
            if (u > 0 && i0 + 256 * u >= total) break;
            const int cols = min(4, p.N - n[u]);
            if (p.e.scale) {
                const float f = *p.e.scale;
#pragma unroll
                for (int j = 0; j < 4; ++j) v[u][j] *= f;
            }
            if (p.e.bias || p.e.preact) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j >= cols) break;
                    if (p.e.bias)
                        v[u][j] += __uint_as_float(static_cast<uint32_t>(p.e.bias[n[u] + j]) << 16);
                    if (p.e.preact) p.e.preact[at[u] + j] = v[u][j];
                }
            }
            with_act(p.e.act, [&](auto A) {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[u][j] = act_value<decltype(A)::value>(v[u][j]);
            });
            if (p.e.residual) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < cols)
                        v[u][j] +=
                            __uint_as_float(static_cast<uint32_t>(p.e.residual[at[u] + j]) << 16);
            }
            uint16_t *o = (seg[u] ? p.out[1] : p.out[0]) + at[u];
            const uint32_t lo = pack_bf16(v[u][0], v[u][1]), hi = pack_bf16(v[u][2], v[u][3]);
            if (p.N % 4 == 0) {
                *reinterpret_cast<uint2 *>(o) = make_uint2(lo, hi);
            } else {
                const uint32_t w[4] = {lo & 0xffffu, lo >> 16, hi & 0xffffu, hi >> 16};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < cols) o[j] = static_cast<uint16_t>(w[j]);
            }
        }
    }
}

pgemm_status op_join_parts(const OpDevice &dev, const float *area, int parts, int segments, int M,
                           int N, uint16_t *const out[2], const OpEpilogue &epi,
                           cudaStream_t s) {
    JoinParams p{};
    p.area = area;
    p.ld = op_parts_ld(N);
    p.rows = op_parts_rows(M);
    p.parts = parts;
    p.segments = segments;
    p.M = M;
    p.N = N;
    p.out[0] = out[0];
    p.out[1] = out[1];
    p.e = epi;
    // four places a thread where there are blocks enough for every SM all the same
    const long long places = static_cast<long long>(M) * op_blocks(N, 4) * segments;
    const bool four = parts <= 4 && places >= 1024ll * 2 * dev.sm_count;
    const long long blocks = (places + (four ? 1023 : 255)) / (four ? 1024 : 256);
    const long long most = dev.sm_count * 8ll;
    return launch_small(four ? join_parts_kernel<4> : join_parts_kernel<1>,
                        dim3(static_cast<unsigned>(blocks < most ? blocks : most)), dim3(256), s, p);
}

// Adds in the order that join_parts_kernel does, so that folding some parts before
// the rest are joined changes no bit.  Memory-bound: a running sum of 4096 x 4096 and
// one more such matrix take 24 us among a piece's products (201 MB, some of it in L2).
__global__ void __launch_bounds__(256)
    fold_parts_kernel(float4 *area, int parts, long long step, long long total) {
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int AHEAD = 4;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < parts; k += AHEAD) {
            float4 x[AHEAD];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j)
                x[j] = k + j < parts ? __ldcs(area + (k + j) * step + i)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                v.x += x[j].x;
                v.y += x[j].y;
                v.z += x[j].z;
                v.w += x[j].w;
            }
        }
        area[i] = v;
    }
}

pgemm_status op_fold_parts(const OpDevice &dev, float *area, int parts, int M, int N,
                           cudaStream_t s) {
    const long long total = op_parts_ld(N) / 4 * M;
    const long long blocks = (total + 255) / 256, most = dev.sm_count * 8ll;
    return launch_small(fold_parts_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)),
                        dim3(256), s, reinterpret_cast<float4 *>(area), parts,
                        op_parts_ld(N) / 4 * op_parts_rows(M), total);
}

// --------------------------------------------------- activation gradient ---
// dZ = dY * act'(Z) (linear), dG = dH * U * act'(G) and dU = dH * act(G)
// (gated), elementwise in fp32 from the kept fp32 pre-activations, rounded to
// bf16 because the tensor core multiplies them next; column sums of the
// dZ for the bias (unrounded here; where a product computed Z again, of the bf16 dZ
// that it left).  Memory-bound: 8 (gated 14) bytes an element; gated
// 8192 x 8192 takes 128 us (7.3 TB/s, some of Z still in L2), linear 4096 x 4096
// 24 us (5.6 TB/s).
// A block covers 256 columns x kGradRows rows; a thread eight columns of every
// eighth row, so its part of a column sum stays in registers.  VEC: the eight
// columns are adjacent (16-byte accesses; row lengths multiples of 8), else 32
// apart (coalesced single elements).
constexpr int kGradRows = 64;

struct ActGradParams {
    OpActGrad g;
    float *colsum;  // [row blocks][N] partial column sums, or nullptr
    int overlap;
};

__device__ __forceinline__ void load8(const float *p, float (&f)[8]) {
    const float4 a = __ldcs(reinterpret_cast<const float4 *>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

template <bool VEC, bool GATED>
__global__ void __launch_bounds__(256) act_grad_kernel(const ActGradParams p) {
    op_begin(p.overlap);
    const OpActGrad &g = p.g;
    const int lane = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int c0 = blockIdx.x * 256;
    auto col = [&](int i) { return VEC ? c0 + lane * 8 + i : c0 + lane + 32 * i; };
    float sum[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
    // row blocks blockIdx.y, blockIdx.y + gridDim.y, ...: rows of stride 8 in each
    for (long long rr = static_cast<long long>(blockIdx.y) * kGradRows + rl; rr < g.M;
         rr += ((rr & (kGradRows - 1)) + 8 < kGradRows
                    ? 8
                    : 8 + static_cast<long long>(gridDim.y - 1) * kGradRows)) {
        const int r = static_cast<int>(rr);
        const long long zi = static_cast<long long>(r) * g.N;
        const long long yi = static_cast<long long>(r) * g.dy_ld;
        float z[8], u[8], dy[8];
        if (VEC) {
            if (col(0) >= g.N) continue;
            if (g.z) load8(g.z + zi + col(0), z);
            if (GATED) load8(g.u + zi + col(0), u);
            const uint4 x = *reinterpret_cast<const uint4 *>(g.dy + yi + col(0));
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dy[2 * i] = bf16_lo(w[i]);
                dy[2 * i + 1] = bf16_hi(w[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool in = col(i) < g.N;
                z[i] = in && g.z ? g.z[zi + col(i)] : 0.0f;
                u[i] = GATED && in ? g.u[zi + col(i)] : 0.0f;
                dy[i] = in ? __uint_as_float(static_cast<uint32_t>(g.dy[yi + col(i)]) << 16) : 0.0f;
            }
        }
        float dz[8], du[8];
        with_act(g.act, [&](auto A) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float value = 0.0f;
                const float d = decltype(A)::value == PGEMM_ACT_NONE && !GATED
                                    ? 1.0f
                                    : act_value_grad<decltype(A)::value>(z[i], value);
                dz[i] = dy[i] * d * (GATED ? u[i] : 1.0f);
                du[i] = dy[i] * value;
            }
        });
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += dz[i];
        const long long oi = static_cast<long long>(r) * g.dz_ld;
        auto put = [&](uint16_t *o, const float (&d)[8]) {
            if (o == nullptr) return;
            if (VEC) {
                *reinterpret_cast<uint4 *>(o + oi + col(0)) =
                    make_uint4(pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3]),
                               pack_bf16(d[4], d[5]), pack_bf16(d[6], d[7]));
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (col(i) < g.N)
                        o[oi + col(i)] = static_cast<uint16_t>(pack_bf16(d[i], 0.0f) & 0xffffu);
            }
        };
        put(g.dz, dz);
        if (GATED) put(g.du, du);
    }
    if (p.colsum != nullptr) {
        __shared__ float s[8][256];
#pragma unroll
        for (int i = 0; i < 8; ++i) s[rl][VEC ? lane * 8 + i : lane + 32 * i] = sum[i];
        __syncthreads();
        const int c = c0 + threadIdx.x;
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += s[i][threadIdx.x];
        if (c < g.N) p.colsum[static_cast<long long>(blockIdx.y) * g.N + c] = t;
    }
    op_end(p.overlap);
}

// dbias = sum of the row blocks' column sums, in order.
__global__ void __launch_bounds__(256)
    colsum_join_kernel(const float *part, int blocks, int N, uint16_t *out, int overlap) {
    op_begin(overlap);
    __shared__ float s[8][32];
    const int lane = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float t = 0.0f;
    if (c < N)
        for (int b = rl; b < blocks; b += 8) t += part[static_cast<long long>(b) * N + c];
    s[rl][lane] = t;
    __syncthreads();
    if (rl == 0 && c < N) {
#pragma unroll
        for (int i = 1; i < 8; ++i) t += s[i][lane];
        out[c] = static_cast<uint16_t>(pack_bf16(t, 0.0f) & 0xffffu);
    }
    op_end(overlap);
}

static int grad_row_blocks(const OpActGrad &g) {
    const int all = op_blocks(g.M, kGradRows);
    return all < 512 ? all : 512;
}

void op_act_grad_plan(OpActGrad &g, OpArena &arena) {
    if (g.dbias != nullptr) g.colsum_at = arena.add(grad_row_blocks(g) * 4ll * g.N);
}

pgemm_status op_act_grad(const OpDevice &, const OpActGrad &g, const OpArena &arena, bool overlap,
                         cudaStream_t s) {
    if (g.M <= 0 || g.N <= 0) return PGEMM_OK;
    const ActGradParams p{g, g.dbias ? arena.at<float>(g.colsum_at) : nullptr, overlap ? 1 : 0};
    const dim3 grid(op_blocks(g.N, 256), grad_row_blocks(g));
    const bool vec = g.N % 8 == 0 && g.dy_ld % 8 == 0;
    if (g.u != nullptr)
        return vec ? launch_small(act_grad_kernel<true, true>, grid, dim3(256), s, p)
                   : launch_small(act_grad_kernel<false, true>, grid, dim3(256), s, p);
    return vec ? launch_small(act_grad_kernel<true, false>, grid, dim3(256), s, p)
               : launch_small(act_grad_kernel<false, false>, grid, dim3(256), s, p);
}

pgemm_status op_act_grad_join(const OpDevice &, const OpActGrad &g, const OpArena &arena,
                              bool overlap, cudaStream_t s) {
    if (g.M <= 0 || g.N <= 0 || g.dbias == nullptr) return PGEMM_OK;
    return launch_small(colsum_join_kernel, dim3(op_blocks(g.N, 32)), dim3(256), s,
                        static_cast<const float *>(arena.at<float>(g.colsum_at)),
                        grad_row_blocks(g), g.N, g.dbias, overlap ? 1 : 0);
}

// --------------------------------------------------------------- relayout ---
pgemm_status OpRelayout::run(const OpDevice &dev, OpArena &arena, cudaStream_t s) {
    for (int i = 0; i < n_; ++i) {
        jobs_[i].out->p = arena.at<uint16_t>(jobs_[i].at);
        jobs_[i].out->ld = jobs_[i].ld;
    }
    for (int i = 0; i < n_; i += 2) {
        const Job &a = jobs_[i];
        const Job *b = i + 1 < n_ ? &jobs_[i + 1] : nullptr;
        if (launch_repack(a.src, a.cols, arena.at<uint16_t>(a.at), a.ld, static_cast<int>(a.rows),
                          static_cast<int>(a.cols), b ? b->src : nullptr, b ? b->cols : 0,
                          b ? arena.at<uint16_t>(b->at) : nullptr, b ? b->ld : 0,
                          b ? static_cast<int>(b->rows) : 0, b ? static_cast<int>(b->cols) : 0, 2,
                          dev.sm_count, s) != cudaSuccess)
            return PGEMM_ERR_CUDA;
    }
    return PGEMM_OK;
}

}  // namespace pg
