// Routing tokens to experts, and tokens sorted by expert and back.
//
//   route_topk     the k largest of a token's E logits (ties to the lowest index) and
//                  their weights: the softmax over the chosen, or over all E.
//   expert_sort    a stable counting sort of the T k slots (token t's j-th choice is slot
//                  t k + j) by expert: offsets[e], the first row of expert e, and
//                  slot_row[slot], the slot's row.
//   expert_gather  Xs[slot_row[t][j]] = X[t].
//   expert_combine Y[t] = R[t] + sum_j w[t][j] Ys[slot_row[t][j]], and its gradients
//                  dYs[slot_row[t][j]] = w[t][j] dY[t], dw[t][j] = <dY[t], Ys[slot_row[t][j]]>.
//                  With weights of one it is the gather's gradient.
//
// Every sum has an order of its own, so results do not depend on timing; no atomics.
// Choosing is bound by its T E logits for many tokens and by latency for few; sorting by
// latency (some 12 bytes a slot); gather and combine by HBM.
#include <cuda_runtime.h>

#include <climits>

#include "op_gemm.cuh"
#include "op_host.h"
#include "op_rows.cuh"

namespace pg {

constexpr int kMaxExperts = 1024;
constexpr int kMaxChoices = 32;

// ---------------------------------------------------------------- routing ---
// A logit as an unsigned number of the same order.  -0 counts as +0, a NaN above
// everything (it is chosen, and the weights say so); -inf is the lowest that occurs.
__device__ __forceinline__ uint32_t order_key(float z) {
    if (z != z) return 0xffffffffu;
    const uint32_t b = __float_as_uint(z + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
constexpr uint32_t kClosedKey = 0x007fffffu;  // order_key(-inf): this expert is not chosen
__device__ __forceinline__ float key_logit(uint32_t key) {
    if (key == 0xffffffffu) return __int_as_float(0x7fc00000);
    return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

struct RouteParams {
    int T, E, k, normalise;
    const float *logits;
    int32_t *experts;
    float *weights;
    const int32_t *experts_in;
    const float *dweights;
    float *dlogits;
    int early;  // op_begin_early
};

__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// A warp a token; lane l holds experts l, l + 32, ...  Up to four of them a lane keeps in
// order, so that a choice compares the lanes' best alone; of more it finds its best again
// every time.  Bound by instructions for many tokens (16384 tokens, eight of 128 experts,
// softmax over all: 9.9 us, without the order 11.3), by latency for few (24 tokens, eight of
// 64 experts: 1.7 us).
template <int NV>
__global__ void __launch_bounds__(128) route_kernel(const RouteParams p) {
    constexpr bool ORDERED = NV <= 4;
    op_begin_early(p.early);
    const int lane = threadIdx.x & 31;
    for (long long t = blockIdx.x * 4ll + (threadIdx.x >> 5); t < p.T; t += gridDim.x * 4ll) {
        const float *row = p.logits + t * p.E;
        float z[NV];
        uint32_t key[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = lane + 32 * i;
            z[i] = e < p.E ? row[e] : -__int_as_float(0x7f800000);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) key[i] = order_key(z[i]);
        // which of the lane's experts key[0], key[1], ... are, two bits each
        uint32_t which = 0xe4u;
        if constexpr (ORDERED) {
#pragma unroll
            for (int pass = 0; pass < NV - 1; ++pass)
#pragma unroll
                for (int i = 0; i + 1 < NV - pass; ++i)
                    if (key[i + 1] > key[i]) {  // (equal ones stay: the lower index first)
                        const uint32_t k = key[i];
                        key[i] = key[i + 1];
                        key[i + 1] = k;
                        const uint32_t two = which >> (2 * i) & 15u;
                        which ^= (two ^ (two >> 2 | two << 2 & 12u)) << (2 * i);
                    }
        }
        // choice `lane`: its expert and the key of its logit
        int mine = -1;
        uint32_t mine_key = 0u, top_key = 0u;
        for (int j = 0; j < p.k; ++j) {
            uint32_t best = key[0];
            int at = lane + 32 * static_cast<int>(which & 3u);
            if constexpr (!ORDERED) {
                at = lane;
#pragma unroll
                for (int i = 1; i < NV; ++i)
                    if (key[i] > best) {
                        best = key[i];
                        at = lane + 32 * i;
                    }
            }
            const uint32_t most = __reduce_max_sync(0xffffffffu, best);
            if (most <= kClosedKey) break;
            at = static_cast<int>(__reduce_min_sync(
                0xffffffffu, best == most ? static_cast<unsigned>(at) : 0xffffffffu));
            if (j == 0) top_key = most;
            if (lane == j) {
                mine = at;
                mine_key = most;
            }
            if constexpr (ORDERED) {
                if (lane == (at & 31)) {
#pragma unroll
                    for (int i = 0; i + 1 < NV; ++i) key[i] = key[i + 1];
                    key[NV - 1] = 0u;
                    which >>= 2;
                }
            } else {
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (at == lane + 32 * i) key[i] = 0u;
            }
        }
        const bool any = top_key != 0u;
        const float top = any ? key_logit(top_key) : 0.0f;
        const float e = mine >= 0 ? expf(key_logit(mine_key) - top) : 0.0f;
        float total = e;
        if (!p.normalise) {
            total = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (any && lane + 32 * i < p.E) total += expf(z[i] - top);
        }
        total = lanes_sum(total);
        if (lane < p.k) {
            p.experts[t * p.k + lane] = mine;
            p.weights[t * p.k + lane] = mine >= 0 ? e / total : 0.0f;
        }
    }
}

// dlogits from dweights: with w the weights and dot = sum over the chosen of w dw,
// w (dw - dot) at the chosen (softmax over the chosen), or p ([chosen] dw - dot)
// everywhere (softmax over all).  A choice outside [0, E) does not count, an expert chosen
// twice counts twice: the first of its lanes adds the others' in their order.  A warp a
// token: lane l takes experts l, l + 32, ... and choice l.  16384 tokens as above 7.0 us.
template <int NV>
__global__ void __launch_bounds__(128) route_backward_kernel(const RouteParams p) {
    op_begin_early(p.early);
    const int lane = threadIdx.x & 31;
    for (long long t = blockIdx.x * 4ll + (threadIdx.x >> 5); t < p.T; t += gridDim.x * 4ll) {
        const float *row = p.logits + t * p.E;
        float z[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = lane + 32 * i;
            z[i] = !p.normalise && e < p.E ? row[e] : -__int_as_float(0x7f800000);
        }
        int mine = -1;
        float dw = 0.0f, logit = 0.0f;
        if (lane < p.k) {
            mine = p.experts_in[t * p.k + lane];
            if (mine >= 0 && mine < p.E) {
                dw = p.dweights[t * p.k + lane];
                logit = row[mine];
            } else {
                mine = -1;
            }
        }
        // the largest of what the softmax is over; none where everything is closed
        uint32_t best = p.normalise && mine >= 0 ? order_key(logit) : 0u;
        if (!p.normalise) {
#pragma unroll
            for (int i = 0; i < NV; ++i) best = max(best, order_key(z[i]));
        }
        best = __reduce_max_sync(0xffffffffu, best);
        const bool any = best > kClosedKey;
        const float top = any ? key_logit(best) : 0.0f;
        const float e = any && mine >= 0 ? expf(logit - top) : 0.0f;
        float total = e;
        if (!p.normalise) {
            total = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                z[i] = any && lane + 32 * i < p.E ? expf(z[i] - top) : 0.0f;
                total += z[i];
            }
        }
        total = lanes_sum(total);
        const float w = any && mine >= 0 ? e / total : 0.0f;
        const float dot = lanes_sum(w * dw);
        float *out = p.dlogits + t * p.E;
        const float scale = p.normalise || !any ? 0.0f : -dot / total;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (lane + 32 * i < p.E)
                out[lane + 32 * i] = p.normalise || !any ? 0.0f : z[i] * scale;
        __syncwarp();  // the chosen ones' values replace those
        const unsigned same = __match_any_sync(0xffffffffu, mine);
        const bool owner = mine >= 0 && lane == __ffs(same) - 1;
        float all = dw;
        for (unsigned rest = __reduce_or_sync(0xffffffffu, owner ? same & (same - 1u) : 0u);
             rest != 0u; rest &= rest - 1u) {  // lanes whose expert an earlier one has
            const int l = __ffs(rest) - 1;
            const float d = __shfl_sync(0xffffffffu, dw, l);
            if (same >> l & 1u) all += d;
        }
        const float times = p.normalise ? static_cast<float>(__popc(same)) : 1.0f;
        if (owner) out[mine] = w * fmaf(-times, dot, all);
        __syncwarp();
    }
}

template <class F>
static pgemm_status with_experts(int E, F &&f) {
    using std::integral_constant;
    if (E <= 32) return f(integral_constant<int, 1>{});
    if (E <= 64) return f(integral_constant<int, 2>{});
    if (E <= 128) return f(integral_constant<int, 4>{});
    if (E <= 256) return f(integral_constant<int, 8>{});
    if (E <= 512) return f(integral_constant<int, 16>{});
    return f(integral_constant<int, 32>{});
}

static pgemm_status route_check(int T, int E, int k) {
    if (T < 0 || E < 1 || k < 1 || k > E) return PGEMM_ERR_INVALID_VALUE;
    return E > kMaxExperts || k > kMaxChoices ? PGEMM_ERR_TOO_LARGE : PGEMM_OK;
}

static dim3 route_grid(const OpDevice &dev, int T) {
    const int blocks = op_blocks(T, 4), most = dev.sm_count * 16;
    return dim3(blocks < most ? blocks : most);
}

static pgemm_status route_forward(int T, int E, int k, const float *logits, int normalise,
                                  int32_t *experts, float *weights, cudaStream_t s) {
    pgemm_status st = route_check(T, E, k);
    if (st != PGEMM_OK || T == 0) return st;
    if (!logits || !experts || !weights) return PGEMM_ERR_INVALID_VALUE;
    if (!op_aligned16(logits) || !op_aligned16(experts) || !op_aligned16(weights))
        return PGEMM_ERR_MISALIGNED;
    OpDevice dev;
    if ((st = op_device(&dev)) != PGEMM_OK) return st;
    RouteParams p{};
    p.T = T;
    p.E = E;
    p.k = k;
    p.normalise = normalise;
    p.logits = logits;
    p.experts = experts;
    p.weights = weights;
    return with_experts(E, [&](auto nv) {
        const dim3 grid = route_grid(dev, T);
        p.early = op_early(dev, grid.x);
        return launch_small(route_kernel<decltype(nv)::value>, grid, dim3(128), s, p);
    });
}

static pgemm_status route_backward(int T, int E, int k, const float *logits, int normalise,
                                   const int32_t *experts, const float *dweights, float *dlogits,
                                   cudaStream_t s) {
    pgemm_status st = route_check(T, E, k);
    if (st != PGEMM_OK || T == 0) return st;
    if (!logits || !experts || !dweights || !dlogits) return PGEMM_ERR_INVALID_VALUE;
    if (!op_aligned16(logits) || !op_aligned16(experts) || !op_aligned16(dweights) ||
        !op_aligned16(dlogits))
        return PGEMM_ERR_MISALIGNED;
    OpDevice dev;
    if ((st = op_device(&dev)) != PGEMM_OK) return st;
    RouteParams p{};
    p.T = T;
    p.E = E;
    p.k = k;
    p.normalise = normalise;
    p.logits = logits;
    p.experts_in = experts;
    p.dweights = dweights;
    p.dlogits = dlogits;
    return with_experts(E, [&](auto nv) {
        const dim3 grid = route_grid(dev, T);
        p.early = op_early(dev, grid.x);
        return launch_small(route_backward_kernel<decltype(nv)::value>, grid, dim3(128), s, p);
    });
}

// ------------------------------------------------------------------- sort ---
// A block takes `chunk` slots, a warp a run of them in order, 32 at a time: slots of one
// expert among the 32 find one another by match, and the warp's counters of each expert
// give the rest of a slot's rank.  Two passes over the slots (count, then place), with the
// counters turned into first rows in between: over the block's warps, over the blocks
// before this one, over the experts before this one.  Up to kSortOne slots one block does
// all of it; more take blocks of 1024, a launch that counts and one that places, each of
// whose blocks sums the others' counts itself, or with many blocks a launch between them.
// Bound by latency: 192 slots of 64 experts 2.7 us, 2048 6.2 (two launches 7.1), 4096 7.1
// (one block 9.8), 32768 8.6 (three launches 9.3), 65536 9.5 (two 10.9).
constexpr int kSortWarps = 32, kSortOne = 2048, kSortChunk = 1024, kSortOwnSums = 32;

struct SortParams {
    long long slots;
    int E, blocks, chunk;
    const int32_t *experts;
    int32_t *offsets, *slot_row;
    int32_t *counts;  // [blocks][E]
    int32_t *totals;  // [E], and counts summed over the blocks before: sort_scan_kernel's
};

// the counters of warp w: count[w * E + e]
__device__ __forceinline__ void sort_count(const SortParams &p, int32_t *count, int warp,
                                           int lane) {
    const int run = p.chunk / kSortWarps;
    const long long first = blockIdx.x * static_cast<long long>(p.chunk) + warp * run;
    int32_t *mine = count + warp * p.E;
#pragma unroll 1
    for (int i = 0; i < run && first + i < p.slots; i += 32) {
        const long long slot = first + i + lane;
        const int e = slot < p.slots ? p.experts[slot] : -1;
        const bool in = e >= 0 && e < p.E;
        const unsigned same = __match_any_sync(0xffffffffu, in ? e : -1);
        if (in && lane == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
    }
}

// f(block, its count of expert e) for the blocks first .. last - 1, eight on the way
// (sixteen: 32768 slots of 64 experts 10.8 us for 8.7).
template <class F>
__device__ __forceinline__ void block_counts(const SortParams &p, int e, int first, int last,
                                             F &&f) {
#pragma unroll 1
    for (int b0 = first; b0 < last; b0 += 8) {
        int n[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            n[i] = b0 + i < last ? p.counts[static_cast<long long>(b0 + i) * p.E + e] : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (b0 + i < last) f(b0 + i, n[i]);
    }
}

template <bool PLACE>
__global__ void __launch_bounds__(kSortWarps * 32) sort_kernel(const SortParams p) {
    extern __shared__ int32_t count[];  // [kSortWarps][E]
    __shared__ int32_t warp_total[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < kSortWarps * p.E; i += blockDim.x) count[i] = 0;
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();
    sort_count(p, count, warp, lane);
    __syncthreads();
    // thread e: the block's count of expert e, and where each warp's part of it begins
    const int e = threadIdx.x;
    int all = 0;
    if (e < p.E) {
#pragma unroll 8
        for (int w = 0; w < kSortWarps; ++w) {
            const int n = count[w * p.E + e];
            count[w * p.E + e] = all;
            all += n;
        }
    }
    if constexpr (!PLACE) {
        if (e < p.E) p.counts[static_cast<long long>(blockIdx.x) * p.E + e] = all;
        return;
    }
    int before = 0;  // rows of this expert in earlier blocks
    if (p.totals != nullptr && e < p.E) {
        before = p.counts[static_cast<long long>(blockIdx.x) * p.E + e];
        all = p.totals[e];
    } else if (p.blocks > 1 && e < p.E) {
        all = 0;
        block_counts(p, e, 0, p.blocks, [&](int b, int n) {
            if (b < static_cast<int>(blockIdx.x)) before += n;
            all += n;
        });
    }
    // first rows: an exclusive sum over the experts
    int sum = all;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += n;
    }
    if (lane == 31) warp_total[warp] = sum;
    __syncthreads();
    if (warp == 0) {
        int t = warp_total[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, t, d);
            if (lane >= d) t += n;
        }
        warp_total[lane] = t;
    }
    __syncthreads();
    const int first_row = sum - all + (warp > 0 ? warp_total[warp - 1] : 0);
    if (e < p.E) {
        if (blockIdx.x == 0) {
            p.offsets[e] = first_row;
            if (e == p.E - 1) p.offsets[p.E] = first_row + all;
        }
#pragma unroll 8
        for (int w = 0; w < kSortWarps; ++w) count[w * p.E + e] += first_row + before;
    }
    __syncthreads();
    const int run = p.chunk / kSortWarps;
    const long long first = blockIdx.x * static_cast<long long>(p.chunk) + warp * run;
    int32_t *mine = count + warp * p.E;
#pragma unroll 1
    for (int i = 0; i < run && first + i < p.slots; i += 32) {
        const long long slot = first + i + lane;
        const int x = slot < p.slots ? p.experts[slot] : -1;
        const bool in = x >= 0 && x < p.E;
        const unsigned same = __match_any_sync(0xffffffffu, in ? x : -1);
        const int row = in ? mine[x] + __popc(same & ((1u << lane) - 1u)) : -1;
        __syncwarp();
        if (in && lane == __ffs(same) - 1) mine[x] += __popc(same);
        __syncwarp();
        if (slot < p.slots) p.slot_row[slot] = row;
    }
}

// Each expert's counts <- their sums over the blocks before: 32 experts a block, a lane
// each, a warp every 32nd part of the blocks.
__global__ void __launch_bounds__(1024) sort_scan_kernel(const SortParams p) {
    __shared__ int32_t sums[32][33];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
    const int per = (p.blocks + 31) / 32;
    const int first = min(warp * per, p.blocks), last = min(first + per, p.blocks);
    int sum = 0;
    if (e < p.E) block_counts(p, e, first, last, [&](int, int n) { sum += n; });
    sums[warp][lane] = sum;
    __syncthreads();
    if (warp == 0) {
        int before = 0;
#pragma unroll
        for (int w = 0; w < 32; ++w) {
            const int n = sums[w][lane];
            sums[w][lane] = before;
            before += n;
        }
        if (e < p.E) p.totals[e] = before;
    }
    __syncthreads();
    if (e < p.E) {
        int before = sums[warp][lane];
        block_counts(p, e, first, last, [&](int b, int n) {
            p.counts[static_cast<long long>(b) * p.E + e] = before;
            before += n;
        });
    }
}

static pgemm_status expert_sort_run(int T, int E, int k, const int32_t *experts, int32_t *offsets,
                                    int32_t *slot_row, cudaStream_t s) {
    if (T < 0 || E < 1 || k < 1) return PGEMM_ERR_INVALID_VALUE;
    const long long slots = static_cast<long long>(T) * k;
    if (E > kMaxExperts || slots > INT_MAX) return PGEMM_ERR_TOO_LARGE;
    if (!offsets || (slots > 0 && (!experts || !slot_row))) return PGEMM_ERR_INVALID_VALUE;
    if (!op_aligned16(experts) || !op_aligned16(offsets) || !op_aligned16(slot_row))
        return PGEMM_ERR_MISALIGNED;
    OpDevice dev;
    pgemm_status st = op_device(&dev);
    if (st != PGEMM_OK) return st;
    if (slots == 0)
        return cudaMemsetAsync(offsets, 0, (static_cast<size_t>(E) + 1) * 4, s) == cudaSuccess
                   ? PGEMM_OK
                   : PGEMM_ERR_CUDA;
    static const KernelInfo place = [] {
        KernelInfo k;
        k.threads = kSortWarps * 32;
        k.smem_bytes = kSortWarps * kMaxExperts * 4;
        k.func = reinterpret_cast<const void *>(sort_kernel<true>);
        return k;
    }();
    static const KernelInfo count = [] {
        KernelInfo k = place;
        k.func = reinterpret_cast<const void *>(sort_kernel<false>);
        return k;
    }();
    if ((st = op_kernel_setup(dev, place, nullptr)) != PGEMM_OK) return st;
    SortParams p{};
    p.slots = slots;
    p.E = E;
    // (a multiple of what the warps take at once, so that they share the slots)
    p.chunk = slots <= kSortOne ? op_blocks(slots, kSortChunk) * kSortChunk : kSortChunk;
    p.blocks = op_blocks(slots, p.chunk);
    p.experts = experts;
    p.offsets = offsets;
    p.slot_row = slot_row;
    OpArena arena(dev, s);
    const bool scan = p.blocks > kSortOwnSums;
    const long long at = arena.add(p.blocks > 1 ? 4ll * p.blocks * E : 0);
    const long long totals_at = arena.add(scan ? 4ll * E : 0);
    if ((st = arena.alloc()) != PGEMM_OK) return st;
    const size_t smem = static_cast<size_t>(kSortWarps) * E * 4;
    if (p.blocks > 1) {
        p.counts = arena.at<int32_t>(at);
        if ((st = op_kernel_setup(dev, count, nullptr)) != PGEMM_OK) return st;
        st = launch_small_smem(sort_kernel<false>, dim3(p.blocks), dim3(kSortWarps * 32), smem, s,
                               p);
        if (st != PGEMM_OK) return st;
        if (scan) {
            p.totals = arena.at<int32_t>(totals_at);
            st = launch_small(sort_scan_kernel, dim3(op_blocks(E, 32)), dim3(1024), s, p);
            if (st != PGEMM_OK) return st;
        }
    }
    return launch_small_smem(sort_kernel<true>, dim3(p.blocks), dim3(kSortWarps * 32), smem, s, p);
}

// ----------------------------------------------------- gather and combine ---
// Rows as 16-byte vectors.  Where D is a multiple of 8 all rows start on one.  Elsewhere a
// row that is written, or summed into, is taken in the aligned vectors that it fills, the
// other rows' eight values are shifted out of the two vectors that hold them, and the values
// at its two ends go one to a lane.  8192 tokens, four rows of 4097 values: gather 69 us,
// combine 95, its gradient 115 (one by one 165, 136 and 189).
struct RowsParams {
    int T, k, D;
    long long rows;  // T k: a slot_row outside [0, rows) does not count
    const uint16_t *x;        // gather: X; combine: the residual; backward: dY
    const uint16_t *ys;       // combine and backward: Ys
    const int32_t *slot_row;
    const float *weights;     // nullptr: ones
    uint16_t *out;            // gather: Xs; combine: Y; backward: dYs
    float *dweights;
    int early;                // op_begin_early
};

constexpr int kRowsThreads = 256;
constexpr int kAhead = 4;  // sorted rows on the way

// Vector i of all tokens': token t, vector v of its row.
struct RowsAt {
    long long t;
    unsigned v;
    __device__ __forceinline__ RowsAt(unsigned long long i, unsigned vecs) {
        if (i >> 32 == 0) {  // (a 32-bit division where it fits)
            const unsigned q = static_cast<unsigned>(i) / vecs;
            t = q;
            v = static_cast<unsigned>(i) - q * vecs;
        } else {
            const unsigned long long q = i / vecs;
            t = static_cast<long long>(q);
            v = static_cast<unsigned>(i - q * vecs);
        }
    }
};

// Rows of whole vectors: a vector of all tokens' a thread.  Bound by HBM: 8192 tokens to four
// rows of 4096 values each, 51 us, 6.6 TB/s.
__global__ void __launch_bounds__(kRowsThreads) gather_kernel(const RowsParams p) {
    op_begin_early(p.early);
    const unsigned vecs = p.D / 8;
    const unsigned long long total = static_cast<unsigned long long>(p.T) * vecs;
    const unsigned long long step = static_cast<unsigned long long>(gridDim.x) * kRowsThreads;
    for (unsigned long long i = 1ull * blockIdx.x * kRowsThreads + threadIdx.x; i < total;
         i += step) {
        const RowsAt at(i, vecs);
        const uint4 x = reinterpret_cast<const uint4 *>(p.x)[i];
        const int32_t *to = p.slot_row + at.t * p.k;
        for (int j = 0; j < p.k; ++j) {
            const int r = to[j];
            if (r >= 0 && r < p.rows)
                reinterpret_cast<uint4 *>(p.out + static_cast<long long>(r) * p.D)[at.v] = x;
        }
    }
}

// Other rows: `per` threads a slot, a vector of its row each at a time.
__global__ void __launch_bounds__(kRowsThreads) gather_any_kernel(const RowsParams p, int per) {
    op_begin_early(p.early);
    const int groups = blockDim.x / per;
    for (long long slot = blockIdx.x * static_cast<long long>(groups) + threadIdx.x / per;
         slot < p.rows; slot += static_cast<long long>(gridDim.x) * groups) {
        const int r = p.slot_row[slot];
        if (r < 0 || r >= p.rows) continue;
        const RowSpan to(r, p.rows, p.D);
        const long long t = static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.k);
        const RowShifted from(p.x, t, p.D, to.shift);
        const RowEnds ends(to);
        const unsigned lane = threadIdx.x % per;
        uint4 *out = reinterpret_cast<uint4 *>(p.out + to.first);
        for (unsigned v = 1 + lane; v < ends.inner; v += 2 * per) {
            uint4 lo[2], hi[2];
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (v + u * per < ends.inner) {
                    lo[u] = from.at[v + u * per];
                    hi[u] = from.at[v + u * per + 1];
                }
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (v + u * per < ends.inner) out[v + u * per] = from.value(lo[u], hi[u]);
        }
        const int c = lane < 32 ? ends.col(lane) : -1;
        if (c >= 0) p.out[static_cast<long long>(r) * p.D + c] = p.x[t * p.D + c];
    }
}

// Rows of whole vectors: a vector of all tokens' a thread, and its next one's choices
// looked up while this one's rows travel.  On twice as many blocks as run at once (four an
// SM): 8192 tokens, four rows of 4096 values, 64 us, 6.3 TB/s; on five an SM 80, a block for
// every 256 vectors 69.
__global__ void __launch_bounds__(kRowsThreads) combine_flat_kernel(const RowsParams p) {
    op_begin_early(p.early);
    const unsigned vecs = p.D / 8;
    const unsigned long long total = static_cast<unsigned long long>(p.T) * vecs;
    const unsigned long long step = static_cast<unsigned long long>(gridDim.x) * kRowsThreads;
    unsigned long long i = blockIdx.x * static_cast<unsigned long long>(kRowsThreads) + threadIdx.x;
    if (i >= total) return;
    RowsAt at(i, vecs);
    int r[kAhead];
    auto look_up = [&](const RowsAt &a, int j0) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) r[j] = j0 + j < p.k ? p.slot_row[a.t * p.k + j0 + j] : -1;
    };
    look_up(at, 0);
    while (true) {
        float sum[8];
        uint4 res = make_uint4(0u, 0u, 0u, 0u);
        if (p.x) res = reinterpret_cast<const uint4 *>(p.x)[i];
#pragma unroll
        for (int c = 0; c < 8; ++c) sum[c] = 0.0f;
        const unsigned long long next = i + step;
        const RowsAt after(next < total ? next : i, vecs);
        for (int j0 = 0; j0 < p.k; j0 += kAhead) {
            uint4 y[kAhead];
            bool in[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                in[j] = r[j] >= 0 && r[j] < p.rows;
                if (in[j])
                    y[j] = reinterpret_cast<const uint4 *>(
                        p.ys + static_cast<long long>(r[j]) * p.D)[at.v];
            }
            if (j0 + kAhead < p.k)
                look_up(at, j0 + kAhead);
            else
                look_up(after, 0);
            const float *w = p.weights ? p.weights + at.t * p.k + j0 : nullptr;
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (in[j]) {
                    const float wj = w ? w[j] : 1.0f;
                    float f[8];
                    unpack8(y[j], f);
#pragma unroll
                    for (int c = 0; c < 8; ++c) sum[c] = fmaf(wj, f[c], sum[c]);
                }
        }
        float f[8];
        unpack8(res, f);
#pragma unroll
        for (int c = 0; c < 8; ++c) sum[c] += f[c];
        reinterpret_cast<uint4 *>(p.out)[i] = pack8(sum);
        if (next >= total) break;
        i = next;
        at = after;
    }
}

// Other rows: `per` threads a token, so that where its rows lie is worked out once for all of
// a thread's vectors; U of them, of AHEAD rows, on the way.  Bound by latency, so few of them
// and four blocks an SM (8192 tokens, one row of 2047 values: 19 us with two vectors on the way,
// 30 with four on three blocks; two rows 34, with two vectors 39).
template <int AHEAD, int U>
__global__ void __launch_bounds__(kRowsThreads, 4) combine_any_kernel(const RowsParams p, int per) {
    op_begin_early(p.early);
    const int groups = blockDim.x / per;
    for (long long t = blockIdx.x * static_cast<long long>(groups) + threadIdx.x / per; t < p.T;
         t += static_cast<long long>(gridDim.x) * groups) {
        const int32_t *slots = p.slot_row + t * p.k;
        const float *w = p.weights ? p.weights + t * p.k : nullptr;
        const RowSpan to(t, p.T, p.D);
        const RowEnds ends(to);
        const unsigned lane = threadIdx.x % per;
        RowShifted row[AHEAD];
        bool in[AHEAD];
        float weight[AHEAD];
        auto choices = [&](int j0) {
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                const int r = j0 + j < p.k ? slots[j0 + j] : -1;
                weight[j] = w && j0 + j < p.k ? w[j0 + j] : 1.0f;
                in[j] = r >= 0 && r < p.rows;
                if (in[j]) row[j] = RowShifted(p.ys, r, p.D, to.shift);
            }
        };
        if (p.k <= AHEAD) choices(0);
        const uint4 *residual = reinterpret_cast<const uint4 *>(p.x + to.first);
        uint4 *out = reinterpret_cast<uint4 *>(p.out + to.first);
        for (unsigned v0 = 1 + lane; v0 < ends.inner; v0 += U * per) {
            float sum[U][8];
            uint4 res[U];
            bool has[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                has[u] = v0 + u * per < ends.inner;
                res[u] = make_uint4(0u, 0u, 0u, 0u);
                if (p.x && has[u]) res[u] = residual[v0 + u * per];
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[u][i] = 0.0f;
            }
            for (int j0 = 0; j0 < p.k; j0 += AHEAD) {
                if (p.k > AHEAD) choices(j0);
                uint4 lo[U][AHEAD], hi[U][AHEAD];
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int j = 0; j < AHEAD; ++j)
                        if (in[j] && has[u]) {
                            lo[u][j] = row[j].at[v0 + u * per];
                            hi[u][j] = row[j].at[v0 + u * per + 1];
                        }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int j = 0; j < AHEAD; ++j)
                        if (in[j]) {
                            float f[8];
                            unpack8(row[j].value(lo[u][j], hi[u][j]), f);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                sum[u][i] = fmaf(weight[j], f[i], sum[u][i]);
                        }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float f[8];
                unpack8(res[u], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[u][i] += f[i];
                if (has[u]) out[v0 + u * per] = pack8(sum[u]);
            }
        }
        const int c = lane < 32 ? ends.col(lane) : -1;
        if (c >= 0) {
            float sum = 0.0f;
            for (int j = 0; j < p.k; ++j) {
                const int r = slots[j];
                if (r >= 0 && r < p.rows)
                    sum = fmaf(w ? w[j] : 1.0f,
                               bf16_at(p.ys + static_cast<long long>(r) * p.D + c), sum);
            }
            if (p.x) sum += bf16_at(p.x + t * p.D + c);
            p.out[t * p.D + c] = static_cast<uint16_t>(pack_bf16(sum, 0.0f) & 0xffffu);
        }
    }
}

// PER threads a token: a warp or more.  The slots' dot products of AHEAD choices at a time,
// over the lanes' columns, then over the lanes, then over the group's warps.  Each slot's row
// in vectors of its own (ALIGNED: all rows' lie alike).  Bound by HBM: 8192 tokens, four rows
// of 4096 values, 90 us, 6.7 TB/s.
template <bool ALIGNED, int PER>
__global__ void __launch_bounds__(kRowsThreads, ALIGNED ? 0 : 4)
    combine_backward_kernel(const RowsParams p) {
    constexpr int GROUPS = kRowsThreads / PER, WARPS = PER / 32;
    constexpr int AHEAD = ALIGNED ? kAhead : kAhead / 2;
    __shared__ float part[GROUPS][WARPS][AHEAD];
    op_begin_early(p.early);
    const int group = threadIdx.x / PER, lane = threadIdx.x % PER;
    // (every group of a block makes as many rounds: they share the barriers)
    for (long long t0 = blockIdx.x * static_cast<long long>(GROUPS); t0 < p.T;
         t0 += static_cast<long long>(gridDim.x) * GROUPS) {
        const long long t = t0 + group;
        const bool have = t < p.T;
        for (int j0 = 0; j0 < p.k; j0 += AHEAD) {
            int row[AHEAD];
            float w[AHEAD], dot[AHEAD];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                int r = -1;
                w[j] = 1.0f;
                dot[j] = 0.0f;
                if (have && j0 + j < p.k) {
                    r = p.slot_row[t * p.k + j0 + j];
                    if (p.weights) w[j] = p.weights[t * p.k + j0 + j];
                }
                row[j] = r < p.rows ? r : -1;
            }
            // eight elements of slot j's row
            auto work = [&](int j, const uint4 &x, const uint4 &y, uint4 *out) {
                float d[8];
                unpack8(x, d);
                if (p.dweights) {
                    float f[8];
                    unpack8(y, f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) dot[j] = fmaf(d[i], f[i], dot[j]);
                }
                if (p.out) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) d[i] *= w[j];
                    *out = pack8(d);
                }
            };
            if constexpr (ALIGNED) {
                const unsigned vecs = p.D / 8;  // (unsigned: a step may pass 2^31)
                for (unsigned v = lane; have && v < vecs; v += PER) {
                    const uint4 x = reinterpret_cast<const uint4 *>(p.x + t * p.D)[v];
                    uint4 y[AHEAD];
                    auto at = [&](int j) { return static_cast<long long>(row[j]) * p.D + 8ll * v; };
#pragma unroll
                    for (int j = 0; j < AHEAD; ++j)
                        if (row[j] >= 0 && p.dweights)
                            y[j] = *reinterpret_cast<const uint4 *>(p.ys + at(j));
#pragma unroll
                    for (int j = 0; j < AHEAD; ++j)
                        if (row[j] >= 0) work(j, x, y[j], reinterpret_cast<uint4 *>(p.out + at(j)));
                }
            } else {
                long long first[AHEAD];
                unsigned inner[AHEAD];
                RowShifted token[AHEAD];  // in slot j's vectors
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) {
                    inner[j] = 0;
                    if (row[j] < 0) continue;
                    const RowSpan span(row[j], p.rows, p.D);
                    const RowEnds ends(span);
                    first[j] = span.first;
                    inner[j] = ends.inner;
                    token[j] = RowShifted(p.x, t, p.D, span.shift);
                    const int c = lane < 32 ? ends.col(lane) : -1;
                    if (c < 0) continue;
                    const long long at = static_cast<long long>(row[j]) * p.D + c;
                    const float d = bf16_at(p.x + t * p.D + c);
                    if (p.dweights) dot[j] = d * bf16_at(p.ys + at);
                    if (p.out)
                        p.out[at] = static_cast<uint16_t>(pack_bf16(w[j] * d, 0.0f) & 0xffffu);
                }
                unsigned most = 0;
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) most = max(most, inner[j]);
                for (unsigned v = 1 + lane; v < most; v += PER) {
                    uint4 lo[AHEAD], hi[AHEAD], y[AHEAD];
#pragma unroll
                    for (int j = 0; j < AHEAD; ++j)
                        if (v < inner[j]) {
                            lo[j] = token[j].at[v];
                            hi[j] = token[j].at[v + 1];
                            if (p.dweights)
                                y[j] = reinterpret_cast<const uint4 *>(p.ys + first[j])[v];
                        }
#pragma unroll
                    for (int j = 0; j < AHEAD; ++j)
                        if (v < inner[j])
                            work(j, token[j].value(lo[j], hi[j]), y[j],
                                 reinterpret_cast<uint4 *>(p.out + first[j]) + v);
                }
            }
            if (!p.dweights) continue;
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) dot[j] = lanes_sum(dot[j]);
            if constexpr (WARPS > 1) {
                if ((lane & 31) == 0) {
#pragma unroll
                    for (int j = 0; j < AHEAD; ++j) part[group][lane >> 5][j] = dot[j];
                }
                __syncthreads();
                if (lane < AHEAD && have && j0 + lane < p.k) {
                    float s = 0.0f;
#pragma unroll
                    for (int i = 0; i < WARPS; ++i) s += part[group][i][lane];
                    p.dweights[t * p.k + j0 + lane] = s;
                }
                __syncthreads();
            } else if (have && lane == 0) {
#pragma unroll
                for (int j = 0; j < AHEAD; ++j)
                    if (j0 + j < p.k) p.dweights[t * p.k + j0 + j] = dot[j];
            }
        }
    }
}

// vectors of a row at most
static int rows_vecs(int D) {
    return static_cast<int>((static_cast<long long>(D) + (D % 8 == 0 ? 0 : 14)) / 8);
}
// Threads of a row, 32 to 256: no more than it has vectors, and no more than it takes to fill
// the SMs, so that looking up where a row lies is paid for by as many of its vectors as can be
// (8192 tokens, two rows of 2047 values, gradients: 32 us with 32 threads a token, 35 with 64).
static int rows_per(const OpDevice &dev, long long rows, int D) {
    const int vecs = rows_vecs(D);
    int per = 32;
    while (per < kRowsThreads && per < vecs && rows * per < 1024ll * dev.sm_count) per *= 2;
    return per;
}
// a thread for each vector, D a multiple of 8
static dim3 vectors_grid(int T, int D) {
    const long long blocks =
        (static_cast<long long>(T) * (D / 8) + kRowsThreads - 1) / kRowsThreads;
    return dim3(static_cast<unsigned>(blocks < INT_MAX ? blocks : INT_MAX));
}

static pgemm_status rows_check(int T, int k, int D) {
    if (T < 0 || k < 1 || D < 0) return PGEMM_ERR_INVALID_VALUE;
    return static_cast<long long>(T) * k > INT_MAX ? PGEMM_ERR_TOO_LARGE : PGEMM_OK;
}

static RowsParams rows_params(int T, int k, int D, const int32_t *slot_row) {
    RowsParams p{};
    p.T = T;
    p.k = k;
    p.D = D;
    p.rows = static_cast<long long>(T) * k;
    p.slot_row = slot_row;
    return p;
}

static pgemm_status gather_run(int T, int k, int D, const uint16_t *X, const int32_t *slot_row,
                               uint16_t *Xs, cudaStream_t s) {
    pgemm_status st = rows_check(T, k, D);
    if (st != PGEMM_OK || T == 0 || D == 0) return st;
    if (!X || !slot_row || !Xs) return PGEMM_ERR_INVALID_VALUE;
    if (!op_aligned16(X) || !op_aligned16(slot_row) || !op_aligned16(Xs))
        return PGEMM_ERR_MISALIGNED;
    OpDevice dev;
    if ((st = op_device(&dev)) != PGEMM_OK) return st;
    RowsParams p = rows_params(T, k, D, slot_row);
    p.x = X;
    p.out = Xs;
    if (D % 8 == 0) {
        const dim3 grid = vectors_grid(T, D);
        p.early = op_early(dev, grid.x);
        return launch_small(gather_kernel, grid, dim3(kRowsThreads), s, p);
    }
    const int per = rows_per(dev, p.rows, D);
    const dim3 grid(op_blocks(p.rows, kRowsThreads / per));
    p.early = op_early(dev, grid.x);
    return launch_small(gather_any_kernel, grid, dim3(kRowsThreads), s, p, per);
}

static pgemm_status combine_run(int T, int k, int D, const uint16_t *Ys, const int32_t *slot_row,
                                const float *weights, const uint16_t *residual, uint16_t *Y,
                                cudaStream_t s) {
    pgemm_status st = rows_check(T, k, D);
    if (st != PGEMM_OK || T == 0 || D == 0) return st;
    if (!Ys || !slot_row || !Y) return PGEMM_ERR_INVALID_VALUE;
    if (!op_aligned16(Ys) || !op_aligned16(slot_row) || !op_aligned16(weights) ||
        !op_aligned16(residual) || !op_aligned16(Y))
        return PGEMM_ERR_MISALIGNED;
    OpDevice dev;
    if ((st = op_device(&dev)) != PGEMM_OK) return st;
    RowsParams p = rows_params(T, k, D, slot_row);
    p.x = residual;
    p.ys = Ys;
    p.weights = weights;
    p.out = Y;
    if (D % 8 == 0) {
        const unsigned all = vectors_grid(T, D).x, most = 8u * dev.sm_count;
        p.early = op_early(dev, all);
        return launch_small(combine_flat_kernel, dim3(all < most ? all : most),
                            dim3(kRowsThreads), s, p);
    }
    const int per = rows_per(dev, T, D);
    const dim3 grid(op_blocks(T, kRowsThreads / per));
    p.early = op_early(dev, grid.x);
    auto go = [&](auto kernel) {
        return launch_small(kernel, grid, dim3(kRowsThreads), s, p, per);
    };
    return k == 1 ? go(combine_any_kernel<1, 2>) : go(combine_any_kernel<2, 1>);
}

static pgemm_status combine_backward_run(int T, int k, int D, const uint16_t *Ys,
                                         const int32_t *slot_row, const float *weights,
                                         const uint16_t *dY, uint16_t *dYs, float *dweights,
                                         cudaStream_t s) {
    pgemm_status st = rows_check(T, k, D);
    if (st != PGEMM_OK || T == 0 || (!dYs && !dweights)) return st;
    if (!slot_row || (D > 0 && (!dY || (dweights && !Ys)))) return PGEMM_ERR_INVALID_VALUE;
    if (!op_aligned16(Ys) || !op_aligned16(slot_row) || !op_aligned16(weights) ||
        !op_aligned16(dY) || !op_aligned16(dYs) || !op_aligned16(dweights))
        return PGEMM_ERR_MISALIGNED;
    OpDevice dev;
    if ((st = op_device(&dev)) != PGEMM_OK) return st;
    RowsParams p = rows_params(T, k, D, slot_row);
    p.x = dY;
    p.ys = Ys;
    p.weights = weights;
    p.out = dYs;
    p.dweights = dweights;
    auto go = [&](auto aligned, auto n) {
        constexpr int PER = decltype(n)::value;
        const int blocks = op_blocks(T, kRowsThreads / PER), most = dev.sm_count * 16;
        const dim3 grid(blocks < most ? blocks : most);
        p.early = op_early(dev, grid.x);
        return launch_small(combine_backward_kernel<decltype(aligned)::value, PER>, grid,
                            dim3(kRowsThreads), s, p);
    };
    auto pick = [&](auto aligned) {
        using std::integral_constant;
        // (whole vectors of long rows have enough on the way with a block a token: 8192
        // tokens, four rows of 4096 values, 90 us, by the rule 94; of 1024 30 and 24)
        const int per = rows_per(dev, decltype(aligned)::value && D > 2048 ? 1 : T, D);
        if (per == 32) return go(aligned, integral_constant<int, 32>{});
        if (per == 64) return go(aligned, integral_constant<int, 64>{});
        if (per == 128) return go(aligned, integral_constant<int, 128>{});
        return go(aligned, integral_constant<int, 256>{});
    };
    return D % 8 == 0 ? pick(std::true_type{}) : pick(std::false_type{});
}

}  // namespace pg

extern "C" {

pgemm_status route_topk(int T, int E, int k, const float *logits, int normalise, int32_t *experts,
                        float *weights, pgemm_stream_t stream) {
    return pg::op_guard([&] {
        return pg::route_forward(T, E, k, logits, normalise, experts, weights, stream);
    });
}

pgemm_status route_topk_backward(int T, int E, int k, const float *logits, int normalise,
                                 const int32_t *experts, const float *dweights, float *dlogits,
                                 pgemm_stream_t stream) {
    return pg::op_guard([&] {
        return pg::route_backward(T, E, k, logits, normalise, experts, dweights, dlogits, stream);
    });
}

pgemm_status expert_sort(int T, int E, int k, const int32_t *experts, int32_t *offsets,
                         int32_t *slot_row, pgemm_stream_t stream) {
    return pg::op_guard(
        [&] { return pg::expert_sort_run(T, E, k, experts, offsets, slot_row, stream); });
}

pgemm_status expert_gather_bf16(int T, int k, int D, const uint16_t *X, const int32_t *slot_row,
                                uint16_t *Xs, pgemm_stream_t stream) {
    return pg::op_guard([&] { return pg::gather_run(T, k, D, X, slot_row, Xs, stream); });
}

pgemm_status expert_combine_bf16(int T, int k, int D, const uint16_t *Ys, const int32_t *slot_row,
                                 const float *weights, const uint16_t *residual, uint16_t *Y,
                                 pgemm_stream_t stream) {
    return pg::op_guard([&] {
        return pg::combine_run(T, k, D, Ys, slot_row, weights, residual, Y, stream);
    });
}

pgemm_status expert_combine_bf16_backward(int T, int k, int D, const uint16_t *Ys,
                                          const int32_t *slot_row, const float *weights,
                                          const uint16_t *dY, uint16_t *dYs, float *dweights,
                                          pgemm_stream_t stream) {
    return pg::op_guard([&] {
        return pg::combine_backward_run(T, k, D, Ys, slot_row, weights, dY, dYs, dweights, stream);
    });
}

}  // extern "C"
