// Rows of a row-major bf16 matrix of any width as aligned 16-byte vectors of the flat matrix
// (its base is 16-byte aligned), masked at a row's two ends.
#pragma once

#include "op_gemm.cuh"

namespace pg {

// One of `rows` rows: vector v covers its elements 8 v - shift .. 8 v - shift + 7.
struct RowSpan {
    long long first;  // flat index of vector 0's first element (a multiple of 8)
    long long end;    // elements of the matrix
    int shift, vecs, D;
    __device__ __forceinline__ RowSpan() {}
    __device__ __forceinline__ RowSpan(long long row, long long rows, int D_) : D(D_) {
        const long long at = row * D_;
        end = rows * D_;
        shift = static_cast<int>(at & 7);
        first = at - shift;
        vecs = static_cast<int>((static_cast<unsigned>(D_) + shift + 7u) >> 3);
    }
    // (unsigned: rows may have up to 2^31 - 1 elements)
    __device__ __forceinline__ int col(int v) const {
        return static_cast<int>(8u * static_cast<unsigned>(v) - shift);
    }
    __device__ __forceinline__ bool whole(int v) const {
        const int c = col(v);
        return c >= 0 && D - c >= 8;
    }
    // whether column c + i is the row's (c >= -7)
    __device__ __forceinline__ bool has(int c, int i) const {
        return static_cast<unsigned>(c) + i < static_cast<unsigned>(D);
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

// The aligned vector that holds vector v of a row: at the row's ends the neighbours'
// elements come with it (row_mask drops them, when the vector is used and not here, where
// that would wait for it); only the matrix's last vector may pass its end.
__device__ __forceinline__ uint4 row_load(const uint16_t *p, const RowSpan &r, int v) {
    const long long from = r.first + 8ll * v;
    const uint16_t *at = p + from;
    if (from + 8 <= r.end) return *reinterpret_cast<const uint4 *>(at);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (from + i < r.end) w[i / 2] |= static_cast<uint32_t>(at[i]) << (i % 2 * 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// Zeros where the row is not.
__device__ __forceinline__ void row_mask(uint4 &x, const RowSpan &r, int v) {
    if (r.whole(v)) return;
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (!r.has(r.col(v), i)) w[i / 2] &= i % 2 ? 0xffffu : 0xffff0000u;
    }
    x = make_uint4(w[0], w[1], w[2], w[3]);
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
        if (r.has(r.col(v), i)) at[i] = static_cast<uint16_t>(w[i / 2] >> (i % 2 * 16));
    }
}

// A row seen in another row's vectors 1 .. vecs - 3 (RowEnds): its eight elements from column
// 8 v - shift on are shifted out of the two aligned vectors that hold them, which lie within
// the matrix there.
struct RowShifted {
    const uint4 *at;
    uint32_t off;
    __device__ __forceinline__ RowShifted() {}
    __device__ __forceinline__ RowShifted(const uint16_t *p, long long row, int D, int shift) {
        const long long begin = row * D - shift;
        at = reinterpret_cast<const uint4 *>(p + (begin & ~7ll));
        off = static_cast<uint32_t>(begin & 7) * 2u;
    }
    __device__ __forceinline__ uint4 value(const uint4 &lo, const uint4 &hi) const {
        uint32_t w[4];
        shift16(lo, hi, off, w);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// The columns of a row outside its vectors 1 .. vecs - 3: 24 at most, one for each lane.
struct RowEnds {
    unsigned inner;  // the vector after the last inner one
    int head, tail, D;
    __device__ __forceinline__ RowEnds(const RowSpan &r) : D(r.D) {
        inner = r.vecs > 2 ? r.vecs - 2 : 0;
        head = min(D, 8 - r.shift);
        tail = max(head, r.vecs > 2 ? r.col(r.vecs - 2) : 0);
    }
    __device__ __forceinline__ int col(int lane) const {  // -1: none
        const unsigned c = lane < head ? lane : static_cast<unsigned>(tail) + (lane - head);
        return c < static_cast<unsigned>(D) ? static_cast<int>(c) : -1;
    }
};

__device__ __forceinline__ float bf16_at(const uint16_t *p) {
    return __uint_as_float(static_cast<uint32_t>(*p) << 16);
}

}  // namespace pg
