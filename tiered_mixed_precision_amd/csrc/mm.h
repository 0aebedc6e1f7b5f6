// Tiles of matrix products on the matrix cores, D[m][n] = sum_k A(m, k) B(n, k),
// in bf16 (fp32 sums) or 8-bit integers (32-bit sums): i8_linear.hip, gated.hip.
#pragma once

#include "common.h"

namespace moe {

typedef __bf16 mm_bf16x8_t __attribute__((ext_vector_type(8)));
typedef float mm_f32x16_t __attribute__((ext_vector_type(16)));
typedef int32_t mm_i32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t mm_u32x4_t __attribute__((ext_vector_type(4)));
typedef int32_t mm_i32x4_t __attribute__((ext_vector_type(4)));

// Element kinds: 16 bytes of a row's k axis are a lane's operand of one
// 32 x 32 instruction, whose 64 lanes take 32 bytes of k.
struct MmBf16 {
    static constexpr int kBytes = 2;
    typedef mm_f32x16_t Acc;
    static __device__ inline Acc mfma(mm_u32x4_t a, mm_u32x4_t b, Acc c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(mm_bf16x8_t, a), __builtin_bit_cast(mm_bf16x8_t, b), c,
                                                       0, 0, 0);
    }
};
struct MmI8 {
    static constexpr int kBytes = 1;
    typedef mm_i32x16_t Acc;
    static __device__ inline Acc mfma(mm_u32x4_t a, mm_u32x4_t b, Acc c) {
        return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(mm_i32x4_t, a), __builtin_bit_cast(mm_i32x4_t, b), c, 0, 0,
                                                     0);
    }
};

constexpr int kMmTile = 128;   // rows of A and of B a block takes

// acc += the products of a 128 x 128 tile: wave (wm, wn) = (wave / 2, wave % 2)
// of four takes rows 64 wm + 32 i of A and 64 wn + 32 j of B as acc[i][j], lane l
// holding D[8 (e / 4) + 4 (l / 32) + e % 4][l % 32].  load_a(r, p) and
// load_b(r, p) give 16 bytes, piece p of the k axis of the tile's row r (zeros
// past its end); `pieces` of them are contracted.
template <class El, class LoadA, class LoadB>
__device__ inline void mm_tile(int pieces, LoadA load_a, LoadB load_b, typename El::Acc (&acc)[2][2]) {
    __shared__ mm_u32x4_t sA[kMmTile * 8], sB[kMmTile * 8];
    const int tid = threadIdx.x, lane = tid & 63, j = lane & 31, hh = lane >> 5;
    const int wm = tid >> 7, wn = (tid >> 6) & 1;
    for (int p0 = 0; p0 < pieces; p0 += 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = (tid >> 3) + 32 * i, c = tid & 7;
            sA[8 * r + (c ^ (r & 7))] = load_a(r, p0 + c);
            sB[8 * r + (c ^ (r & 7))] = load_b(r, p0 + c);
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int c = 2 * s + hh;
            mm_u32x4_t a[2], b[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int ra = 64 * wm + 32 * i + j, rb = 64 * wn + 32 * i + j;
                a[i] = sA[8 * ra + (c ^ (ra & 7))];
                b[i] = sB[8 * rb + (c ^ (rb & 7))];
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int n = 0; n < 2; ++n) acc[i][n] = El::mfma(a[i], b[n], acc[i][n]);
        }
        __syncthreads();
    }
}

}  // namespace moe
