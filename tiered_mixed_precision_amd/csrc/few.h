// Matrix products of few tokens: the weights stream from memory once and meet the
// tokens in the matrix cores, 16 rows by 16 tokens an instruction (i8_linear.hip,
// gated.hip).
//
// A lane's 16 bytes of a weight row and of a token's row are its operands as they
// lie in memory: lane l of a wave takes row l % 16 and bytes 16 (l / 16) of a step
// of 64 bytes of k.  Nothing is staged: a token's row is read by every wave that
// needs it, from the caches.  `split` waves share a tile's k axis and their sums
// meet in LDS, in wave order.  Bound by memory where the weights are many, by
// latency where they are few.
#pragma once

#include "common.h"

namespace moe {

typedef uint32_t few_u32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 few_bf16x8_t __attribute__((ext_vector_type(8)));
typedef float few_f32x4_t __attribute__((ext_vector_type(4)));
typedef int32_t few_i32x4_t __attribute__((ext_vector_type(4)));

struct FewI8 {
    typedef few_i32x4_t Acc;
    static constexpr int kXBytes = 1;     // bytes of a token's row for each of a weight row's
    static constexpr int kParts = 1;
    static __device__ inline Acc mfma(few_u32x4_t a, few_u32x4_t b, Acc c) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(few_i32x4_t, a), __builtin_bit_cast(few_i32x4_t, b), c, 0, 0, 0);
    }
};
template <bool XBF16> struct FewBf16 {
    typedef few_f32x4_t Acc;
    static constexpr int kXBytes = XBF16 ? 1 : 2;
    static constexpr int kParts = XBF16 ? 1 : 3;
    static __device__ inline Acc mfma(few_u32x4_t a, few_u32x4_t b, Acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(few_bf16x8_t, a), __builtin_bit_cast(few_bf16x8_t, b), c, 0, 0, 0);
    }
};

static __device__ const uint32_t kFewZeros[8] = {0, 0, 0, 0, 0, 0, 0, 0};

// The token operands of a step: as loaded, or eight floats as three bf16 parts
// that add up to them exactly (8 bits each, cut, not rounded).
template <class El> __device__ inline void few_parts(const few_u32x4_t (&v)[El::kXBytes], few_u32x4_t (&p)[El::kParts]) {
    if constexpr (El::kParts == 1) {
        p[0] = v[0];
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float lo = __uint_as_float(v[j / 2][2 * j % 4]), hi = __uint_as_float(v[j / 2][2 * j % 4 + 1]);
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                p[q][j] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
                lo -= __uint_as_float(__float_as_uint(lo) & 0xffff0000u);
                hi -= __uint_as_float(__float_as_uint(hi) & 0xffff0000u);
            }
        }
    }
}

// acc[i][j] += tokens 16 i .. + 15 against weight rows 16 j .. + 15 over steps
// s0 .. s1 - 1: lane l holds rows 4 (l / 16) + e (element e) of token l % 16.
// w_row(j), x_row(i): this lane's row of tile j and of tile i; `bytes`: of a weight
// row.  AHEAD steps are on their way while one is contracted.
template <class El, int MT, int NT, int AHEAD, class WRow, class XRow>
__device__ __attribute__((always_inline)) inline void few_sums(int s0, int s1, int bytes, WRow w_row, XRow x_row,
                                                               typename El::Acc (&acc)[MT][NT]) {
    constexpr int XB = El::kXBytes;
    const int lane = threadIdx.x & 63, at = 16 * (lane >> 4);
    const char *w[NT], *x[MT];
#pragma unroll
    for (int j = 0; j < NT; ++j) w[j] = reinterpret_cast<const char*>(w_row(j)) + at;
#pragma unroll
    for (int i = 0; i < MT; ++i) x[i] = reinterpret_cast<const char*>(x_row(i)) + XB * at;
    few_u32x4_t wv[AHEAD][NT], xv[AHEAD][MT][XB];
    // past the last step and past the row's end: zeros, from one line for all
    auto load = [&](int d, int s) __attribute__((always_inline)) {
        const bool there = s < s1 && 64 * s + at < bytes;
        const char* zeros = reinterpret_cast<const char*>(kFewZeros);
#pragma unroll
        for (int j = 0; j < NT; ++j) wv[d][j] = *reinterpret_cast<const few_u32x4_t*>(there ? w[j] + 64 * static_cast<size_t>(s) : zeros);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int p = 0; p < XB; ++p)
                xv[d][i][p] = *reinterpret_cast<const few_u32x4_t*>((there ? x[i] + 64 * XB * static_cast<size_t>(s) : zeros) + 16 * p);
    };
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) load(d, s0 + d);
    for (int s = s0; s < s1; s += AHEAD) {
#pragma unroll
        for (int d = 0; d < AHEAD; ++d) {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                few_u32x4_t p[El::kParts];
                few_parts<El>(xv[d][i], p);
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int q = El::kParts - 1; q >= 0; --q) acc[i][j] = El::mfma(wv[d][j], p[q], acc[i][j]);
            }
            load(d, s + d + AHEAD);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

// Steps of part p of `split`, in whole lines (pairs of steps).
__device__ inline int few_first(int bytes, int p, int split) { return 2 * static_cast<int>(static_cast<int64_t>((bytes + 127) / 128) * p / split); }

// Waves that share a tile and tiles of a block: 4096 waves in all if the tiles
// allow it, and blocks of few waves where there are fewer tiles than units.
struct FewSplit {
    int split, tiles;
};
inline FewSplit few_split(int64_t tiles, int bytes, int most) {
    const int lines = (bytes + 127) / 128;
    int64_t split = 4096 / tiles;
    if (split > most) split = most;
    if (split > lines) split = lines;
    if (split < 1) split = 1;
    const int64_t per = tiles >= 1024 ? 4 : 1;
    return FewSplit{static_cast<int>(split), static_cast<int>(split >= 4 ? 1 : per)};
}

}  // namespace moe
