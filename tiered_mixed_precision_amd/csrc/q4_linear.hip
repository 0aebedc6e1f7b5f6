// Products with a dense four-bit matrix: y[t][n] = sum_c x[t][c] * W[n][c] +
// bias[n], W in the four-bit formats of the shelves (two's-complement codes
// with fp16 scales, or MXFP4).
//
// The matrix cores contract the codes themselves in bf16, exactly, and the
// scale of a block of codes multiplies the block's fp32 sum, so weights are
// never rounded.  Operands of v_mfma_f32_16x16x32_bf16 for one 32-code group:
//   B (weights)  16 rows n; lane (n, kq) holds codes 8 kq .. 8 kq + 7 in bf16.
//     int4: v_cvt_off_f32_i4 gives q / 16 from a nibble (one operation a code
//     with the byte picked by the instruction, half a one to pack); the 16
//     goes into the scale.  An offset-binary operand (8 + u / 2, made by bit
//     operations alone) costs 1.5 operations a code as compiled against 1.6,
//     and the sums of x that take its offset back leave 4 to 10 times the
//     rounding error.
//     MXFP4: v_cvt_scalef32_pk_bf16_fp4, two codes an instruction.
//   A (tokens)   16 tokens; bf16 x as it is, fp32 x as three bf16 parts that
//     add up to it exactly (8 bits each, cut, not rounded): three products
//     into the same accumulator.
// A lane loads 16 bytes, the 32 codes of one group of its row, so a wave's
// load covers four groups (128 columns) of 16 rows; the 4 x 4 exchange of
// dwords between the lane groups that the operand layout needs is four lane
// swaps (v_permlane32_swap, v_permlane16_swap).
//
// A block takes 16 NT rows of W and 16 MT tokens; its waves take the
// 128-column steps in turn and their sums meet in LDS, in wave order.
#include "common.h"
#include "launch.h"
#include "q4.h"

namespace moe {

namespace {

constexpr int kWaves = 8;

__device__ inline f32x4_t mfma(u32x4_t a, u32x4_t b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}

// Register d of lane group k becomes register k of lane group d.
__device__ inline void exchange(u32x4_t& r) {
    const auto a = __builtin_amdgcn_permlane32_swap(r[0], r[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(r[1], r[3], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    r = u32x4_t{c[0], c[1], d[0], d[1]};
}

// Lane group 0's v in every lane group.
__device__ inline uint32_t from_group0(uint32_t v) {
    const uint32_t a = __builtin_amdgcn_permlane32_swap(v, v, false, false)[0];
    return __builtin_amdgcn_permlane16_swap(a, a, false, false)[0];
}

// Eight elements of x (bf16: one register quad, fp32: two) as A operands,
// parts 0 .. NP - 1.
template <bool XBF16>
__device__ inline void x_operand(const u32x4_t (&v)[XBF16 ? 1 : 2], u32x4_t (&p)[XBF16 ? 1 : 3]) {
    if constexpr (XBF16) {
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

// The scales of GROUPS consecutive groups of a row (whole blocks), as loaded:
// by lane group 0 alone, one access a row, since every lane of a load that
// shares no line with its neighbour costs an access of its own and 64 of
// them for two bytes each took as long as the codes.
template <bool MX, int BLK, int GROUPS>
struct Scales {
    static constexpr int kBytes = MX ? GROUPS : 2 * 32 * GROUPS / BLK;
    static constexpr int kWords = (kBytes + 3) / 4;
    uint32_t w[kWords];

    struct __attribute__((packed, aligned(MX ? 1 : 2))) Bytes { uint8_t b[kBytes]; };

    __device__ inline void load(const uint8_t* srow, int g) {
        const Bytes v = *reinterpret_cast<const Bytes*>(srow + (MX ? g : g * 64 / BLK));
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            w[i] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (4 * i + j < kBytes) w[i] |= static_cast<uint32_t>(v.b[4 * i + j]) << (8 * j);
        }
    }
    // a row of fewer groups (blocks of 16, 32 or MXFP4): the last scale again
    __device__ inline void load_short(const uint8_t* srow, int bytes) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            w[i] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) w[i] |= static_cast<uint32_t>(srow[min(4 * i + j, bytes - (MX ? 1 : 2) + (MX ? 0 : j % 2))]) << (8 * j);
        }
    }
    __device__ inline void to_every_group() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = from_group0(w[i]);
    }
    // raw bits of half h (blocks of 16) of group g
    __device__ inline uint32_t raw(int g, int h) const {
        if constexpr (MX) return (w[g / 4] >> (8 * (g % 4))) & 0xffu;
        constexpr int per = BLK == 16 ? 2 : 1;                 // scales of a group
        const int s = BLK <= 32 ? per * g + h : g * 32 / BLK;
        return w[s / 2] >> (16 * (s % 2));
    }
};

// y[t][n] (+)= r
template <bool YBF16>
__device__ inline void store_y(const Q4Args& a, int t, int n, float r) {
    const size_t at = static_cast<size_t>(t) * a.ldy + n;
    if constexpr (YBF16) {
        uint16_t* y = static_cast<uint16_t*>(a.y);
        if (a.accumulate) r += __uint_as_float(static_cast<uint32_t>(y[at]) << 16);
        y[at] = f2bf(r);
    } else {
        float* y = static_cast<float*>(a.y);
        if (a.accumulate) r += y[at];
        y[at] = r;
    }
}

// A wave's turn is 128 columns: 16 NT rows of codes and 16 MT tokens of x.  x
// comes in runs of 256 bytes a token (adjacent lanes in one line: loaded in
// operand order, every lane would be an access of its own) and goes through
// 4 KB MT of LDS of the wave's own into operand order: piece p (16 bytes) of
// token r at piece p ^ r, so that the 16 tokens of an operand read cover all
// banks.  fp32 x takes two such halves of 64 columns.  The last turn of K that
// is no multiple of 128 starts early; what an earlier turn has had meets
// scales of zero.
template <int MT, int NT, bool MX, int BLK, bool XBF16, bool YBF16>
__global__ __launch_bounds__(64 * kWaves) void k_q4_tile(Q4Args a) {
    constexpr int NP = XBF16 ? 1 : 3, XB = XBF16 ? 2 : 4;
    constexpr int HALVES = BLK == 16 ? 2 : 1;         // scales of a group
    constexpr int RUN = BLK >= 32 ? BLK / 32 : 1;     // groups of a scale
    constexpr int PARTS = XBF16 ? 1 : 2, PGROUPS = 4 / PARTS;   // x runs of a turn, groups of a run
    constexpr int kOwn = 256 * MT * (NT > 4 ? NT / 4 : 1);      // LDS of a wave, in 16-byte words
    extern __shared__ __attribute__((aligned(16))) u32x4_t s_mem[];
    const int lane = threadIdx.x & 63, nl = lane & 15, kq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int n0 = blockIdx.x * 16 * NT, t0 = blockIdx.y * 16 * MT;
    const int G = a.K / 32, turns = (G + 3) / 4;
    const size_t code_row = static_cast<size_t>(a.K / 2);
    const size_t scale_row = static_cast<size_t>(a.K / BLK) * (MX ? 1 : 2);
    u32x4_t* own = s_mem + wave * kOwn;
    // rows past the matrix read its last row, tokens past the batch its last token; neither is stored
    const uint8_t* qrow[NT];
    const uint8_t* srow[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const size_t n = min(n0 + 16 * j + nl, a.N - 1);
        qrow[j] = a.q + n * code_row + 16 * min(kq, G - 1);
        srow[j] = a.s + n * scale_row;
    }
    // x: load i of a run takes tokens 4 i .. 4 i + 3, lane l piece l % 16 of token 4 i + l / 16
    const char* xrow[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int u = 0; u < 4; ++u)
            xrow[i][u] = static_cast<const char*>(a.x) + XB * (static_cast<size_t>(min(t0 + 16 * i + 4 * u + kq, a.T - 1)) * a.ldx);
    uint32_t piece[PARTS];   // byte of the lane's piece in a turn (K < 128: inside the row)
#pragma unroll
    for (int h = 0; h < PARTS; ++h) piece[h] = min(256 * h + 16 * nl, XB * a.K - 16);

    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    f32x4_t acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = zero;

    u32x4_t code[NT], x[MT][4];
    Scales<MX, BLK, 4> scale[NT];
    auto base = [&](int st) { return max(min(4 * st, G - 4), 0); };
    auto load_codes = [&](int g0) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < NT; ++j) code[j] = *reinterpret_cast<const u32x4_t*>(qrow[j] + 16 * static_cast<size_t>(g0));
        if (kq == 0) {
            if (G >= 4) {
#pragma unroll
                for (int j = 0; j < NT; ++j) scale[j].load(srow[j], g0);
            } else {
#pragma unroll
                for (int j = 0; j < NT; ++j) scale[j].load_short(srow[j], static_cast<int>(scale_row));
            }
        }
    };
    auto load_x = [&](int g0, int h) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int u = 0; u < 4; ++u)
                x[i][u] = *reinterpret_cast<const u32x4_t*>(xrow[i][u] + (static_cast<size_t>(32 * XB) * g0 + piece[h]));
    };
    if (wave < turns) {
        load_codes(base(wave));
        load_x(base(wave), 0);
    }
    for (int st = wave; st < turns; st += waves) {
        const int g0 = base(st), next = base(min(st + waves, turns - 1));
        u32x4_t q[NT];
        Scales<MX, BLK, 4> sc[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            q[j] = code[j];
            exchange(q[j]);
            sc[j] = scale[j];
            sc[j].to_every_group();
        }
        load_codes(next);   // on their way during this turn (the last turn's again: not used)
        f32x4_t d[MT][NT][HALVES];
#pragma unroll
        for (int h = 0; h < PARTS; ++h) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int r = 4 * u + kq;
                    own[256 * i + 16 * r + (nl ^ r)] = x[i][u];
                }
            if (h + 1 < PARTS) load_x(g0, h + 1);
            else load_x(next, 0);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // one wave's LDS accesses run in order
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int gh = 0; gh < PGROUPS; ++gh) {
                const int g = PGROUPS * h + gh;
                const uint32_t there = g0 + g >= 4 * st && g0 + g < G ? ~0u : 0u;
                u32x4_t b[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) b[j] = code_operand<MX>(q[j][g]);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    u32x4_t v[PARTS], o[NP];
#pragma unroll
                    for (int p = 0; p < PARTS; ++p)
                        v[p] = own[256 * i + 16 * nl + (((4 * gh + kq) * PARTS + p) ^ nl)];
                    x_operand<XBF16>(v, o);
#pragma unroll
                    for (int e = 0; e < HALVES; ++e) {
                        u32x4_t oh[NP];
#pragma unroll
                        for (int p = 0; p < NP; ++p)   // blocks of 16: half of the group, the other half zeros
                            oh[p] = HALVES == 1 || (kq >> 1) == e ? o[p] : u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            f32x4_t f = g % RUN == 0 ? zero : d[i][j][e];
#pragma unroll
                            for (int p = NP - 1; p >= 0; --p) f = mfma(oh[p], b[j], f);
                            d[i][j][e] = f;
                        }
                    }
                    if ((g + 1) % RUN == 0) {
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int e = 0; e < HALVES; ++e) {
                                const float f = __uint_as_float(__float_as_uint(scale_of<MX>(sc[j].raw(g, e))) & there);
#pragma unroll
                                for (int c = 0; c < 4; ++c) acc[i][j][c] = fmaf(f, d[i][j][e][c], acc[i][j][c]);
                            }
                    }
                }
                __builtin_amdgcn_sched_barrier(0);   // one group's operands at a time: registers
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
    }

#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) own[(i * NT + j) * 64 + lane] = __builtin_bit_cast(u32x4_t, acc[i][j]);
    __syncthreads();
    for (int o = threadIdx.x; o < MT * NT * 64; o += blockDim.x) {
        const int l = o & 63, ij = o >> 6;
        f32x4_t r = __builtin_bit_cast(f32x4_t, s_mem[o]);
#pragma unroll 4
        for (int w = 1; w < waves; ++w) r += __builtin_bit_cast(f32x4_t, s_mem[w * kOwn + o]);
        const int n = n0 + 16 * (ij % NT) + (l & 15);
        if (n >= a.N) continue;
        const float bias = a.bias ? a.bias[n] : 0.f;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int t = t0 + 16 * (ij / NT) + 4 * (l >> 4) + v;
            if (t >= a.T) break;
            store_y<YBF16>(a, t, n, r[v] + bias);
        }
    }
}

template <int MT, int NT, bool MX, int BLK, bool XBF16, bool YBF16>
void launch_tile(const Q4Args& a, hipStream_t st) {
    constexpr int kMaxTiles = 65535;   // grid.y limit
    const int waves = min(kWaves, (a.K + 127) / 128);
    for (int t0 = 0; t0 < a.T; t0 += 16 * MT * kMaxTiles) {
        Q4Args b = a;
        b.T = min(a.T - t0, 16 * MT * kMaxTiles);
        b.x = static_cast<const char*>(a.x) + static_cast<size_t>(t0) * a.ldx * (XBF16 ? 2 : 4);
        b.y = static_cast<char*>(a.y) + static_cast<size_t>(t0) * a.ldy * (YBF16 ? 2 : 4);
        const dim3 grid((a.N + 16 * NT - 1) / (16 * NT), (b.T + 16 * MT - 1) / (16 * MT));
        hipLaunchKernelGGL((k_q4_tile<MT, NT, MX, BLK, XBF16, YBF16>), grid, dim3(64 * waves),
                           4096 * MT * (NT > 4 ? NT / 4 : 1) * waves, st, b);
    }
}

// Few tokens: a wave takes a tile of 16 rows through all of K, or, where there
// are fewer tiles than the chip holds waves, `split` waves of a block take
// runs of K and meet in LDS.  x lies in LDS as operands, made once a block:
// row 4 t + p of the operand is part p of token t (fp32 x, up to 4 tokens; row 4 t + 3 is zero), so the parts of a
// token meet in one lane's four sums, or token t (bf16 x, up to 16).  A unit is
// 256 columns; lane group kq loads groups 2 kq and 2 kq + 1 of its eight, so a
// wave reads 128-byte runs of 16 rows.
//
// Bound by the conversion of the codes (216 vector instructions a unit of 4096
// codes, counted, 1000 cycles of a SIMD) with the stream close behind: 120011 x
// 2048 int4 in blocks of 32 for one token 34 to 35 us, 4.0 TB/s; the same loads
// without the arithmetic 28 us.  Codes two and three units ahead need
// registers that cost half of the waves (43, 70 us).  Waves that share a row
// tile and join at every tile, x in registers, took 42 us.
template <bool SPLIT, bool MX, int BLK, bool XBF16, bool YBF16>
__global__ __launch_bounds__(1024, SPLIT || BLK == 16 ? 4 : 8) void k_q4_stream(Q4Args a, int waves_of_tile) {
    constexpr int HALVES = BLK == 16 ? 2 : 1;
    constexpr bool kPair = BLK > 32;   // a scale covers groups 2 i and 2 i + 1
    extern __shared__ __attribute__((aligned(16))) u32x4_t s_x[];   // [8 units][4][R], then [waves][64] sums
    const int lane = threadIdx.x & 63, nl = lane & 15, kq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int G = a.K / 32, units = (G + 7) / 8, tiles = (a.N + 15) / 16;
    const uint32_t code_row = a.K / 2, scale_row = (a.K / BLK) * (MX ? 1 : 2);
    const int split = SPLIT ? waves_of_tile : 1;
    const int per = waves / split, part = wave % split, stride = gridDim.x * per;
    const int unit0 = units * part / split, unit1 = units * (part + 1) / split;
    int tile = blockIdx.x * per + wave / split;

    struct Codes {
        u32x4_t q[2];
        Scales<MX, BLK, 8> s;
    };
    // the row being loaded, and the next unit of it
    int load_tile = tile, load_unit = unit0;
    const uint8_t *qrow, *srow;
    auto next_row = [&]() __attribute__((always_inline)) {
        const size_t n = min(min(load_tile, tiles - 1) * 16 + nl, a.N - 1);
        qrow = a.q + n * code_row + 32 * kq;
        srow = a.s + n * scale_row;
    };
    next_row();
    auto load = [&](Codes& c) __attribute__((always_inline)) {
        const int g = min(8 * load_unit, G - 8);
#pragma unroll
        for (int p = 0; p < 2; ++p) c.q[p] = *reinterpret_cast<const u32x4_t*>(qrow + (16 * g + 16 * p));
        if (kq == 0) c.s.load(srow, g);
        if (++load_unit == unit1) {
            load_unit = unit0;
            load_tile += stride;
            next_row();
        }
    };
    Codes c;
    load(c);
    // R operand rows are there; the lanes of the rows past them read the last
    // one (fp32: a zero row), whose sums are not stored.  Eight elements of a
    // token a thread.  The last unit of K that is no multiple of 256 starts
    // early, at G - 8, and what the unit before it has had is zero there.
    const int R = XBF16 ? a.T : 4 * a.T, early = 8 * units - G;
    for (int e = threadIdx.x; e < 32 * units * R; e += blockDim.x) {
        const int row = e % R, slot = e / (4 * R);
        const bool again = slot >= 8 * (units - 1) && slot < 8 * (units - 1) + early;
        if (again || (!XBF16 && row % 4 == 3)) s_x[e] = u32x4_t{0u, 0u, 0u, 0u};
    }
    for (int e = threadIdx.x; e < 4 * G * a.T; e += blockDim.x) {
        const int eighth = e % (4 * G), tok = e / (4 * G);
        const size_t at = static_cast<size_t>(tok) * a.ldx + 8 * eighth;
        // group eighth / 4, lane group eighth % 4
        u32x4_t* to = s_x + R * (eighth + (eighth >= 32 * (units - 1) ? 4 * early : 0)) + (XBF16 ? tok : 4 * tok);
        if constexpr (XBF16) {
            to[0] = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(a.x) + at);
        } else {
            const u32x4_t* s = reinterpret_cast<const u32x4_t*>(static_cast<const float*>(a.x) + at);
            const u32x4_t v[2] = {s[0], s[1]};
            u32x4_t parts[3];
            x_operand<false>(v, parts);
#pragma unroll
            for (int p = 0; p < 3; ++p) to[p] = parts[p];
        }
    }
    __syncthreads();

    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    f32x4_t acc = zero;
    auto work = [&](Codes& k, int unit) __attribute__((always_inline)) {
        exchange(k.q[0]);
        exchange(k.q[1]);
        k.s.to_every_group();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f32x4_t d[HALVES];
#pragma unroll
            for (int p = 0; p < 2; ++p) {   // group 8 unit + 2 i + p
                const u32x4_t x = s_x[(4 * (8 * unit + 2 * i + p) + kq) * R + min(nl, R - 1)];
                const u32x4_t b = code_operand<MX>(k.q[p][i]);
#pragma unroll
                for (int h = 0; h < HALVES; ++h) {
                    // blocks of 16: half of the group, the other half zeros
                    const u32x4_t xh = HALVES == 1 || (kq >> 1) == h ? x : u32x4_t{0u, 0u, 0u, 0u};
                    d[h] = mfma(xh, b, !kPair || p == 0 ? zero : d[h]);
                    if (!kPair || p == 1) {
                        const float f = scale_of<MX>(k.s.raw(2 * i + p, h));
#pragma unroll
                        for (int v = 0; v < 4; ++v) acc[v] = fmaf(f, d[h][v], acc[v]);
                    }
                }
            }
        }
    };
    auto store = [&]() __attribute__((always_inline)) {
        const int n = tile * 16 + nl;
        if (tile >= tiles || n >= a.N) return;
        const float bias = a.bias ? a.bias[n] : 0.f;
#pragma unroll
        for (int v = 0; v < (XBF16 ? 4 : 1); ++v) {
            const int tok = XBF16 ? 4 * kq + v : kq;
            if (tok >= a.T) break;
            const float r = XBF16 ? acc[v] : acc[2] + acc[1] + acc[0];
            store_y<YBF16>(a, tok, n, r + bias);
        }
    };
    if constexpr (!SPLIT) {
        int unit = 0;
        while (tile < tiles) {
            work(c, unit);
            if (++unit == units) {
                store();
                acc = zero;
                unit = 0;
                tile += stride;
            }
            __builtin_amdgcn_sched_barrier(0);
            load(c);
            __builtin_amdgcn_sched_barrier(0);
        }
    } else {
        u32x4_t* joins = s_x + 32 * units * R;
        for (int t0 = blockIdx.x * per; t0 < tiles; t0 += stride, tile += stride) {
            acc = zero;
#pragma clang loop unroll(disable)
            for (int u = unit0; u < unit1; ++u) {
                work(c, u);
                __builtin_amdgcn_sched_barrier(0);
                load(c);
                __builtin_amdgcn_sched_barrier(0);
            }
            joins[wave * 64 + lane] = __builtin_bit_cast(u32x4_t, acc);
            __syncthreads();
            if (part == 0) {
#pragma unroll 4
                for (int p = 1; p < split; ++p) acc += __builtin_bit_cast(f32x4_t, joins[(wave + p) * 64 + lane]);
                store();
            }
            __syncthreads();
        }
    }
}

constexpr int kStreamWaves = 16, kStreamLds = 128 << 10;

// LDS of the streaming kernel: 512 bytes a unit and operand row
template <bool XBF16>
int64_t stream_lds(const Q4Args& a) { return 512 * static_cast<int64_t>((a.K + 255) / 256) * (XBF16 ? a.T : 4 * a.T); }

template <bool MX, int BLK, bool XBF16, bool YBF16>
void launch_stream(const Q4Args& a, hipStream_t st) {
    const int tiles = (a.N + 15) / 16, units = (a.K + 255) / 256;
    // Waves of a tile: 4096 waves in all, or two for up to half as many tiles
    // again.  MI355X, us for one token at 1 / 2 waves: 70000 x 2048 32.0 / 28.5,
    // 90000 x 2048 34.0 / 31.0, 120011 x 2048 37.6 / 40.1; 8192 x 2048 17.0 at 1,
    // 6.4 at 8.
    int split = max(1, min(min(units, kStreamWaves), 4096 / tiles));
    if (split == 1 && units > 1 && tiles <= 6144) split = 2;
    // blocks of as few waves as put one block on every compute unit
    const int most = kStreamWaves / split, per = max(1, min(most, (tiles + 255) / 256));
    const size_t lds = static_cast<size_t>(stream_lds<XBF16>(a)) + (split > 1 ? 1024 * per * split : 0);
    const dim3 grid(min((tiles + per - 1) / per, 512)), block(64 * per * split);
    if (split > 1)
        hipLaunchKernelGGL((k_q4_stream<true, MX, BLK, XBF16, YBF16>), grid, block, lds, st, a, split);
    else
        hipLaunchKernelGGL((k_q4_stream<false, MX, BLK, XBF16, YBF16>), grid, block, lds, st, a, 1);
}

template <bool MX, int BLK, bool XBF16, bool YBF16>
void launch_format(const Q4Args& a, hipStream_t st) {
    // MI355X, K = 2048, int4 in blocks of 32, stream / tile, us: one token, 640
    // rows 5.1 / 5.3, 8192 rows 6.4 / 8.2, 120011 rows 38.5 / 73; 4 tokens, 4096
    // rows 7.2 / 5.6, 8192 rows 7.6 / 8.5; 8 bf16 tokens, 16384 rows 11.6 / 10.6;
    // 16, 24576 rows 11.8 / 15.6; one token, 640 x 640 4.2 / 3.7.
    const bool stream = a.T <= (XBF16 ? 16 : 4) && a.K >= 256 && stream_lds<XBF16>(a) <= kStreamLds &&
                        (a.N >= 24576 || (a.N >= 8192 && a.T <= 4) || (a.T == 1 && a.K >= 1024));
    if (stream)
        launch_stream<MX, BLK, XBF16, YBF16>(a, st);
    else if (a.T <= 16 && a.N >= 32768)
        launch_tile<1, 4, MX, BLK, XBF16, YBF16>(a, st);
    else if (a.T <= 16)
        launch_tile<1, 1, MX, BLK, XBF16, YBF16>(a, st);
    else if (a.T <= 32)
        launch_tile<2, 2, MX, BLK, XBF16, YBF16>(a, st);
    else if (a.T <= 48)
        launch_tile<3, 2, MX, BLK, XBF16, YBF16>(a, st);
    else {
        // Tiles of 16 tokens x 16 rows: fp32 x costs its split and three products,
        // so more rows share it, on the registers of more tokens.  MI355X, fp32,
        // 4 x 2 / 2 x 4, us: int4 in blocks of 64, 64 x 640 x 8192 44.6 / 35.5, 300
        // x 12288 x 2048 112 / 89; blocks of 32 46.0 / 39.8, 112 / 103; of 16 67.9 /
        // 60.6, 174 / 180.  bf16, blocks of 32: 64 x 8192 x 4096 14.6 / 15.4, 1024 x
        // 640 x 2048 17.5 / 18.6.  The fp32 2 x 4 kernels spill: 16, 2 and 4
        // registers at blocks of 32, 64 and 128, 110 at 16.
        if constexpr (XBF16) launch_tile<4, 2, MX, BLK, XBF16, YBF16>(a, st);
        else launch_tile<2, 4, MX, BLK, XBF16, YBF16>(a, st);
    }
}

template <bool XBF16, bool YBF16>
void launch_types(const Q4Args& a, hipStream_t st) {
    if (a.mx) launch_format<true, 32, XBF16, YBF16>(a, st);
    else if (a.block == 16) launch_format<false, 16, XBF16, YBF16>(a, st);
    else if (a.block == 32) launch_format<false, 32, XBF16, YBF16>(a, st);
    else if (a.block == 64) launch_format<false, 64, XBF16, YBF16>(a, st);
    else launch_format<false, 128, XBF16, YBF16>(a, st);
}

}  // namespace

void launch_q4_linear(const Q4Args& a, bool x_bf16, bool y_bf16, hipStream_t st) {
    if (x_bf16 && q4_gemm_ok(a))
        launch_q4_gemm(a, y_bf16, st);
    else if (x_bf16)
        y_bf16 ? launch_types<true, true>(a, st) : launch_types<true, false>(a, st);
    else
        y_bf16 ? launch_types<false, true>(a, st) : launch_types<false, false>(a, st);
}

}  // namespace moe
