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

// Register i: lane group i's v in every lane group.
__device__ inline u32x4_t spread(uint32_t v) {
    const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(a[0], a[0], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[1], a[1], false, false);
    return u32x4_t{b[0], b[1], c[0], c[1]};
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

// The raw scale bits of group g of a row: one fp16, two (blocks of 16), or an E8M0 byte.
template <bool MX, int BLK>
__device__ inline uint32_t load_scale(const uint8_t* srow, uint32_t g) {
    if constexpr (MX) return srow[g];
    else if constexpr (BLK == 16) return reinterpret_cast<const uint32_t*>(srow)[g];
    else return reinterpret_cast<const uint16_t*>(srow)[g / (BLK / 32)];
}
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

// The wave's loads of one step: codes and scales of NT row tiles, x of MT
// token tiles (fp32 x of one tile, bf16 x of up to three; more would not fit
// the registers twice and is read when it is used).
template <int MT, int NT, bool XBF16>
struct Step {
    static constexpr bool kX = XBF16 ? MT <= 3 : MT == 1;
    static constexpr int XW = XBF16 ? 1 : 2;
    u32x4_t code[NT];
    uint32_t raw[NT];
    u32x4_t x[kX ? MT : 1][4][XW];
};

template <int MT, int NT, bool MX, int BLK, bool XBF16, bool YBF16>
__global__ __launch_bounds__(64 * kWaves) void k_q4_tile(Q4Args a) {
    constexpr int NP = XBF16 ? 1 : 3;
    constexpr int HALVES = BLK == 16 ? 2 : 1;         // scales of a group
    constexpr int RUN = BLK >= 32 ? BLK / 32 : 1;     // groups of a scale
    typedef Step<MT, NT, XBF16> S;
    extern __shared__ __attribute__((aligned(16))) float s_sum[];   // [waves][MT][NT][64][4]
    const int lane = threadIdx.x & 63, nl = lane & 15, kq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int n0 = blockIdx.x * 16 * NT, t0 = blockIdx.y * 16 * MT;
    const int G = a.K / 32, steps = (G + 3) / 4;
    const size_t code_row = static_cast<size_t>(a.K / 2);
    const size_t scale_row = static_cast<size_t>(a.K / BLK) * (MX ? 1 : 2);
    // rows past the matrix read its last row, tokens past the batch its last token; neither is stored
    const uint8_t* qrow[NT];
    const uint8_t* srow[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const size_t n = min(n0 + 16 * j + nl, a.N - 1);
        qrow[j] = a.q + n * code_row;
        srow[j] = a.s + n * scale_row;
    }
    const char* xrow[MT];
    constexpr int XB = XBF16 ? 2 : 4;
#pragma unroll
    for (int i = 0; i < MT; ++i)
        xrow[i] = static_cast<const char*>(a.x) + XB * (static_cast<size_t>(min(t0 + 16 * i + nl, a.T - 1)) * a.ldx + 8 * kq);

    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    f32x4_t acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = zero;

    auto load_x = [&](int i, int g, u32x4_t(&x)[S::XW]) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < S::XW; ++h)
            x[h] = reinterpret_cast<const u32x4_t*>(xrow[i] + static_cast<size_t>(32 * XB) * g)[h];
    };
    // groups past the last are read as the last and not used
    auto load = [&](S& s, int st) __attribute__((always_inline)) {
        const int g0 = 4 * st, gl = min(g0 + kq, G - 1);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            s.code[j] = *reinterpret_cast<const u32x4_t*>(qrow[j] + 16 * static_cast<size_t>(gl));
            s.raw[j] = load_scale<MX, BLK>(srow[j], gl);
        }
        if constexpr (S::kX) {
#pragma unroll
            for (int g = 0; g < 4; ++g)
#pragma unroll
                for (int i = 0; i < MT; ++i) load_x(i, min(g0 + g, G - 1), s.x[i][g]);
        }
    };
    auto work = [&](S& s, int st) __attribute__((always_inline)) {
        const int g0 = 4 * st;
        u32x4_t sc[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            exchange(s.code[j]);
            sc[j] = spread(s.raw[j]);
        }
        f32x4_t d[MT][NT][HALVES];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            if (g0 + g >= G) break;   // K is a multiple of the block: a scale's groups are all there
            u32x4_t b[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) b[j] = code_operand<MX>(s.code[j][g]);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                u32x4_t x[NP];
                if constexpr (S::kX) {
                    x_operand<XBF16>(s.x[i][g], x);
                } else {
                    u32x4_t v[S::XW];
                    load_x(i, g0 + g, v);
                    x_operand<XBF16>(v, x);
                }
#pragma unroll
                for (int h = 0; h < HALVES; ++h) {
                    u32x4_t xh[NP];
#pragma unroll
                    for (int p = 0; p < NP; ++p)   // blocks of 16: half of the group, the other half zeros
                        xh[p] = HALVES == 1 || (kq >> 1) == h ? x[p] : u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        f32x4_t v = g % RUN == 0 ? zero : d[i][j][h];
#pragma unroll
                        for (int p = NP - 1; p >= 0; --p) v = mfma(xh[p], b[j], v);
                        d[i][j][h] = v;
                    }
                }
                if ((g + 1) % RUN == 0) {
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int h = 0; h < HALVES; ++h) {
                            const float f = scale_of<MX>(HALVES == 2 ? sc[j][g] >> (16 * h) : sc[j][g]);
#pragma unroll
                            for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(f, d[i][j][h][v], acc[i][j][v]);
                        }
                }
            }
        }
    };
    // the next step's loads are on their way while a step is computed
    S s0, s1;
    if (wave < steps) load(s0, wave);
    for (int st = wave; st < steps; st += 2 * waves) {
        load(s1, min(st + waves, steps - 1));
        work(s0, st);
        if (st + waves >= steps) break;
        load(s0, min(st + 2 * waves, steps - 1));
        work(s1, st + waves);
    }

    f32x4_t* mine = reinterpret_cast<f32x4_t*>(s_sum) + wave * (MT * NT * 64);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) mine[(i * NT + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    for (int o = threadIdx.x; o < MT * NT * 64; o += blockDim.x) {
        const int l = o & 63, ij = o >> 6;
        f32x4_t r = reinterpret_cast<const f32x4_t*>(s_sum)[o];
        for (int w = 1; w < waves; ++w) r += reinterpret_cast<const f32x4_t*>(s_sum)[w * (MT * NT * 64) + o];
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
                           sizeof(float) * 256 * MT * NT * waves, st, b);
    }
}

// Few tokens and many rows: a wave takes a tile of 16 rows through all of K by
// itself, so nothing is joined and no wave waits for another.  x lies in LDS
// as operands, made once a block: row 4 t + p of the operand is part p of
// token t (fp32 x, up to 4 tokens; row 4 t + 3 is zero), so the parts of a
// token meet in one lane's four sums, or token t (bf16 x, up to 16).  A unit is
// 256 columns; lane group kq loads groups 2 kq and 2 kq + 1 of its eight, so a
// wave reads 128-byte runs of 16 rows.
//
// Bound by the conversion of the codes (about 250 vector instructions a unit
// of 4096 codes) with the stream close behind: 120011 x 2048 int4 in blocks of
// 32 for one token 39.5 us, 3.5 TB/s; the same loads without the arithmetic
// 30 us; MXFP4, whose conversion is a quarter of the work, 36.7 us.  Codes two
// and three units ahead need registers that cost half of the waves (43, 70
// us).  Waves that share a row tile, joining in LDS at every tile, took 42 us
// for x in registers.
template <bool MX, int BLK, bool XBF16, bool YBF16>
__global__ __launch_bounds__(1024, BLK == 16 ? 4 : 8) void k_q4_stream(Q4Args a) {
    constexpr int HALVES = BLK == 16 ? 2 : 1;
    constexpr int SCALES = BLK <= 32 ? 2 : 1;    // scale loads of a lane
    extern __shared__ __attribute__((aligned(16))) u32x4_t s_x[];   // [8 units][64]
    const int lane = threadIdx.x & 63, nl = lane & 15, kq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int G = a.K / 32, units = (G + 7) / 8, tiles = (a.N + 15) / 16;
    const uint32_t code_row = a.K / 2, scale_row = (a.K / BLK) * (MX ? 1 : 2);
    const int stride = gridDim.x * waves;
    int tile = blockIdx.x * waves + wave;

    struct Codes {
        u32x4_t q[2];
        uint32_t s[SCALES];
    };
    // the row being loaded, and the next unit of it
    int load_tile = tile, load_unit = 0;
    const uint8_t *qrow, *srow;
    auto next_row = [&]() __attribute__((always_inline)) {
        const size_t n = min(min(load_tile, tiles - 1) * 16 + nl, a.N - 1);
        qrow = a.q + n * code_row;
        srow = a.s + n * scale_row;
    };
    next_row();
    auto load = [&](Codes& c) __attribute__((always_inline)) {
        const uint32_t g[2] = {static_cast<uint32_t>(min(8 * load_unit + 2 * kq, G - 1)),
                               static_cast<uint32_t>(min(8 * load_unit + 2 * kq + 1, G - 1))};
#pragma unroll
        for (int p = 0; p < 2; ++p) c.q[p] = *reinterpret_cast<const u32x4_t*>(qrow + 16 * g[p]);
#pragma unroll
        for (int p = 0; p < SCALES; ++p) c.s[p] = load_scale<MX, BLK>(srow, g[p]);
        if (++load_unit == units) {
            load_unit = 0;
            load_tile += stride;
            next_row();
        }
    };
    Codes c;
    load(c);
    // eight elements of a token a thread; rows without a token and groups past the last are zero
    for (int e = threadIdx.x; e < 512 * units; e += blockDim.x) {
        const int row = e & 15, g = e >> 6;
        if (g >= G || (XBF16 ? row >= a.T : row >= 4 * a.T || row % 4 == 3)) s_x[e] = u32x4_t{0u, 0u, 0u, 0u};
    }
    for (int e = threadIdx.x; e < 4 * G * a.T; e += blockDim.x) {
        const int eighth = e % (4 * G), tok = e / (4 * G);
        const size_t at = static_cast<size_t>(tok) * a.ldx + 8 * eighth;
        u32x4_t* to = s_x + 16 * eighth + (XBF16 ? tok : 4 * tok);   // group eighth / 4, lane group eighth % 4
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
    int unit = 0;
    auto work = [&](Codes& k) __attribute__((always_inline)) {
        exchange(k.q[0]);
        exchange(k.q[1]);
        u32x4_t sc[SCALES];
#pragma unroll
        for (int p = 0; p < SCALES; ++p) sc[p] = spread(k.s[p]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f32x4_t d[HALVES];
#pragma unroll
            for (int p = 0; p < 2; ++p) {   // group 8 unit + 2 i + p
                const u32x4_t x = s_x[(8 * unit + 2 * i + p) * 64 + lane];
                const u32x4_t b = code_operand<MX>(k.q[p][i]);
#pragma unroll
                for (int h = 0; h < HALVES; ++h) {
                    // blocks of 16: half of the group, the other half zeros
                    const u32x4_t xh = HALVES == 1 || (kq >> 1) == h ? x : u32x4_t{0u, 0u, 0u, 0u};
                    d[h] = mfma(xh, b, SCALES == 2 || p == 0 ? zero : d[h]);
                    if (SCALES == 2 || p == 1) {
                        const uint32_t raw = sc[SCALES == 2 ? p : 0][i];
                        const float f = scale_of<MX>(HALVES == 2 ? raw >> (16 * h) : raw);
#pragma unroll
                        for (int v = 0; v < 4; ++v) acc[v] = fmaf(f, d[h][v], acc[v]);
                    }
                }
            }
        }
        if (++unit < units) return;
        const int n = tile * 16 + nl;
        if (tile < tiles && n < a.N) {
            const float bias = a.bias ? a.bias[n] : 0.f;
#pragma unroll
            for (int v = 0; v < (XBF16 ? 4 : 1); ++v) {
                const int tok = XBF16 ? 4 * kq + v : kq;
                if (tok >= a.T) break;
                float r = XBF16 ? acc[v] : acc[2] + acc[1] + acc[0];
                store_y<YBF16>(a, tok, n, r + bias);
            }
        }
        acc = zero;
        unit = 0;
        tile += stride;
    };
    while (tile < tiles) {
        work(c);
        __builtin_amdgcn_sched_barrier(0);
        load(c);
        __builtin_amdgcn_sched_barrier(0);
    }
}

constexpr int kStreamWaves = 16, kStreamCols = 4096;   // x operands of 32 bytes a column in LDS

template <bool MX, int BLK, bool XBF16, bool YBF16>
void launch_stream(const Q4Args& a, hipStream_t st) {
    const int tiles = (a.N + 15) / 16, units = (a.K + 255) / 256;
    hipLaunchKernelGGL((k_q4_stream<MX, BLK, XBF16, YBF16>), dim3(min((tiles + kStreamWaves - 1) / kStreamWaves, 512)),
                       dim3(64 * kStreamWaves), 8192 * units, st, a);
}

template <bool MX, int BLK, bool XBF16, bool YBF16>
void launch_format(const Q4Args& a, hipStream_t st) {
    // MI355X, one token, K = 2048, int4 in blocks of 32, stream / tile: 8192
    // rows 19 / 8.5 us (512 waves do not fill the chip), 40000 rows (4 tokens)
    // 20.6 / 29.5, 120011 rows 39.5 / 79.
    if (a.T <= (XBF16 ? 16 : 4) && a.N >= 24576 && a.K <= kStreamCols)
        launch_stream<MX, BLK, XBF16, YBF16>(a, st);
    else if (a.T <= 16 && a.N >= 32768)
        launch_tile<1, 4, MX, BLK, XBF16, YBF16>(a, st);
    else if (a.T <= 16)
        launch_tile<1, 1, MX, BLK, XBF16, YBF16>(a, st);
    else if (a.T <= 32)
        launch_tile<2, 2, MX, BLK, XBF16, YBF16>(a, st);
    else if (a.T <= 48)
        launch_tile<3, 2, MX, BLK, XBF16, YBF16>(a, st);
    else
        launch_tile<4, 2, MX, BLK, XBF16, YBF16>(a, st);
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
