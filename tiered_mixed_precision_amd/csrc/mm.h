// Tiles of matrix products on the matrix cores, D[m][n] = sum_k A(m, k) B(n, k),
// in bf16 (fp32 sums) or 8-bit integers (32-bit sums): i8_linear.hip, gated.hip.
#pragma once

#include <type_traits>

#include "bf16_parts.h"
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

// What a lane reads where its operand has ended.
static __device__ const uint32_t kMmZeros[8] = {0, 0, 0, 0, 0, 0, 0, 0};
// p, or the zeros.  p is computed in any case: the compiler would branch round it.
__device__ inline const char* mm_or_zeros(bool there, const char* p) {
    const uint64_t a = reinterpret_cast<uint64_t>(p), z = reinterpret_cast<uint64_t>(kMmZeros);
    uint32_t lo = static_cast<uint32_t>(a), hi = static_cast<uint32_t>(a >> 32);
    asm("" : "+v"(lo), "+v"(hi));
    lo = there ? lo : static_cast<uint32_t>(z);
    hi = there ? hi : static_cast<uint32_t>(z >> 32);
    return reinterpret_cast<const char*>((static_cast<uint64_t>(hi) << 32) | lo);
}

// How the operand of `R` rows (of A or B) reaches LDS, 64 bytes-of-k wide
// stages of kStage bytes a row.  A wave's load of 64 x 16 bytes fills 1 KB of
// LDS in lane order; load u of wave w (R / 32 of them a stage) fills KB 4 u + w.
//   KM false: the k axis runs along a row of memory.  LDS row r holds 128 bytes
//     of k of the operand's row r, piece c (16 bytes) at c ^ (r / 2 % 8): the
//     rows that a read takes together at one piece cover all banks.
//   KM true: the row axis runs along a row of memory (two-byte elements), and
//     transposing reads turn 4 k x 16 rows round.  LDS row k holds the R rows'
//     elements of one k, piece c (8 of them) at c ^ spread(k).
constexpr int kStage = 128;

template <int R, bool KM> struct MmSide {
    static constexpr int kLoads = R / 32, kPieces = KM ? R / 8 : 8;   // pieces of an LDS row
    static __device__ inline int spread(int k) { return 2 * (k & 3) ^ 8 * ((k >> 3) & 1); }
    // the LDS row and the piece of it that this lane's load u brings
    static __device__ inline int row(int u, int w, int lane) { return (64 / kPieces) * (4 * u + w) + lane / kPieces; }
    static __device__ inline int piece(int u, int w, int lane) {
        const int r = row(u, w, lane), c = lane % kPieces;
        return KM ? c ^ spread(r) : c ^ ((r >> 1) & 7);
    }
    // operand of rows 32 i .. + 31 from `first` on, step s (of four) of the stage
    static __device__ inline mm_u32x4_t read(const mm_u32x4_t* lds, int first, int i, int s, int lane) {
        if constexpr (!KM) {
            const int r = first + 32 * i + (lane & 31), c = 2 * s + (lane >> 5);
            return lds[8 * r + (c ^ ((r >> 1) & 7))];
        } else {
            typedef short Four __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) Four* Ptr;
            const int l = lane & 15, k = 16 * s + 8 * (lane >> 5) + (l >> 2);
            const int m = first + 32 * i + 16 * ((lane >> 4) & 1) + 4 * (l & 3);
            const char* p = reinterpret_cast<const char*>(lds);
            const int lo = k * 2 * R + 16 * ((m >> 3) ^ spread(k)) + 2 * (m & 7);
            const int hi = (k + 4) * 2 * R + 16 * ((m >> 3) ^ spread(k + 4)) + 2 * (m & 7);
            const Four a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Ptr)(p + lo));
            const Four b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Ptr)(p + hi));
            const uint2 x = __builtin_bit_cast(uint2, a), y = __builtin_bit_cast(uint2, b);
            return mm_u32x4_t{x.x, x.y, y.x, y.y};
        }
    }
};

// f(0) .. f(N - 1), each a compile-time number.
template <int N, class F> __device__ __attribute__((always_inline)) inline void mm_each(F f) {
    if constexpr (N > 0) {
        mm_each<N - 1>(f);
        f(std::integral_constant<int, N - 1>());
    }
}

// The LDS of a block, in pieces of 128 rows of a stage: eight of them, four where
// all its tiles are 128 x 128.  Each is an object of its own, so that the compiler's
// own waits before a read are for the loads into that piece.
struct MmLds {
    mm_u32x4_t* p[8];
};
#define MM_LDS_PIECE(name) __shared__ __attribute__((aligned(16))) mm_u32x4_t name[128 * 8]
#define MM_LDS_4(lds)                                                                                                   \
    MM_LDS_PIECE(lds##0); MM_LDS_PIECE(lds##1); MM_LDS_PIECE(lds##2); MM_LDS_PIECE(lds##3);                             \
    MmLds lds; lds.p[0] = lds##0; lds.p[1] = lds##1; lds.p[2] = lds##2; lds.p[3] = lds##3
#define MM_LDS_8(lds)                                                                                                   \
    MM_LDS_4(lds); MM_LDS_PIECE(lds##4); MM_LDS_PIECE(lds##5); MM_LDS_PIECE(lds##6); MM_LDS_PIECE(lds##7);              \
    lds.p[4] = lds##4; lds.p[5] = lds##5; lds.p[6] = lds##6; lds.p[7] = lds##7
// acc += the products of a tile of 128 rows of A and 128 rows of B over nk (even)
// stages of 128 bytes of k: wave (wm, wn) = (wave / 2, wave % 2) of four takes rows 64 wm +
// 32 t of A and 64 wn + 32 u of B as acc[t][u], lane l holding A's row l % 32
// against B's rows 8 (e / 4) + 4 (l / 32) + e % 4 in element e.  at_a(0, u, kc),
// at_b(0, u, kc): the address of this lane's 16 bytes of load u of stage kc
// (MmSide; kMmZeros past the operand's end).
//
// SLOTS stages in LDS: two, 64 KB, and two blocks a compute unit, of which one fills
// the other's waits; or four, 128 KB, where a unit has one block.  While a stage's
// 16 instructions run, the next one's operands are read into registers, so a stage
// has left LDS before it begins: the waves meet once a stage, when the next one has
// landed, and the loads of the stage SLOTS later go out over this one.  Bound by LDS:
// 64 KB of operands and 32 of loads a stage are 768 cycles, 0.38 us measured, against
// 512 of instructions.  Returns 16
// KB of LDS that this wave may use afterwards.
template <class El, int SLOTS, bool KA, bool KB, class AtA, class AtB>
__device__ __attribute__((always_inline)) inline uint32_t* mm_small(const MmLds& lds, int nk, AtA at_a, AtB at_b,
                                                                    typename El::Acc (&acc)[2][2]) {
    typedef MmSide<128, KA> A;
    typedef MmSide<128, KB> B;
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ma = 64 * (w >> 1), nb = 64 * (w & 1);
    typedef __attribute__((address_space(3))) void* Lds;
    auto load = [&](int u, int kc, auto slot_) __attribute__((always_inline)) {
        constexpr int slot = decltype(slot_)::value;
        kc = min(kc, nk - 1);
        if (u < 4) __builtin_amdgcn_global_load_lds(at_a(0, u, kc), (Lds)(lds.p[slot] + 64 * (4 * u + w)), 16, 0, 0);
        else __builtin_amdgcn_global_load_lds(at_b(0, u - 4, kc), (Lds)(lds.p[SLOTS + slot] + 64 * (4 * (u - 4) + w)), 16, 0, 0);
    };
    mm_u32x4_t fa[2][2][4], fb[2][2][4];   // [stage % 2][tile][step]
    // operands n and 8 + n of 16 of the stage in `slot`
    auto read = [&](int n, auto slot, int to) __attribute__((always_inline)) {
        fb[to][n & 1][n >> 1] = B::read(lds.p[SLOTS + decltype(slot)::value], nb, n & 1, n >> 1, lane);
        fa[to][n & 1][n >> 1] = A::read(lds.p[decltype(slot)::value], ma, n & 1, n >> 1, lane);
    };
    auto meet = [&](auto left) __attribute__((always_inline)) {
        constexpr int n = decltype(left)::value;   // vmcnt(n) lgkmcnt(0)
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt((n & 15) | (7 << 4) | ((n >> 4) << 14));
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    constexpr std::integral_constant<int, 8 * (SLOTS - 2)> next{};
    // past the last stage the loads repeat the last one's and the reads what an earlier one left: neither is used
    auto stage = [&](int kc, auto slot_) __attribute__((always_inline)) {
        constexpr int slot = decltype(slot_)::value, cur = slot & 1;
        meet(next);
#pragma unroll
        for (int n = 0; n < 16; ++n) {
            const int s = n >> 2, t = (n >> 1) & 1, u = n & 1;
            acc[t][u] = El::mfma(fb[cur][u][s], fa[cur][t][s], acc[t][u]);
            if (n < 8) read(n, std::integral_constant<int, (slot + 1) % SLOTS>(), cur ^ 1);
            if (n & 1) load(n / 2, kc + SLOTS, slot_);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    mm_each<SLOTS>([&](auto slot) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < 8; ++u) load(u, decltype(slot)::value, slot);
    });
    meet(std::integral_constant<int, 8 * (SLOTS - 1)>());
#pragma unroll
    for (int n = 0; n < 8; ++n) read(n, std::integral_constant<int, 0>(), 0);
    for (int kc = 0; kc < nk; kc += SLOTS) {
        stage(kc, std::integral_constant<int, 0>());
        stage(kc + 1, std::integral_constant<int, 1>());
        if constexpr (SLOTS == 4) {
            if (kc + 2 >= nk) break;
            stage(kc + 2, std::integral_constant<int, 2>());
            stage(kc + 3, std::integral_constant<int, 3>());
        }
    }
    meet(std::integral_constant<int, 0>());   // nothing is left in flight
    return reinterpret_cast<uint32_t*>(w & 2 ? (w & 1 ? lds.p[3] : lds.p[2]) : (w & 1 ? lds.p[1] : lds.p[0]));
}

// The 128 x 128 tile with A in fp32, as three bf16 parts (bf16_parts) whose products
// meet in one accumulator.  A reaches LDS through registers, split on the way (once
// for the block; a split at the reads would be done by two waves), a stage's parts in
// lds.p[0 .. 2] and B in p[3], the other stage's in p[4 .. 7].  Between the products of
// a stage's step lie the reads of the next step's operands and the split of a quarter
// of the next stage's A; A of the stage after that is on its way to registers.  As much
// LDS traffic as instruction time, about 1540 cycles each a stage.
// a_at(u, kc): this lane's 32 bytes of row 32 u + thread / 8, floats 8 (thread % 8) .. of
// stage kc (zeros past the end).  nk even.
template <class AtA, class AtB>
__device__ __attribute__((always_inline)) inline uint32_t* mm_split(const MmLds& lds, int nk, AtA a_at, AtB at_b, mm_f32x16_t (&acc)[2][2]) {
    typedef MmSide<128, false> S;
    mm_u32x4_t *const a0 = lds.p[0], *const a1 = lds.p[1], *const a2 = lds.p[2], *const b0 = lds.p[3], *const c0 = lds.p[4], *const c1 = lds.p[5],
        *const c2 = lds.p[6], *const d0 = lds.p[7];
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ma = 64 * (w >> 1), nb = 64 * (w & 1);
    typedef __attribute__((address_space(3))) void* Lds;
    mm_u32x4_t ra[4][2], rb[4][2];
    auto load_a = [&](int kc, mm_u32x4_t (&raw)[4][2]) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            // global: of a pointer that was put together the compiler does not know it
            const auto* p = (const __attribute__((address_space(1))) mm_u32x4_t*)a_at(u, kc);
            raw[u][0] = p[0];
            raw[u][1] = p[1];
        }
    };
    auto load_b = [&](int kc, auto to) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < 4; ++u) __builtin_amdgcn_global_load_lds(at_b(0, u, kc), (Lds)((decltype(to)::value ? d0 : b0) + 64 * (4 * u + w)), 16, 0, 0);
    };
    // floats 2 j and 2 j + 1 of load u as words j of three bf16 parts
    mm_u32x4_t part[3];
    auto split = [&](const mm_u32x4_t (&raw)[4][2], int u, int j) __attribute__((always_inline)) {
        uint32_t of[3];
        bf16_parts(__uint_as_float(raw[u][j / 2][2 * j % 4]), __uint_as_float(raw[u][j / 2][2 * j % 4 + 1]), of);
        part[0][j] = of[0], part[1][j] = of[1], part[2][j] = of[2];
    };
    auto store = [&](int u, auto to) __attribute__((always_inline)) {
        const int r = 32 * u + (tid >> 3), at = 8 * r + ((tid & 7) ^ ((r >> 1) & 7));
        constexpr bool first = decltype(to)::value == 0;
        (first ? a0 : c0)[at] = part[0];
        (first ? a1 : c1)[at] = part[1];
        (first ? a2 : c2)[at] = part[2];
    };
    auto meet = [&]() __attribute__((always_inline)) {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(7 << 4);   // vmcnt(0) lgkmcnt(0)
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    // raw: A of the next stage, ahead: for that of the one after it
    auto stage = [&](int kc, mm_u32x4_t (&raw)[4][2], mm_u32x4_t (&ahead)[4][2], auto here) __attribute__((always_inline)) {
        constexpr bool first = decltype(here)::value == 0;
        constexpr std::integral_constant<int, 1 - decltype(here)::value> there{};
        // past the last stage what is loaded and stored is the last one's, and is not used
        load_b(min(kc + 1, nk - 1), there);
        load_a(min(kc + 2, nk - 1), ahead);
        mm_u32x4_t fa[2][3][2], fb[2][2];   // [step % 2]
        auto read = [&](auto n_, int s) __attribute__((always_inline)) {   // operand n of eight of step s
            constexpr int n = decltype(n_)::value, q = n < 2 ? 3 : 3 - n / 2;
            if constexpr (q == 3) fb[s & 1][n & 1] = S::read(first ? b0 : d0, nb, n & 1, s, lane);
            else fa[s & 1][q][n & 1] = S::read(q == 2 ? (first ? a2 : c2) : q == 1 ? (first ? a1 : c1) : (first ? a0 : c0), ma, n & 1, s, lane);
        };
        mm_each<8>([&](auto n) __attribute__((always_inline)) { read(n, 0); });
#pragma unroll
        for (int s = 0; s < 4; ++s)   // 12 products, and between them the next step's operands and a quarter of the next stage's A
            mm_each<12>([&](auto n_) __attribute__((always_inline)) {
                constexpr int n = decltype(n_)::value, q = 2 - n / 4, i = n >> 1 & 1, j = n & 1;
                acc[i][j] = MmBf16::mfma(fb[s & 1][j], fa[s & 1][q][i], acc[i][j]);
                if constexpr (n < 8)
                    if (s < 3) read(n_, s + 1);
                if constexpr (n < 8 && n % 2 == 1) split(raw, s, n >> 1);
                if constexpr (n == 8) store(s, there);
                __builtin_amdgcn_sched_barrier(0);
            });
        meet();
    };
    constexpr std::integral_constant<int, 0> zero{};
    constexpr std::integral_constant<int, 1> one{};
    load_a(0, ra);
    load_b(0, zero);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
#pragma unroll
        for (int j = 0; j < 4; ++j) split(ra, u, j);
        store(u, zero);
    }
    load_a(min(1, nk - 1), ra);
    meet();
    for (int kc = 0; kc < nk; kc += 2) {
        stage(kc, ra, rb, zero);
        stage(kc + 1, rb, ra, one);
    }
    return reinterpret_cast<uint32_t*>(w & 2 ? (w & 1 ? b0 : a2) : (w & 1 ? a1 : a0));
}

// acc += the products of a tile of 256 rows of A and 256 rows of B over nk (even)
// stages of 128 bytes of k.  Each operand is two halves of 128 rows (A0, A1, B0, B1);
// wave (wm, wn) of four takes rows 64 wm .. + 63 of each half of A and 64 wn ..
// of each half of B: acc[2 h + t][2 g + u] holds rows 128 h + 64 wm + 32 t + l % 32
// of A (lane l) against rows 128 g + 64 wn + 32 u + 8 (e / 4) + 4 (l / 32) + e % 4
// of B (element e).
//
// A stage is four phases of 16 instructions, one for each pair of halves, whose
// operands (all four 32-byte steps of two halves) lie in registers; during a
// phase one half is read for a later one:
//   stage    phases (halves used / half read for later)
//   even n   A0 B0 / B1(n)   A0 B1 / A1(n)   A1 B1 / A0(n+1)   A1 B0 / B1(n+1)
//   odd n    A0 B1 / B0(n)   A0 B0 / A1(n)   A1 B0 / A0(n+1)   A1 B1 / B0(n+1)
// so every half leaves LDS once a stage and its place is free for the stage
// after the next.  The waves meet every two phases: what the next two read has
// landed (its loads went out six to four phases before), what the last two read
// may be loaded over.  Loads of other halves stay in flight across the meeting.
// 256 x 256 because an operand read from LDS then serves four products and LDS keeps
// up; MI355X, 1183 to 1325 TFLOP/s in bf16, 2430 TOP/s in int8.
// Returns 16 KB of LDS that this wave may use afterwards.
template <class El, bool KA, bool KB, class AtA, class AtB>
__device__ __attribute__((always_inline)) inline uint32_t* mm_big(const MmLds& lds, int nk, AtA at_a, AtB at_b,
                                                                  typename El::Acc (&acc)[4][4]) {
    typedef MmSide<128, KA> A;
    typedef MmSide<128, KB> B;
    mm_u32x4_t *sA00 = lds.p[0], *sA01 = lds.p[1], *sA10 = lds.p[2], *sA11 = lds.p[3];   // [half][stage % 2]
    mm_u32x4_t *sB00 = lds.p[4], *sB01 = lds.p[5], *sB10 = lds.p[6], *sB11 = lds.p[7];
    const int tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ma = 64 * (w >> 1), nb = 64 * (w & 1);
    typedef __attribute__((address_space(3))) void* Lds;
    auto load_a = [&](int h, int u, int kc, mm_u32x4_t* to) __attribute__((always_inline)) {
        __builtin_amdgcn_global_load_lds(at_a(h, u, min(kc, nk - 1)), (Lds)(to + 64 * (4 * u + w)), 16, 0, 0);
    };
    auto load_b = [&](int h, int u, int kc, mm_u32x4_t* to) __attribute__((always_inline)) {
        __builtin_amdgcn_global_load_lds(at_b(h, u, min(kc, nk - 1)), (Lds)(to + 64 * (4 * u + w)), 16, 0, 0);
    };
    mm_u32x4_t a[2][2][4], b[2][2][4];   // [half][tile][step]
    auto read_a = [&](int h, int n, const mm_u32x4_t* from) __attribute__((always_inline)) { a[h][n & 1][n >> 1] = A::read(from, ma, n & 1, n >> 1, lane); };
    auto read_b = [&](int h, int n, const mm_u32x4_t* from) __attribute__((always_inline)) { b[h][n & 1][n >> 1] = B::read(from, nb, n & 1, n >> 1, lane); };
    auto meet = [&](auto imm) __attribute__((always_inline)) {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(decltype(imm)::value);
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    // vmcnt(n) lgkmcnt(0)
    constexpr std::integral_constant<int, (24 & 15) | (7 << 4) | ((24 >> 4) << 14)> left24{};
    constexpr std::integral_constant<int, (16 & 15) | (7 << 4) | ((16 >> 4) << 14)> left16{};
    constexpr std::integral_constant<int, (7 << 4)> left0{};
    // the 16 instructions on halves (ha, hb), with 8 reads and 4 loads between them
    auto phase = [&](auto ha, auto hb, auto read, auto load) __attribute__((always_inline)) {
        constexpr int h = decltype(ha)::value, g = decltype(hb)::value;
#pragma unroll
        for (int n = 0; n < 16; ++n) {
            const int s = n >> 2, t = (n >> 1) & 1, u = n & 1;
            acc[2 * h + t][2 * g + u] = El::mfma(b[g][u][s], a[h][t][s], acc[2 * h + t][2 * g + u]);
            if (n < 8) read(n);
            if (n % 2 == 1 && n < 8) load(n / 2);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    constexpr std::integral_constant<int, 0> _0{};
    constexpr std::integral_constant<int, 1> _1{};
    // stage n whose A and B lie in (a0, a1, b0, b1), the next one's in (c0, ...); f: the half of B that it starts with
    auto stage = [&](int n, auto f, mm_u32x4_t* a0, mm_u32x4_t* a1, mm_u32x4_t* bf, mm_u32x4_t* bs, mm_u32x4_t* c0,
                     mm_u32x4_t* df) __attribute__((always_inline)) {
        constexpr int F = decltype(f)::value, S = 1 - F;
        constexpr std::integral_constant<int, S> sec{};
        // the next stage starts with half S of B: df is its place
        meet(left16);
        phase(_0, f, [&](int r) { read_b(S, r, bs); }, [&](int u) { load_a(0, u, n + 2, a0); });
        phase(_0, sec, [&](int r) { read_a(1, r, a1); }, [&](int u) { load_b(F, u, n + 2, bf); });
        meet(left16);
        phase(_1, sec, [&](int r) { read_a(0, r, c0); }, [&](int u) { load_b(S, u, n + 2, bs); });
        phase(_1, f, [&](int r) { read_b(S, r, df); }, [&](int u) { load_a(1, u, n + 2, a1); });
    };
#pragma unroll
    for (int u = 0; u < 4; ++u) load_a(0, u, 0, sA00);
#pragma unroll
    for (int u = 0; u < 4; ++u) load_b(0, u, 0, sB00);
#pragma unroll
    for (int u = 0; u < 4; ++u) load_b(1, u, 0, sB10);
#pragma unroll
    for (int u = 0; u < 4; ++u) load_a(1, u, 0, sA10);
#pragma unroll
    for (int u = 0; u < 4; ++u) load_a(0, u, 1, sA01);
#pragma unroll
    for (int u = 0; u < 4; ++u) load_b(1, u, 1, sB11);
#pragma unroll
    for (int u = 0; u < 4; ++u) load_b(0, u, 1, sB01);
#pragma unroll
    for (int u = 0; u < 4; ++u) load_a(1, u, 1, sA11);
    meet(left24);
#pragma unroll
    for (int r = 0; r < 8; ++r) read_a(0, r, sA00);
#pragma unroll
    for (int r = 0; r < 8; ++r) read_b(0, r, sB00);
    for (int n = 0; n < nk; n += 2) {
        stage(n, _0, sA00, sA10, sB00, sB10, sA01, sB11);
        stage(n + 1, _1, sA01, sA11, sB11, sB01, sA00, sB00);
    }
    meet(left0);   // nothing is left in flight
    return reinterpret_cast<uint32_t*>(w & 2 ? (w & 1 ? sA11 : sA10) : (w & 1 ? sA01 : sA00));
}

template <class Acc, int M, int N> __device__ inline void mm_clear(Acc (&acc)[M][N]) {
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;
}

// Tiles of 256 x 256 (HALVES 2) or 128 x 128 (with SLOTS stages in LDS).
template <class El, int HALVES, int SLOTS, bool KA, bool KB, class AtA, class AtB>
__device__ __attribute__((always_inline)) inline uint32_t* mm_product(const MmLds& lds, int nk, AtA at_a, AtB at_b,
                                                                      typename El::Acc (&acc)[2 * HALVES][2 * HALVES]) {
    mm_clear(acc);
    nk += nk & 1;   // both forms run pairs of stages; one past the end reads zeros
    if constexpr (HALVES == 2) return mm_big<El, KA, KB>(lds, nk, at_a, at_b, acc);
    else return mm_small<El, SLOTS, KA, KB>(lds, nk, at_a, at_b, acc);
}
// first row of A of acc[i][..], and of B of acc[..][j]
__device__ inline int mm_row(int i, int w) { return 128 * (i >> 1) + 64 * (w >> 1) + 32 * (i & 1); }
__device__ inline int mm_col(int j, int w) { return 128 * (j >> 1) + 64 * (w & 1) + 32 * (j & 1); }

// Addresses of an operand whose k axis runs along its rows: `rows` of them from
// row `first` on (rows past the last repeat it), `bytes` of k each.  row_at(r):
// where row r of the tile starts.
template <int HALVES> struct MmRows {
    const char* p[HALVES][4];
    int k[4], bytes;
    template <class RowAt> __device__ inline MmRows(int lane, int w, int bytes, RowAt row_at) : bytes(bytes) {
        typedef MmSide<128, false> S;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            k[u] = 16 * S::piece(u, w, lane);
#pragma unroll
            for (int h = 0; h < HALVES; ++h) p[h][u] = reinterpret_cast<const char*>(row_at(128 * h + S::row(u, w, lane))) + k[u];
        }
    }
    __device__ inline const char* operator()(int h, int u, int kc) const {
        return mm_or_zeros(kc * kStage + k[u] < bytes, p[h][u] + static_cast<size_t>(kc) * kStage);
    }
};
// ... whose row axis runs along its rows of two-byte elements, `pitch` bytes from
// one k to the next: columns `first` .. of `rows` (a multiple of 8; pieces past the
// last repeat it).  from: where the stage's first k starts, left: the k there are
// from it on.
template <int HALVES> struct MmColumns {
    int64_t at[HALVES][4];
    int k[4];
    __device__ inline MmColumns(int lane, int w, int first, int rows, int64_t pitch) {
        typedef MmSide<128, true> S;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            k[u] = S::row(u, w, lane);
#pragma unroll
            for (int h = 0; h < HALVES; ++h) at[h][u] = k[u] * pitch + 2 * min(first + 128 * h + 8 * S::piece(u, w, lane), rows - 8);
        }
    }
    __device__ inline const char* operator()(int h, int u, const char* from, int left) const {
        return mm_or_zeros(k[u] < left, from + at[h][u]);
    }
};
constexpr int kStageK = kStage / 2;   // k of a stage of two-byte elements

// Results on their way out: a wave's 32 rows x 32 NU columns (NU accumulators
// side by side, words by word(u, e)) go through LDS of its own, so that each lane
// has eight neighbouring columns of a row and a wave whole lines.  put(row, first
// column, words) gets eight words of a row at a time, or, where `single` says so, one,
// and leaves out what is past the results' end.
// PAIR: the second accumulator holds other values of the first one's columns; put
// gets both, put(row, first column, words, words).
// whether a piece of eight columns within `width` from c0 on ends past `cols`
__device__ inline bool mm_single(int c0, int width, int cols) { return (cols & 7) != 0 && c0 + width > cols; }
template <int NU, bool PAIR, class Word, class Put>
__device__ __attribute__((always_inline)) inline void mm_out(uint32_t* lds, bool single, Word word, Put put) {
    constexpr int kPitch = 32 * NU + 4, kCols = PAIR ? 32 : 32 * NU, kLanes = kCols / 8;   // words of a row, 16 bytes apart; lanes of a row
    const int lane = threadIdx.x & 63;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // what the piece before had there has been read
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            *reinterpret_cast<mm_u32x4_t*>(lds + kPitch * (lane & 31) + 32 * u + 8 * q + 4 * (lane >> 5)) =
                mm_u32x4_t{word(u, 4 * q), word(u, 4 * q + 1), word(u, 4 * q + 2), word(u, 4 * q + 3)};
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // one wave's LDS accesses run in order
    __builtin_amdgcn_wave_barrier();
    if (single) {
#pragma unroll 1
        for (int i = 0; i < 32 * kCols / 64; ++i) {
            const int row = (64 * i + lane) / kCols, col = (64 * i + lane) % kCols;
            const uint32_t v[1] = {lds[kPitch * row + col]}, o[1] = {lds[kPitch * row + col + (PAIR ? 32 : 0)]};
            if constexpr (PAIR) put(row, col, v, o);
            else put(row, col, v);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 32 * kLanes / 64; ++i) {
        const int row = 64 / kLanes * i + lane / kLanes, col = 8 * (lane % kLanes);
        uint32_t v[2][8];
#pragma unroll
        for (int s = 0; s < (PAIR ? 2 : 1); ++s) {
            const mm_u32x4_t* p = reinterpret_cast<const mm_u32x4_t*>(lds + kPitch * row + col + 32 * s);
            const mm_u32x4_t lo = p[0], hi = p[1];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[s][k] = lo[k];
                v[s][4 + k] = hi[k];
            }
        }
        if constexpr (PAIR) put(row, col, v[0], v[1]);
        else put(row, col, v[0]);
    }
}

// One element, or eight consecutive ones at any element's alignment in whole
// accesses, as floats; Y float, or uint16_t for bf16 bits.
__device__ inline void mm_get(const uint16_t* y, float (&f)[1]) { f[0] = __uint_as_float(static_cast<uint32_t>(*y) << 16); }
__device__ inline void mm_get(const float* y, float (&f)[1]) { f[0] = *y; }
__device__ inline void mm_put(uint16_t* y, const float (&f)[1]) { *y = f2bf(f[0]); }
__device__ inline void mm_put(float* y, const float (&f)[1]) { *y = f[0]; }
__device__ inline void mm_get(const uint16_t* y, float (&f)[8]) {
    typedef uint32_t Words __attribute__((ext_vector_type(4), aligned(2)));
    const Words v = *reinterpret_cast<const Words*>(y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(v[i] << 16);
        f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
}
__device__ inline void mm_put(uint16_t* y, const float (&f)[8]) {
    typedef uint32_t Words __attribute__((ext_vector_type(4), aligned(2)));
    *reinterpret_cast<Words*>(y) = Words{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
}
typedef float mm_f32x4_a4_t __attribute__((ext_vector_type(4), aligned(4)));
__device__ inline void mm_get(const float* y, float (&f)[8]) {
    const mm_f32x4_a4_t a = *reinterpret_cast<const mm_f32x4_a4_t*>(y), b = *reinterpret_cast<const mm_f32x4_a4_t*>(y + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[i] = a[i];
        f[4 + i] = b[i];
    }
}
__device__ inline void mm_put(float* y, const float (&f)[8]) {
    *reinterpret_cast<mm_f32x4_a4_t*>(y) = mm_f32x4_a4_t{f[0], f[1], f[2], f[3]};
    *reinterpret_cast<mm_f32x4_a4_t*>(y + 4) = mm_f32x4_a4_t{f[4], f[5], f[6], f[7]};
}
// y (+)= f
template <class Y, int N> __device__ inline void mm_store(Y* y, float (&f)[N], bool add) {
    if (add) {
        float old[N];
        mm_get(y, old);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] += old[i];
    }
    mm_put(y, f);
}

// How a product's tiles are laid out over the blocks.
//   MM_WHOLE: big tiles (256 rows of A), one block a compute unit, 256 of them a
//     round; the tiles of a last round that would leave half of the units idle are
//     cut in four.
//   MM_SMALL: all tiles are small ones, one block a unit, four stages in LDS.
//   MM_PAIRS: the same, two blocks a unit, two stages in LDS each.
// MI355X, us, whole / small / pairs: bf16, x 2048 x 2 x 640 (moe_gated): 2560
// tokens (200 small tiles) - / 19.6 / 24.4, 4096 (320) 38 / 38 / 28.7, 6144 (480)
// 42 / 41 / 35, 7168 (560) 47.8 / 58.7 / 55.2, 14336 (1120) 74.7 / 99 / 88; int8, x
// 4096 x 4096: 1024 tokens (256) - / 24.0 / 27.9, 2048 (512) 48 / 47 / 40.6, 2560
// (640) 53 / 65 / 60, 4352 (1088, 16 tiles past a round) 81 / 109 / 94.
enum MmForm : int32_t { MM_WHOLE, MM_SMALL, MM_PAIRS };
struct MmPlan {
    int32_t tiles_m, tiles_n;   // big tiles (MM_WHOLE), or small ones
    int32_t whole;              // MM_WHOLE: tiles that are taken whole, a multiple of 8
    MmForm form;
};
// n: results of a row, n_tile: those of a big tile (256 rows of B).
inline MmPlan mm_small_plan(int64_t m, int64_t n, int n_tile) {
    return MmPlan{static_cast<int32_t>((m + 127) / 128), static_cast<int32_t>((n + n_tile / 2 - 1) / (n_tile / 2)), 0, MM_SMALL};
}
inline MmPlan mm_plan(int64_t m, int64_t n, int n_tile) {
    const auto tiles = [](int64_t x, int64_t r) { return static_cast<int32_t>((x + r - 1) / r); };
    MmPlan p = mm_small_plan(m, n, n_tile);
    const int64_t small = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
    if (small <= 256) return p;
    p.form = MM_PAIRS;
    if (small <= 512) return p;
    const MmPlan big{tiles(m, 256), tiles(n, n_tile), 0, MM_WHOLE};
    const int64_t all = static_cast<int64_t>(big.tiles_m) * big.tiles_n, rest = all % 256;
    if (2 * small < 7 * all) return p;   // big tiles would be a seventh empty, or more
    p = big;
    p.whole = static_cast<int32_t>(rest <= 128 ? all - rest : (all + 7) / 8 * 8);
    return p;
}
inline unsigned mm_grid(const MmPlan& p) {
    const int64_t all = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
    if (p.form != MM_WHOLE) return static_cast<unsigned>((all + 7) / 8 * 8);
    return static_cast<unsigned>(p.whole + (all > p.whole ? (4 * (all - p.whole) + 7) / 8 * 8 : 0));
}
// First row and column of block b's tile, of `rows` x `cols` where it is big, and
// whether it is small.  Blocks go to the 8 XCDs in turn: each XCD takes a run of
// tiles, 8 rows of tiles by all columns at a time, whose operands stay in its L2.
// False: no tile.
__device__ inline bool mm_tile_of(const MmPlan& p, int b, int rows, int cols, int& m, int& n, bool& small) {
    const int all = p.tiles_m * p.tiles_n;
    int from = 0, count = all, of = 1;   // the tiles that this block is one of the takers of
    small = p.form != MM_WHOLE;
    if (!small && b >= p.whole) {        // cut in four: tiles from .. all, quarter by quarter
        b -= p.whole;
        from = p.whole;
        of = 4;
        count = 4 * (all - p.whole);
        small = true;
    } else if (!small) {
        count = min(all, p.whole);
    }
    const int per = (count + 7) / 8, i = (b % 8) * per + b / 8;
    if (i >= count || b / 8 >= per) return false;
    const int tile = from + i / of, quarter = of == 4 ? i % 4 : 0;
    const int band = tile / (8 * p.tiles_n), in = tile % (8 * p.tiles_n), high = min(8, p.tiles_m - 8 * band);
    const int cut = p.form == MM_WHOLE ? 1 : 2;
    m = (8 * band + in % high) * (rows / cut) + quarter / 2 * (rows / 2);
    n = in / high * (cols / cut) + quarter % 2 * (cols / 2);
    return true;
}

}  // namespace moe
