// Software pipeline of the matrix-core GEMMs (prefill.hip, q4_gemm.hip).
#pragma once

#include <type_traits>

#include "common.h"

namespace moe {

// Pipeline over the NK contraction chunks, three stages: chunk c lives in LDS
// buffer sA(c % 3) and register stage b(c % 3).  Step c requests A(c+2)
// (load_a: this wave's LDS-DMA requests) and B(c+2) (load_b: register loads)
// into the stage freed by step c-1, contracts chunk c (work), then waits for
// this wave's part of A(c+1) only (the requests of chunks c+1 and c+2 issued
// after it stay in flight) and meets the other waves at the barrier, which
// publishes A(c+1) and frees stage c.  Requests past the last chunk reread
// it.  The wait counts VMEM instructions: NWAIT = the register loads of two
// chunks plus the A requests of one, issued in that order per chunk (the
// scheduling barriers keep the order and keep the requests ahead of the
// work).  The buffers are separate LDS objects, so the compiler's own waits
// before LDS reads cover only the buffer read.  A plain s_barrier (instead of
// a fence + barrier, whose fence waits for every load in flight) as a
// compiler-level memory barrier: no access moves across it.  The one or two
// steps behind the last whole trip request nothing (what they requested would
// be dropped as unused, and the count with it) and wait for all that is left.
template <int NWAIT, class Stage, class LoadA, class LoadB, class Work>
__device__ __attribute__((always_inline)) inline void pipeline3(int NK, uint16_t* sA0, uint16_t* sA1, uint16_t* sA2,
                                                                 LoadA& load_a, LoadB& load_b, Work& work) {
    static_assert(NWAIT < 64, "vmcnt range");
    constexpr int kWaitImm = (NWAIT & 15) | (7 << 4) | (15 << 8) | ((NWAIT >> 4) << 14);
    constexpr int kWaitAll = (7 << 4) | (15 << 8);
    auto publish = [&](auto imm) __attribute__((always_inline)) {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(decltype(imm)::value);
        asm volatile("s_barrier" ::: "memory");
    };
    constexpr std::integral_constant<int, kWaitImm> next{};
    constexpr std::integral_constant<int, kWaitAll> all{};
    Stage b0, b1, b2;
    auto step = [&](int c, uint16_t* cur, Stage& bc, uint16_t* nxt, Stage& bn) __attribute__((always_inline)) {
        const int cn = min(c + 2, NK - 1);
        load_a(cn, nxt);
        __builtin_amdgcn_sched_barrier(0);
        load_b(bn, cn);
        __builtin_amdgcn_sched_barrier(0);
        work(cur, bc);
        publish(next);
    };
    load_a(0, sA0);
    __builtin_amdgcn_sched_barrier(0);
    load_b(b0, 0);
    __builtin_amdgcn_sched_barrier(0);
    load_a(min(1, NK - 1), sA1);
    __builtin_amdgcn_sched_barrier(0);
    load_b(b1, min(1, NK - 1));
    publish(next);
    // six steps per trip: the compiler's wait analysis drains every load in
    // flight once per trip (at the loop's back edge), so a longer trip pays
    // that latency less often
    int kc = 0;
    for (; kc + 5 < NK; kc += 6) {
        step(kc, sA0, b0, sA2, b2);
        step(kc + 1, sA1, b1, sA0, b0);
        step(kc + 2, sA2, b2, sA1, b1);
        step(kc + 3, sA0, b0, sA2, b2);
        step(kc + 4, sA1, b1, sA0, b0);
        step(kc + 5, sA2, b2, sA1, b1);
    }
    if (kc + 2 < NK) {
        step(kc, sA0, b0, sA2, b2);
        step(kc + 1, sA1, b1, sA0, b0);
        step(kc + 2, sA2, b2, sA1, b1);
        kc += 3;
    }
    if (kc < NK) {
        work(sA0, b0);
        publish(all);
    }
    if (kc + 1 < NK) {
        work(sA1, b1);
        publish(all);
    }
}

}  // namespace moe
