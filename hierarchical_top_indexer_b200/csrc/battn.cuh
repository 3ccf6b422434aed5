// What the two block-attention kernels share (battn.cu: up to 128 (row, head)
// pairs per tile; battn_dec.cu: single rows with few heads): a CTA's place in
// the list of tiles, and tcgen05 forms.
#pragma once

#include "hisa_kernels.cuh"

namespace hisa {

constexpr float kBaGrow = 8.f;      // log2 of how far a maximum may outgrow its reference

// D[tmem] (+)= A[tmem] * B[smem]^T, f16 or bf16 inputs, fp32 accumulate.
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// The whole warp waits on a barrier (bounded); all lanes learn the outcome.
// A barrier that is through already costs one poll and a vote.  The rest is
// out of line, for the kernels wait in some twenty places and run partly cold;
// there lane 0 polls, and reads the timer that bounds the wait only once 64
// polls have failed, since a read takes longer than most of these waits.
static __device__ __noinline__ bool ba_wait_slow(uint32_t a, uint32_t parity, volatile int* abort_flag) {
    bool ok = true;
    if ((threadIdx.x & 31) == 0) {
        uint64_t t0 = 0;
#pragma unroll 1
        for (uint32_t it = 1; !mbar_try_wait(a, parity); ++it) {
            if ((it & 63u) != 0) continue;
            if (abort_flag && *abort_flag) {
                ok = false;
                break;
            }
            const uint64_t t = global_ns();
            if (t0 == 0) {
                t0 = t;
            } else if (t - t0 > kWaitLimitNs) {
                ok = false;
                break;
            }
        }
    }
    return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
}

__device__ __forceinline__ bool warp_wait_b(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    const uint32_t a = smem_addr(bar);
    if (__all_sync(0xffffffffu, mbar_try_wait(a, parity))) return true;
    const bool ok = ba_wait_slow(a, parity, abort_flag);
    // every lane has seen the phase, so that what came before it is visible to each
    if (ok) mbar_try_wait(a, parity);
    __syncwarp();
    return ok;
}

// 32 lanes x 32 bit, 4 consecutive columns per thread, without waiting.
__device__ __forceinline__ void tmem_ld4_nowait(uint32_t taddr, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld32_nowait(uint32_t taddr, uint32_t* r) {
    tmem_ld16_nowait(taddr, r);
    tmem_ld16_nowait(taddr + 16, r + 16);
}

// Issuing MMAs: a thread that builds a 64-bit descriptor per instruction in a
// divergent branch takes 120 to 170 cycles for each, more than the MMAs
// themselves (22 to 64 cycles at M = 128, K = 16).  So the whole warp runs the
// loop, one elected lane issues, the descriptors' upper halves are constants,
// and their lower halves are made known to be the same in every lane, which
// puts the additions on the uniform datapath.
__device__ __forceinline__ uint32_t uni(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// A descriptor's halves: start address and leading offset (bytes); stride
// offset (bytes), version 1 and swizzle mode (2: 128 bytes, 6: 32 bytes).
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lead) { return (saddr >> 4) | ((lead >> 4) << 16); }
__host__ __device__ constexpr uint32_t desc_hi(uint32_t stride, uint32_t swizzle) { return (stride >> 4) | (1u << 14) | (swizzle << 29); }
constexpr uint32_t kHi128 = desc_hi(1024, 2);   // both majors, 128-byte swizzle: 8-row groups 1 KB apart

__device__ __forceinline__ uint64_t desc64(uint32_t lo, uint32_t hi) { return static_cast<uint64_t>(hi) << 32 | lo; }

__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// A run's place: key head h, group g, tiles [t0, t0 + n) of the group's T.
// (p.direct: of the row g at position pos of sequence seq).
struct BaSeg {
    int h, g, t0, n, T;
    int seq, pos;
};

// Tiles of group g.  p.direct: a lone row over its whole prefix has the pieces
// 0, 1, 2, ... of its sequence, and needs no plan.  LONE: the kernel may be
// asked for that.
template <bool LONE>
__device__ __forceinline__ int ba_tiles(const BattnParams& p, int g, int* seq, int* pos) {
    if (!LONE || !p.direct) return __ldcg(p.tiles + g);
    *pos = query_position(p.q_seq, p.q_pos, p.len, p.batch, p.cap, g, seq);
    return *pos >= 0 ? *pos / 128 + 1 : 0;
}

__device__ __forceinline__ int ba_pieces(const BattnParams& p, const BaSeg& s) { return p.direct ? s.T : p.pieces[s.g]; }

// Piece e of the segment's group: {sequence << 8 | tokens of it that a row sees, piece}.
__device__ __forceinline__ int2 ba_piece(const BattnParams& p, const BaSeg& s, int e) {
    if (p.direct) return make_int2(s.seq << 8 | min(128, s.pos + 1 - 128 * e), e);
    return p.list[static_cast<size_t>(s.g) * p.lcap + e];
}

// The CTA's run [at, end) of all (key head, group, tile) slots; b0: tiles of
// the groups before g.
struct BaCursor {
    long long at, end;
    int tot, h, g, b0;

    template <bool LONE>
    __device__ __forceinline__ bool next(const BattnParams& p, BaSeg* s) {
        if (at >= end) return false;
        const int x = static_cast<int>(at - static_cast<long long>(h) * tot);
        int T = ba_tiles<LONE>(p, g, &s->seq, &s->pos);
        while (x >= b0 + T) {   // done with, or empty
            b0 += T;
            T = ba_tiles<LONE>(p, ++g, &s->seq, &s->pos);
        }
        s->h = h;
        s->g = g;
        s->t0 = x - b0;
        s->T = T;
        const long long left = end - at;
        s->n = left < b0 + T - x ? static_cast<int>(left) : b0 + T - x;
        at += s->n;
        if (x + s->n == tot) {
            ++h;
            g = b0 = 0;
        }
        return true;
    }
};

// Every thread of the CTA: adds the groups' tiles up and finds the run's
// start.  scratch: 40 ints of shared memory.  CTA 0 leaves the sums in tile0
// for join_kernel.
template <bool LONE>
__device__ __forceinline__ BaCursor ba_start(const BattnParams& p, int* scratch) {
    const int tid = threadIdx.x, n = blockDim.x, warp = tid >> 5, lane = tid & 31;
    const int per = (p.groups + n - 1) / n;
    const int g0 = min(tid * per, p.groups), g1 = min(g0 + per, p.groups);
    int sum = 0;
    int seq, pos;
    for (int g = g0; g < g1; ++g) {
        const int T = ba_tiles<LONE>(p, g, &seq, &pos);
        sum += T;
        if (LONE && p.direct && T == 0 && blockIdx.x == 0) set_status(p.status, HISA_DEV_BAD_QUERY);
    }
    int x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    BaCursor c;
    int before = x - sum;
    c.tot = 0;
    for (int w = 0; w < n / 32; ++w) {
        if (w < warp) before += scratch[w];
        c.tot += scratch[w];
    }
    // CTAs past the number of slots have none, so that no CTA between two others is idle
    const long long all = static_cast<long long>(c.tot) * p.Hkv;
    const long long ctas = min(static_cast<long long>(gridDim.x), all), i = min(static_cast<long long>(blockIdx.x), ctas);
    c.at = ctas > 0 ? all * i / ctas : 0;
    c.end = ctas > 0 ? all * min(i + 1, ctas) / ctas : 0;
    c.h = c.at < c.end ? static_cast<int>(c.at / c.tot) : 0;
    const int at = c.at < c.end ? static_cast<int>(c.at - static_cast<long long>(c.h) * c.tot) : 0;
    if (blockIdx.x == 0) {
        int b = before;
        if (tid == 0) p.tile0[0] = 0;
        for (int g = g0; g < g1; ++g) p.tile0[g + 1] = b += ba_tiles<LONE>(p, g, &seq, &pos);
    }
    if (sum > 0 && at >= before && at < before + sum) {
        int g = g0, b = before;
        for (int T; at >= b + (T = ba_tiles<LONE>(p, g, &seq, &pos)); ++g) b += T;
        scratch[32] = g;
        scratch[33] = b;
    }
    if (c.tot == 0 && tid == 0) scratch[32] = scratch[33] = 0;
    __syncthreads();
    c.g = scratch[32];
    c.b0 = scratch[33];
    __syncthreads();   // the scratch is free again
    return c;
}

}  // namespace hisa
