// Block attention of lone rows with few heads (decode: one row per sequence,
// up to 16 query heads per key head), the plan and the join being battn.cu's.
//
// With one row the 128-row MMA of battn.cu would hold 16 live rows, all of one
// warp: that warp's 2^x and its quarter of the SM bound the tile.  Here the
// tokens are the MMA's rows:
//   S^T [128 tokens, 16 heads] = K [128, d] Q^T     (A = K tile, B = Q)
//   P^T: every thread of the four softmax warps has a token and its 16 logits
//   O^T [d, 16 heads] += V^T [d, 128] P             (A = V tile, MN-major; B = P)
// so the softmax is spread over 128 threads, and an MMA reads its A tile once
// (256 cycles of shared memory) and little else.
//
// A head's maximum over the tokens lies across the threads, but it is needed
// only to keep P in range: the threads share a reference per head, and the
// warps tell each other per tile whether any logit passed it by 2^8.  Only
// then (the first tile of a segment, and a few more) are the maxima reduced
// and O^T rescaled.
//
// 4-bit rows: K goes from its codes straight into tensor memory as the MMA's A
// operand (a thread expands its token's row: no shared memory is written or
// read by the MMA for it); V, whose A operand is transposed, goes into shared
// memory.  The code tiles come by TMA with their 16-byte chunks swizzled, so
// that a row per lane reads without bank conflicts.
//
// Two CTAs per SM, so that one's softmax runs while the other's tiles load.
#include "battn.cuh"

namespace hisa {

namespace {

constexpr int kBdN = kBattnDecHeads;   // MMA columns: heads
constexpr int kBdWarpKd = 4;           // warps 4-7 expand K, 8-11 expand V (4-bit rows)
constexpr int kBdWarpVd = 8;

template <int D, bool FP4>
struct BdLayout {
    static constexpr int tile = 128 * D * 2;
    static constexpr int slots = FP4 ? 256 / D : 384 / D;   // operand tiles: V (4-bit rows), K and V in turn (bf16)
    static constexpr int raws = FP4 ? 256 / D : 0;          // stages of 4-bit rows
    static constexpr int raw_codes = 128 * D / 2, raw_scales = 128 * D / 16;
    static constexpr int raw = 2 * (raw_codes + raw_scales);
    static constexpr int ring = 0;
    static constexpr int raw0 = ring + slots * tile;
    static constexpr int p0 = raw0 + raws * raw;            // two P operands
    static constexpr int q = p0 + 2 * kBdN * 256;
    static constexpr int misc = q + kBdN * D * 2;
    static constexpr int refs = misc + 256;                 // [4 warps][16] references
    static constexpr int mx = refs + 256;                   // [4 warps][16] maxima, or sums
    static constexpr int c2 = mx + 256;                     // [2 segments][16] logit scales
    static constexpr int flags = c2 + 128;                  // [2][4]
    static constexpr int total = misc + 1024;
    static constexpr int warps = FP4 ? 14 : 6;              // softmax, (expanders,) load, MMA
    static constexpr int tmem_k = 0, tmem_s = 128, tmem_o = 160;   // columns of 256
};

__host__ __device__ constexpr uint32_t idesc_bd(bool f16, bool a_mn_major) {
    return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (a_mn_major ? (1u << 15) : 0u) |
           (static_cast<uint32_t>(kBdN >> 3) << 17) | ((128u >> 4) << 24);
}

// MN-major A operand of V: atoms of 64 dims x 8 tokens.  d = 64: the MMA's
// upper 64 rows re-read bytes 1 KB further on (their results are not used).
template <int D>
__device__ __forceinline__ uint64_t v_desc(uint32_t saddr) {
    constexpr uint32_t lead = D == 128 ? 16384 : 1024;
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(lead >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
    tmem_st16(taddr, r);
    tmem_st16(taddr + 16, r + 16);
}

// 16-byte chunk c of code row r, as the swizzled TMA load placed it.
template <int D>
__device__ __forceinline__ int code_chunk(int r, int c) {
    return r * (D / 2) + ((D == 128 ? c ^ ((r >> 1) & 3) : c ^ ((r >> 2) & 1)) << 4);
}

template <int D, bool FP4>
__global__ void __launch_bounds__(BdLayout<D, FP4>::warps * 32, 2)
    battn_dec_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map, const BattnParams p) {
    using L = BdLayout<D, FP4>;
    constexpr int kS = L::slots, kRaw = L::raws > 0 ? L::raws : 1, kWarps = L::warps;
    constexpr int kWarpLoad = kWarps - 2, kWarpMma = kWarps - 1;
    constexpr float kRef = FP4 ? 7.f : 0.f;   // log2 of the largest P of a fresh maximum
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::misc);
    uint64_t* full = bars;              // [<= 6] operand tile ready (bytes; 4-bit: 4 warps)
    uint64_t* empty = full + 6;         // [<= 6] its MMA is done (commit)
    uint64_t* rfull = empty + 6;        // [<= 4] 4-bit rows landed (bytes)
    uint64_t* rempty = rfull + 4;       // [<= 4] they have been expanded (8 warps)
    uint64_t* kfull = rempty + 4;       // [2] K expanded into TMEM (4 warps)
    uint64_t* sfull = kfull + 2;        // [2] S written, and the P V before the last done (commit)
    uint64_t* pfull = sfull + 2;        // [2] P written, O rescaled (4 warps)
    uint64_t* qfull = pfull + 2;        // query heads ready (bytes; 4-bit: 4 warps)
    uint64_t* qempty = qfull + 1;       // the segment's S MMAs are done (commit)
    uint64_t* pvdone = qempty + 1;      // a P V is done (commit)
    uint64_t* xbar = pvdone + 1;        // the warps' flags written (4 warps)
    uint64_t* mbar = xbar + 1;          // the warps' maxima, or sums, written (4 warps)
    uint64_t* done = mbar + 1;          // every MMA issued is done (commit)
    static_assert(32 * 8 <= L::refs - L::misc, "barriers");
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::flags + 32);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    static_assert(L::flags + 40 <= L::total, "misc area");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == kWarpMma) {
        if (lane == 0) {
            for (int i = 0; i < kS; ++i) {
                mbar_init(full + i, FP4 ? 4 : 1);
                mbar_init(empty + i, 1);
            }
            for (int i = 0; i < (FP4 ? kRaw : 0); ++i) {
                mbar_init(rfull + i, 1);
                mbar_init(rempty + i, 8);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(kfull + i, 4);
                mbar_init(sfull + i, 1);
                mbar_init(pfull + i, 4);
            }
            mbar_init(qfull, FP4 ? 4 : 1);
            mbar_init(qempty, 1);
            mbar_init(pvdone, 1);
            mbar_init(xbar, 4);
            mbar_init(mbar, 4);
            mbar_init(done, 1);
            *abort_flag = 0;
            fence_barrier_init();
        }
        __syncwarp();
        tmem_alloc(tmem_slot, 256);
        tmem_relinquish();
    }
    // columns without a head: zero queries
    for (int i = threadIdx.x; i < kBdN * D * 2 / 16; i += kWarps * 32)
        *reinterpret_cast<uint4*>(smem + L::q + i * 16) = make_uint4(0, 0, 0, 0);
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_dependency_wait();
    grid_launch_dependents();
    BaCursor cur = ba_start(p, reinterpret_cast<int*>(smem + L::refs));
    BaSeg sg;
    bool ok = true;

    if (warp < 4) {
        // --------------------------------------------------------- softmax
        const int tok = warp * 32 + lane;                 // of the tile; also the dim of O this thread has
        const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
        float* refs = reinterpret_cast<float*>(smem + L::refs) + warp * kBdN;
        float* mx = reinterpret_cast<float*>(smem + L::mx);
        const float* c2s = reinterpret_cast<const float*>(smem + L::c2);
        volatile int* flags = reinterpret_cast<volatile int*>(smem + L::flags);
        const int piece = tok / p.PB, in_piece = tok - piece * p.PB;
        const int chunk = (tok & 63) >> 3;
        uint32_t it = 0, seg = 0, xn = 0, mn = 0;
        while (ok && cur.next(p, &sg)) {
            const int2* list = p.list + static_cast<size_t>(sg.g) * p.lcap;
            const int np = p.pieces[sg.g];
            float l[kBdN];
#pragma unroll
            for (int h = 0; h < kBdN; ++h) l[h] = 0.f;
            if (lane < kBdN) refs[lane] = 0.f;   // set by the segment's first tile
            __syncwarp();
            int e = sg.t0 * p.S + piece;
            int nv = e < np ? list[e].x & 255 : 0;        // visible tokens of this thread's piece
            for (int j = 0; j < sg.n; ++j, ++it) {
                const uint32_t buf = it & 1;
                const bool vis = in_piece < nv;
                const int tail = nv < p.PB;
                e += p.S;
                const int nv_next = e < np ? list[e].x & 255 : 0;
                if (!(ok = warp_wait_b(sfull + buf, (it >> 1) & 1, abort_flag))) break;
                tc_fence_after();
                float z[kBdN];
                {
                    uint32_t v[kBdN];
                    tmem_ld16_nowait(tmem + lane_off + L::tmem_s + buf * kBdN, v);
                    tmem_ld_wait();
                    bool over = false;
#pragma unroll
                    for (int q = 0; q < kBdN / 4; ++q) {
                        const float4 r4 = *reinterpret_cast<const float4*>(refs + 4 * q);
                        float4 c4 = make_float4(p.scale_log2, p.scale_log2, p.scale_log2, p.scale_log2);
                        if (FP4) c4 = *reinterpret_cast<const float4*>(c2s + (seg & 1) * kBdN + 4 * q);
                        const float r[4] = {r4.x, r4.y, r4.z, r4.w}, c[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            z[4 * q + i] = vis ? __uint_as_float(v[4 * q + i]) * c[i] - r[i] : -INFINITY;
                            over |= z[4 * q + i] > kRef + kBaGrow;
                        }
                    }
                    over = __any_sync(0xffffffffu, over);
                    if (lane == 0) {
                        flags[buf * 4 + warp] = over;
                        mbar_arrive(xbar);
                    }
                    if (!(ok = warp_wait_b(xbar, xn & 1, abort_flag))) break;
                    ++xn;
                }
                const int4 f = *reinterpret_cast<const int4*>(smem + L::flags + buf * 16);
                if (j == 0 || (f.x | f.y | f.z | f.w)) {
                    // the maxima of all heads over the tile, and new references
                    float mine = 0.f;
#pragma unroll
                    for (int h = 0; h < kBdN; ++h) {
                        float m = z[h];
#pragma unroll
                        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                        if (lane == h) mine = m;
                    }
                    if (lane < kBdN) mx[warp * kBdN + lane] = mine;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(mbar);
                    if (!(ok = warp_wait_b(mbar, mn & 1, abort_flag))) break;
                    ++mn;
                    if (j > 0) {
                        if (!(ok = warp_wait_b(pvdone, (it - 1) & 1, abort_flag))) break;
                        tc_fence_after();
                    }
                    float up = 0.f;   // lane h: how far head h's reference moves
                    if (lane < kBdN) {
                        const float m = fmaxf(fmaxf(mx[lane], mx[kBdN + lane]), fmaxf(mx[2 * kBdN + lane], mx[3 * kBdN + lane]));
                        if (j == 0) up = m > -INFINITY ? m - kRef : 0.f;
                        else up = fmaxf(m - kRef, 0.f);
                        refs[lane] += up;
                    }
                    __syncwarp();
                    uint32_t o[kBdN];
                    if (j > 0) {
                        tmem_ld16_nowait(tmem + lane_off + L::tmem_o, o);
                        tmem_ld_wait();
                    }
#pragma unroll
                    for (int h = 0; h < kBdN; ++h) {
                        const float u = __shfl_sync(0xffffffffu, up, h);
                        const float a = ex2_approx(-u);
                        z[h] -= u;
                        l[h] *= a;
                        if (j > 0) o[h] = __float_as_uint(__uint_as_float(o[h]) * a);
                    }
                    if (j > 0) {
                        tmem_st16(tmem + lane_off + L::tmem_o, o);
                        tmem_st_wait();
                    }
                }
                const uint32_t prow = smem_addr(smem + L::p0) + buf * (kBdN * 256) + (tok >> 6) * (kBdN * 128) + (tok & 7) * 2;
#pragma unroll
                for (int h = 0; h < kBdN; h += 2) {
                    const float a = ex2_approx(z[h]), b = ex2_approx(z[h + 1]);
                    l[h] += a;
                    l[h + 1] += b;
                    const uint32_t w = FP4 ? pack_f16(a, b) : pack_bf16(a, b);
                    asm volatile("st.shared.u16 [%0], %1;" ::"r"(prow + h * 128 + ((chunk ^ (h & 7)) << 4)),
                                 "h"(static_cast<unsigned short>(w))
                                 : "memory");
                    asm volatile("st.shared.u16 [%0], %1;" ::"r"(prow + (h + 1) * 128 + ((chunk ^ ((h + 1) & 7)) << 4)),
                                 "h"(static_cast<unsigned short>(w >> 16))
                                 : "memory");
                }
                if (!FP4 && __any_sync(0xffffffffu, tail)) {
                    // V rows past the last visible token: zeros, for 0 * NaN is NaN
                    const uint32_t vi = 2 * it + 1;
                    if (!(ok = warp_wait_b(full + vi % kS, (vi / kS) & 1, abort_flag))) break;
                    if (!vis) {
                        uint8_t* v = smem + L::ring + (vi % kS) * L::tile + tok * 128;
                        for (int a = 0; a < D / 64; ++a)
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                *reinterpret_cast<uint4*>(v + a * 16384 + c * 16) = make_uint4(0, 0, 0, 0);
                    }
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(pfull + buf);
                nv = nv_next;
            }
            if (!ok) break;
            // the heads' sums over the threads, and the output
#pragma unroll
            for (int h = 0; h < kBdN; ++h) {
#pragma unroll
                for (int o = 16; o; o >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], o);
            }
            if (!(ok = warp_wait_b(pvdone, (it - 1) & 1, abort_flag))) break;
            tc_fence_after();
#pragma unroll
            for (int h = 0; h < kBdN; ++h)
                if (lane == h) mx[warp * kBdN + h] = l[h];
            __syncwarp();
            if (lane == 0) mbar_arrive(mbar);
            if (!(ok = warp_wait_b(mbar, mn & 1, abort_flag))) break;
            ++mn;
            const bool whole = sg.n == sg.T;
            const int slot = 2 * blockIdx.x + (sg.t0 == 0 ? 1 : 0);
            const size_t orow = static_cast<size_t>(sg.g) * p.Hq + sg.h * p.G;
            uint32_t o[kBdN];
            tmem_ld16_nowait(tmem + lane_off + L::tmem_o, o);
            tmem_ld_wait();
            float mysum = 0.f;
            if (lane < kBdN) mysum = (mx[lane] + mx[kBdN + lane]) + (mx[2 * kBdN + lane] + mx[3 * kBdN + lane]);
            const float scale = mysum > 0.f ? p.out_mul / mysum : 0.f;
#pragma unroll
            for (int h = 0; h < kBdN; ++h) {
                const float sc = __shfl_sync(0xffffffffu, scale, h);
                if (h < p.G && tok < D) {
                    if (whole) {
                        const uint32_t w = pack_bf16(__uint_as_float(o[h]) * sc, 0.f);
                        p.out[(orow + h) * D + tok] = static_cast<uint16_t>(w);
                    } else {
                        p.part_o[(static_cast<size_t>(slot) * kBdN + h) * D + tok] = __uint_as_float(o[h]);
                    }
                }
            }
            if (warp == 0 && lane < p.G) {
                if (!whole) p.part_ml[slot * kBdN + lane] = make_float2(refs[lane], mysum);
                else if (p.lse) p.lse[orow + lane] = (refs[lane] + log2f(mysum)) * 0.6931471805599453f;
            }
            __syncwarp();
            ++seg;
        }
    } else if (FP4 && warp < kBdWarpVd) {
        // -------------------------------------------- queries; K into TMEM
        const int dw = warp - kBdWarpKd;
        const int row = dw * 32 + lane;
        uint32_t it = 0, seg = 0;
        while (ok && cur.next(p, &sg)) {
            if (seg > 0 && !(ok = warp_wait_b(qempty, (seg - 1) & 1, abort_flag))) break;
            for (int h = dw; h < p.G; h += 4) {
                // scaled by a power of two so that the largest element lies in [2^14, 2^15):
                // in f16 then no element loses more than 2^-40 of that
                constexpr int E = D / 32;
                const uint16_t* src = p.q + (static_cast<size_t>(sg.g) * p.Hq + sg.h * p.G + h) * D + lane * E;
                uint32_t w[2] = {*reinterpret_cast<const uint32_t*>(src), 0u};
                if (E == 4) w[1] = *reinterpret_cast<const uint32_t*>(src + 2);
                uint32_t m = max(max(w[0] & 0x7FFF0000u, (w[0] & 0x7FFFu) << 16), max(w[1] & 0x7FFF0000u, (w[1] & 0x7FFFu) << 16));
                m = __reduce_max_sync(0xffffffffu, m);
                const int ex = m > 0 ? min(14 - ilogbf(__uint_as_float(m)), 120) : 0;
                const float up = __int_as_float((ex + 127) << 23);
                uint32_t f[2];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    f[i] = pack_f16(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xFFFF0000u) * up);
                const int byte = lane * E * 2;
                uint8_t* dst = smem + L::q + (byte >> 7) * (kBdN * 128) + h * 128 + ((((byte & 127) >> 4) ^ (h & 7)) << 4) + (byte & 15);
                *reinterpret_cast<uint32_t*>(dst) = f[0];
                if (E == 4) *reinterpret_cast<uint32_t*>(dst + 4) = f[1];
                if (lane == 0) reinterpret_cast<float*>(smem + L::c2)[(seg & 1) * kBdN + h] = ldexpf(p.scale_log2, -ex);
            }
            if (dw == 0 && lane >= p.G && lane < kBdN) reinterpret_cast<float*>(smem + L::c2)[(seg & 1) * kBdN + lane] = 0.f;
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(qfull);
            ++seg;
            for (int j = 0; j < sg.n; ++j, ++it) {
                const uint32_t rs = it % kRaw, buf = it & 1;
                if (!(ok = warp_wait_b(rfull + rs, (it / kRaw) & 1, abort_flag))) break;
                const uint8_t* raw = smem + L::raw0 + rs * L::raw;
                // S of tile it - 2, the last reader of this TMEM buffer
                if (it >= 2 && !(ok = warp_wait_b(sfull + buf, ((it >> 1) - 1) & 1, abort_flag))) break;
                tc_fence_after();
                const uint32_t tk = tmem + (static_cast<uint32_t>(dw * 32) << 16) + L::tmem_k + buf * (D / 2);
                uint32_t sc[D / 32];   // two scales each
                if (D == 128) {
                    const uint2 s2 = *reinterpret_cast<const uint2*>(raw + 2 * L::raw_codes + row * 8);
                    sc[0] = s2.x & 0xFFFF;
                    sc[1] = s2.x >> 16;
                    sc[D / 32 - 2] = s2.y & 0xFFFF;
                    sc[D / 32 - 1] = s2.y >> 16;
                } else {
                    const uint32_t s1 = *reinterpret_cast<const uint32_t*>(raw + 2 * L::raw_codes + row * 4);
                    sc[0] = s1 & 0xFFFF;
                    sc[1] = s1 >> 16;
                }
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    const uint4 x = *reinterpret_cast<const uint4*>(raw + code_chunk<D>(row, c));
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                    const uint32_t sh = e4m3x2_to_f16(sc[c]);
                    const __half2 s0 = __half2half2(__ushort_as_half(static_cast<unsigned short>(sh)));
                    const __half2 s1 = __half2half2(__ushort_as_half(static_cast<unsigned short>(sh >> 16)));
                    uint32_t r[16];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t f[4];
                        e2m1x8_to_f16(w[q], f);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const __half2 pr = __hmul2(*reinterpret_cast<const __half2*>(&f[i]), q < 2 ? s0 : s1);
                            r[4 * q + i] = *reinterpret_cast<const uint32_t*>(&pr);
                        }
                    }
                    tmem_st16(tk + c * 16, r);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(rempty + rs);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(kfull + buf);
            }
        }
    } else if (FP4 && warp < kWarpLoad) {
        // ------------------------------------------- V into shared memory
        const int dw = warp - kBdWarpVd;
        constexpr int kCh = D / 32;       // 16-byte chunks of codes (32 elements) per row
        constexpr int kRows = 32 / kCh;   // rows a warp expands at a time
        const int ch = lane % kCh, rl = lane / kCh;
        uint32_t it = 0;
        while (ok && cur.next(p, &sg)) {
            const int2* list = p.list + static_cast<size_t>(sg.g) * p.lcap;
            const int np = p.pieces[sg.g];
            const int r = dw * 32 + lane, s = r / p.PB;
            int e = sg.t0 * p.S + s;
            bool sees = e < np && r - s * p.PB < (list[e].x & 255);
            for (int j = 0; j < sg.n; ++j, ++it) {
                const uint32_t seen = __ballot_sync(0xffffffffu, sees);   // the other rows become zeros
                e += p.S;
                sees = j + 1 < sg.n && e < np && r - s * p.PB < (list[e].x & 255);
                const uint32_t rs = it % kRaw, slot = it % kS;
                if (!(ok = warp_wait_b(rfull + rs, (it / kRaw) & 1, abort_flag))) break;
                if (it >= kS && !(ok = warp_wait_b(empty + slot, (it / kS - 1) & 1, abort_flag))) break;
                const uint8_t* raw = smem + L::raw0 + rs * L::raw;
                uint8_t* dst = smem + L::ring + slot * L::tile;
#pragma unroll
                for (int i = 0; i < kCh; ++i) {
                    const int rw = i * kRows + rl, row = dw * 32 + rw;
                    uint4 x = *reinterpret_cast<const uint4*>(raw + L::raw_codes + code_chunk<D>(row, ch));
                    uint32_t sch = e4m3x2_to_f16(*reinterpret_cast<const uint16_t*>(raw + 2 * L::raw_codes + L::raw_scales +
                                                                                   row * (D / 16) + ch * 2));
                    if (!((seen >> rw) & 1u)) {
                        x = make_uint4(0, 0, 0, 0);
                        sch = 0;
                    }
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                    const __half2 s0 = __half2half2(__ushort_as_half(static_cast<unsigned short>(sch)));
                    const __half2 s1 = __half2half2(__ushort_as_half(static_cast<unsigned short>(sch >> 16)));
                    // the order of the four stores keeps a quarter warp's rows and chunks on different banks
                    const int turn = (ch >> 1) * 2;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int qq = q ^ turn;
                        uint32_t f[4];
                        e2m1x8_to_f16(turn ? w[q ^ 2] : w[q], f);
                        const __half2 sh = qq < 2 ? s0 : s1;
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const __half2 pr = __hmul2(*reinterpret_cast<const __half2*>(&f[z]), sh);
                            f[z] = *reinterpret_cast<const uint32_t*>(&pr);
                        }
                        *reinterpret_cast<uint4*>(dst + sw128_off(row, ch * 4 + qq)) = make_uint4(f[0], f[1], f[2], f[3]);
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(rempty + rs);
                    mbar_arrive(full + slot);
                }
            }
        }
    } else if (warp == kWarpLoad) {
        // ------------------------------------------------------------ load
        // Lane s < S loads piece s of each tile.
        uint32_t it = 0, seg = 0, issued = 0;
        while (ok && cur.next(p, &sg)) {
            const int2* list = p.list + static_cast<size_t>(sg.g) * p.lcap;
            const int np = p.pieces[sg.g];
            if (!FP4) {
                if (seg > 0 && !(ok = warp_wait_b(qempty, (seg - 1) & 1, abort_flag))) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(qfull, static_cast<uint32_t>(p.G * D * 2));
#pragma unroll
                    for (int a = 0; a < D / 64; ++a)
                        tma_load_3d(smem + L::q + a * (kBdN * 128), &q_map, qfull, a * 64, sg.h * p.G, sg.g);
                }
                __syncwarp();
            }
            ++seg;
            int e = sg.t0 * p.S + lane;
            const bool mine = lane < p.S;
            int2 pc = mine && e < np ? list[e] : make_int2(-1, 0);
            for (int j = 0; j < sg.n; ++j, ++it) {
                const int2 now = pc;
                e += p.S;
                pc = mine && j + 1 < sg.n && e < np ? list[e] : make_int2(-1, 0);
                const bool have = now.x >= 0;
                const int bh = have ? (now.x >> 8) * p.Hkv + sg.h : 0;
                if (!FP4) {
                    const int rowc = have ? now.y * p.PB : p.cap;   // a missing piece: rows past the end, zeros
                    for (int kv = 0; kv < 2; ++kv) {
                        const uint32_t n = 2 * it + kv, slot = n % kS;
                        if (n >= kS && !(ok = warp_wait_b(empty + slot, (n / kS - 1) & 1, abort_flag))) break;
                        if (lane == 0) mbar_arrive_expect_tx(full + slot, L::tile);
                        issued = n + 1;
                        __syncwarp();
                        if (mine) {
                            uint8_t* dst = smem + L::ring + slot * L::tile + lane * p.PB * 128;
#pragma unroll
                            for (int a = 0; a < D / 64; ++a) {
                                if (kv) tma_load_3d(dst + a * 16384, &v_map, full + slot, a * 64, rowc, bh);
                                else tma_load_3d(dst + a * 16384, &k_map, full + slot, a * 64, rowc, bh);
                            }
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                } else {
                    const uint32_t slot = it % kRaw;
                    if (it >= kRaw && !(ok = warp_wait_b(rempty + slot, (it / kRaw - 1) & 1, abort_flag))) break;
                    const int row = now.y * p.PB;
                    const int rows = have ? min(p.PB, p.cap - row) : 0;
                    const uint32_t bytes = have ? p.PB * D + rows * (D / 8) : 0;
                    const uint32_t all = __reduce_add_sync(0xffffffffu, bytes);
                    if (lane == 0) mbar_arrive_expect_tx(rfull + slot, all);
                    issued = it + 1;
                    __syncwarp();
                    if (have) {
                        const size_t r0 = static_cast<size_t>(bh) * p.cap + row;
                        uint8_t* dst = smem + L::raw0 + slot * L::raw;
                        const int at = lane * p.PB;
                        tma_load_3d(dst + at * (D / 2), &k_map, rfull + slot, 0, row, bh);
                        tma_load_3d(dst + L::raw_codes + at * (D / 2), &v_map, rfull + slot, 0, row, bh);
                        bulk_load(dst + 2 * L::raw_codes + at * (D / 16), p.k_scale + r0 * (D / 16), rows * (D / 16), rfull + slot);
                        bulk_load(dst + 2 * L::raw_codes + L::raw_scales + at * (D / 16), p.v_scale + r0 * (D / 16),
                                  rows * (D / 16), rfull + slot);
                    }
                    __syncwarp();
                }
            }
        }
        if (!ok && lane == 0) {
            // the copies in flight land before the CTA gives up its shared memory
            volatile int keep_waiting = 0;
            *abort_flag = 1;
            constexpr uint32_t n = FP4 ? kRaw : kS;
            if (!FP4 && seg > 0) mbar_wait(qfull, (seg - 1) & 1, &keep_waiting);
            for (uint32_t i = issued > n ? issued - n : 0; i < issued; ++i)
                mbar_wait((FP4 ? rfull : full) + i % n, (i / n) & 1, &keep_waiting);
        }
    } else {
        // ------------------------------------------------------------- MMA
        if (lane == 0) {
            constexpr uint32_t id_s = idesc_bd(FP4, false), id_o = idesc_bd(FP4, true);
            const uint32_t bq = smem_addr(smem + L::q), ring = smem_addr(smem + L::ring), bp = smem_addr(smem + L::p0);
            uint32_t it = 0, seg = 0;
            auto issue_s = [&](uint32_t n) -> bool {   // S of tile n of the run
                const uint32_t buf = n & 1, slot = (2 * n) % kS;
                if (FP4 ? !mbar_wait(kfull + buf, (n >> 1) & 1, abort_flag) : !mbar_wait(full + slot, (2 * n / kS) & 1, abort_flag))
                    return false;
                tc_fence_after();
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint64_t q = sw128_kmajor_desc(bq + (s >> 2) * (kBdN * 128) + (s & 3) * 32);
                    if (FP4)
                        umma_f16_ts(tmem + L::tmem_s + buf * kBdN, tmem + L::tmem_k + buf * (D / 2) + s * 8, q, id_s, s > 0);
                    else
                        umma_bf16(tmem + L::tmem_s + buf * kBdN,
                                  sw128_kmajor_desc(ring + slot * L::tile + (s >> 2) * 16384 + (s & 3) * 32), q, id_s, s > 0);
                }
                if (!FP4) umma_commit(empty + slot);
                umma_commit(sfull + buf);
                return true;
            };
            while (ok && cur.next(p, &sg)) {
                if (!(ok = mbar_wait(qfull, seg & 1, abort_flag))) break;
                tc_fence_after();
                ok = issue_s(it);
                for (int j = 0; j < sg.n && ok; ++j, ++it) {
                    if (j + 1 < sg.n) ok = issue_s(it + 1);
                    else umma_commit(qempty);
                    const uint32_t buf = it & 1, n = FP4 ? it : 2 * it + 1, slot = n % kS;
                    ok = ok && mbar_wait(pfull + buf, (it >> 1) & 1, abort_flag) && mbar_wait(full + slot, (n / kS) & 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        umma_bf16(tmem + L::tmem_o, v_desc<D>(ring + slot * L::tile + s * 2048),
                                  sw128_kmajor_desc(bp + buf * (kBdN * 256) + (s >> 2) * (kBdN * 128) + (s & 3) * 32), id_o,
                                  (j > 0 || s > 0) ? 1u : 0u);
                    umma_commit(empty + slot);
                    umma_commit(pvdone);
                }
                ++seg;
            }
            if (!ok) *abort_flag = 1;
            // every MMA done before TMEM is freed (a bounded wait that an abort does not cut short)
            volatile int keep_waiting = 0;
            umma_commit(done);
            if (!mbar_wait(done, 0, &keep_waiting)) ok = false;
        }
        __syncwarp();
    }
    if (!ok && lane == 0) {
        *abort_flag = 1;
        set_status(p.status, HISA_DEV_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

template <int D, bool FP4>
cudaError_t launch_typed(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm, const BattnParams& p, int grid,
                         cudaStream_t s) {
    using L = BdLayout<D, FP4>;
    cudaError_t e = smem_limit(reinterpret_cast<const void*>(battn_dec_kernel<D, FP4>), L::total);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(L::warps * 32);
    cfg.dynamicSmemBytes = L::total;
    return cudaLaunchKernelEx(&cfg, battn_dec_kernel<D, FP4>, qm, km, vm, p);
}

}  // namespace

cudaError_t launch_battn_dec(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm, const BattnParams& p, bool fp4,
                             int grid, cudaStream_t s) {
    if (fp4) return p.d == 128 ? launch_typed<128, true>(qm, km, vm, p, grid, s) : launch_typed<64, true>(qm, km, vm, p, grid, s);
    return p.d == 128 ? launch_typed<128, false>(qm, km, vm, p, grid, s) : launch_typed<64, false>(qm, km, vm, p, grid, s);
}

}  // namespace hisa
