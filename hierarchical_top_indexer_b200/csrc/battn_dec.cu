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
// Roles: softmax (a set of four warps; 4-bit rows: two sets, a tile each in
// turn, with accumulators of their own that are merged at a segment's end), a
// warp that loads, one that issues S, one that issues P V; 4-bit rows: four
// warps that expand K and two teams of four that expand V.  bf16 rows: 112 KB,
// two CTAs per SM, a ring of three 32 KB tiles each.  4-bit rows: one CTA per
// SM, for its bytes are a quarter and the chain from row to output is longer:
// six 18 KB stages of rows, four K buffers, three V tiles.
//
// Bound (d = 128): bf16 rows by HBM, 64 rows of 8192 kept keys and 8 key heads
// in 338 to 342 us, 6.3 TB/s.  4-bit rows: 16 prefixes of about 115K keys and 4
// key heads in 279 to 302 us, 3.5 to 3.8 TB/s; 211 us of 277 remained when
// neither the expanding nor the softmax did anything, so the hand-over from
// stage to stage bounds it (shared memory moves about 110 KB a tile, 860 of the
// 1400 cycles a tile takes).  At 80 registers for 23 warps it spills 140 bytes
// (312 loaded); bf16 rows have 114 and spill none.
#include "battn.cuh"

namespace hisa {

namespace {

constexpr int kBdN = kBattnDecHeads;   // MMA columns: heads

template <int D, bool FP4>
struct BdLayout {
    static constexpr int sets = FP4 ? 2 : 1;                // softmax sets of four warps; tiles alternate between them
    static constexpr int sbufs = 4;                         // S buffers (and K, 4-bit rows) in TMEM
    static constexpr int bufs = 2 * sets;                   // P buffers
    static constexpr int tile = 128 * D * 2;
    // operand tiles: V (4-bit rows; fewer than P buffers, so that a tile's V cannot arrive at
    // the barrier of an unfinished one), K and V in turn (bf16)
    static constexpr int slots = FP4 ? 3 : 384 / D;
    static_assert(FP4 || 6 % slots == 0, "a slot holds a K (or a V) every sixth tile");
    static constexpr int raws = FP4 ? (D == 128 ? 6 : 8) : 0;   // stages of 4-bit rows
    static constexpr int raw_codes = 128 * D / 2, raw_scales = 128 * D / 16;
    static constexpr int raw = 2 * (raw_codes + raw_scales);
    static constexpr int ring = 0;
    static constexpr int raw0 = ring + slots * tile;
    static constexpr int p0 = raw0 + raws * raw;            // P operands
    static constexpr int q = p0 + bufs * kBdN * 256;
    static constexpr int misc = q + kBdN * D * 2;           // barriers
    static constexpr int refs = misc + 512;                 // [4 * sets warps][16] references
    static constexpr int mx = refs + sets * 256;            // [4 * sets warps][16] maxima
    static constexpr int fin = mx + sets * 256;             // [2 segments][sets][4 warps' sums, references][16]
    static constexpr int c2 = fin + 2 * sets * 320;         // [2 segments][16] logit scales
    static constexpr int flags = c2 + 128;                  // [bufs][4]
    static constexpr int slot = flags + bufs * 16;          // tensor memory address, abort flag
    static constexpr int total = slot + 16;
    static_assert(total <= (FP4 ? 232448 : 115712), "shared memory of one (bf16: half an) SM");
    static constexpr int ctas = FP4 ? 1 : 2;                // per SM
    static constexpr int warp_kd = 4 * sets;                // K expanders (4-bit rows), then V expanders
    static constexpr int warp_vd = warp_kd + (FP4 ? 4 : 0);
    static constexpr int warp_load = warp_vd + (FP4 ? 8 : 0);
    static constexpr int warp_s = warp_load + 1;            // issues the S MMAs
    static constexpr int warp_pv = warp_s + 1;              // issues the P V MMAs
    static constexpr int warps = warp_pv + 1;
    static constexpr int tmem_cols = FP4 ? 512 : 256;
    static constexpr int tmem_k = 0, tmem_s = FP4 ? 256 : 0, tmem_o = tmem_s + sbufs * kBdN;   // columns
};

__host__ __device__ constexpr uint32_t idesc_bd(bool f16, bool a_mn_major, bool b_mn_major) {
    return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (a_mn_major ? (1u << 15) : 0u) | (b_mn_major ? (1u << 16) : 0u) |
           (static_cast<uint32_t>(kBdN >> 3) << 17) | ((128u >> 4) << 24);
}

// P as the MN-major B operand in the 32-byte swizzled layout: a token's 16
// heads are 32 contiguous bytes, their two 16-byte halves swapped in every
// other group of four tokens; 8-token groups 256 B apart.
constexpr uint32_t kHiP = desc_hi(256, 6);

// 16-byte chunk c of code row r, as the swizzled TMA load placed it.
template <int D>
__device__ __forceinline__ int code_chunk(int r, int c) {
    return r * (D / 2) + ((D == 128 ? c ^ ((r >> 1) & 3) : c ^ ((r >> 2) & 1)) << 4);
}

template <int D, bool FP4>
__global__ void __launch_bounds__(BdLayout<D, FP4>::warps * 32, BdLayout<D, FP4>::ctas)
    battn_dec_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map, const BattnParams p) {
    using L = BdLayout<D, FP4>;
    constexpr int kS = L::slots, kRaw = L::raws > 0 ? L::raws : 1, kSets = L::sets, kBufs = L::bufs, kSB = L::sbufs;
    constexpr float kRef = FP4 ? 7.f : 0.f;   // log2 of the largest P of a fresh maximum
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::misc);
    // A wait names a phase by its parity alone, so a role may wait only on barriers whose every
    // phase it waits for: a slot that holds K and V in turn has a barrier for each.  (With one
    // for both, S of a tile took the arrival of the V before it for its own K.)
    uint64_t* kland = bars;             // [kS] the slot's K landed (bytes; bf16)
    uint64_t* vland = kland + kS;       // [kS] the slot's V landed
    uint64_t* empty = vland + kS;       // [kS] the slot's MMA is done (commit)
    uint64_t* rfull = empty + kS;       // [kRaw] 4-bit rows landed (bytes)
    uint64_t* rempty = rfull + kRaw;    // [kRaw] they have been expanded (8 warps)
    uint64_t* kfull = rempty + kRaw;    // [kSB] K expanded into TMEM (4 warps)
    uint64_t* sfull = kfull + kSB;      // [kSB] S written (commit)
    uint64_t* sread = sfull + kSB;      // [kSB] and read (4 warps)
    uint64_t* pfull = sread + kSB;      // [kBufs] P and the warps' flags written (4 warps), V expanded (4-bit: 4 more)
    uint64_t* pempty = pfull + kBufs;   // [kBufs] the P V is done (commit)
    uint64_t* fix = pempty + kBufs;     // [kSets] P written anew, O rescaled (4 warps)
    uint64_t* mbar = fix + kSets;       // [kSets] the warps' maxima written (4 warps)
    uint64_t* odone = mbar + kSets;     // [2] a segment's P V MMAs are done (commit; segments in turn)
    uint64_t* qfull = odone + 2;        // query heads ready (bytes; 4-bit: 4 warps)
    uint64_t* qempty = qfull + 1;       // the segment's S MMAs are done (commit)
    uint64_t* sums = qempty + 1;        // every set's references and sums written (all softmax warps)
    uint64_t* oempty = sums + 1;        // the segment's outputs have been read (all softmax warps)
    uint64_t* done = oempty + 1;        // every MMA issued is done (two commits)
    static_assert((3 * kS + 2 * kRaw + 3 * kSB + 2 * kBufs + 2 * kSets + 7) * 8 <= L::refs - L::misc, "barriers");
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::slot);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == L::warp_pv) {
        if (lane == 0) {
            for (int i = 0; i < kS; ++i) {
                mbar_init(kland + i, 1);
                mbar_init(vland + i, 1);
                mbar_init(empty + i, 1);
            }
            for (int i = 0; i < kRaw; ++i) {
                mbar_init(rfull + i, 1);
                mbar_init(rempty + i, 8);
            }
            for (int i = 0; i < kSB; ++i) {
                mbar_init(kfull + i, 4);
                mbar_init(sfull + i, 1);
                mbar_init(sread + i, 4);
            }
            for (int i = 0; i < kBufs; ++i) {
                mbar_init(pfull + i, FP4 ? 8 : 4);
                mbar_init(pempty + i, 1);
            }
            for (int i = 0; i < kSets; ++i) {
                mbar_init(fix + i, 4);
                mbar_init(mbar + i, 4);
            }
            mbar_init(qfull, FP4 ? 4 : 1);
            mbar_init(qempty, 1);
            mbar_init(sums, 4 * kSets);
            mbar_init(oempty, 4 * kSets);
            mbar_init(odone, 1);
            mbar_init(odone + 1, 1);
            mbar_init(done, 2);
            *abort_flag = 0;
            fence_barrier_init();
        }
        __syncwarp();
        tmem_alloc(tmem_slot, L::tmem_cols);
        tmem_relinquish();
    }
    // columns without a head: zero queries
    for (int i = threadIdx.x; i < kBdN * D * 2 / 16; i += L::warps * 32)
        *reinterpret_cast<uint4*>(smem + L::q + i * 16) = make_uint4(0, 0, 0, 0);
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    grid_dependency_wait();
    grid_launch_dependents();
    BaCursor cur = ba_start<true>(p, reinterpret_cast<int*>(smem + L::refs));
    BaSeg sg;
    bool ok = true;

    if (warp < 4 * kSets) {
        // --------------------------------------------------------- softmax
        const int set = warp >> 2, quad = warp & 3;
        const int tok = quad * 32 + lane;                 // of the tile; also the dim of O this thread has
        const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
        float* refs = reinterpret_cast<float*>(smem + L::refs) + warp * kBdN;
        float* mx = reinterpret_cast<float*>(smem + L::mx) + set * 4 * kBdN;      // this set's
        const float* c2s = reinterpret_cast<const float*>(smem + L::c2);
        volatile int* flags = reinterpret_cast<volatile int*>(smem + L::flags);
        const int piece = tok / p.PB, in_piece = tok - piece * p.PB;
        const int half = ((tok >> 2) & 1) << 4;
        const uint32_t to = tmem + lane_off + L::tmem_o + set * kBdN;
        uint32_t it0 = 0, seg = 0, mn = 0;                // tiles before the segment, segments, uses of mbar
        while (ok && cur.next<true>(p, &sg)) {
            const int np = ba_pieces(p, sg);
            float l[kBdN];
#pragma unroll
            for (int h = 0; h < kBdN; ++h) l[h] = 0.f;
            if (lane < kBdN) refs[lane] = 0.f;
            __syncwarp();
            const int j0 = (set + kSets - static_cast<int>(it0 % kSets)) % kSets;   // this set's first tile
            int e = (sg.t0 + j0) * p.S + piece;
            int nv = e < np ? ba_piece(p, sg, e).x & 255 : 0;        // visible tokens of this thread's piece
            for (int j = j0; j < sg.n; j += kSets) {
                const uint32_t it = it0 + j, buf = it % kBufs, sb = it % kSB;
                const bool first = j < kSets;
                const bool vis = in_piece < nv;
                const bool tail = nv < p.PB;
                e += kSets * p.S;
                const int nv_next = e < np ? ba_piece(p, sg, e).x & 255 : 0;
                const uint32_t ts = tmem + lane_off + L::tmem_s + sb * kBdN;
                uint8_t* prow = smem + L::p0 + buf * (kBdN * 256) + tok * 32;
                if (!(ok = warp_wait_b(sfull + sb, (it / kSB) & 1, abort_flag))) break;
                tc_fence_after();
                // the P operand's last reader, P V of tile it - kBufs
                if (it >= kBufs && !(ok = warp_wait_b(pempty + buf, (it / kBufs - 1) & 1, abort_flag))) break;
                float z[kBdN];
                auto logits = [&]() {                     // relative to the references, in log2
                    uint32_t v[kBdN];
                    tmem_ld16_nowait(ts, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int q = 0; q < kBdN / 4; ++q) {
                        const float4 r4 = *reinterpret_cast<const float4*>(refs + 4 * q);
                        float4 c4 = make_float4(p.scale_log2, p.scale_log2, p.scale_log2, p.scale_log2);
                        if (FP4) c4 = *reinterpret_cast<const float4*>(c2s + (seg & 1) * kBdN + 4 * q);
                        const float r[4] = {r4.x, r4.y, r4.z, r4.w}, c[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            z[4 * q + i] = vis ? fmaf(__uint_as_float(v[4 * q + i]), c[i], -r[i]) : -INFINITY;
                    }
                };
                auto weights = [&]() {                    // z becomes P, unrounded
                    uint32_t w[kBdN / 2];
#pragma unroll
                    for (int h = 0; h < kBdN; h += 2) {
                        z[h] = ex2_approx(z[h]);
                        z[h + 1] = ex2_approx(z[h + 1]);
                        w[h / 2] = FP4 ? pack_f16(z[h], z[h + 1]) : pack_bf16(z[h], z[h + 1]);
                    }
                    *reinterpret_cast<uint4*>(prow + half) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4*>(prow + (half ^ 16)) = make_uint4(w[4], w[5], w[6], w[7]);
                };
                logits();
                bool redo = first;
                if (!first) {
                    // P as if no maximum had passed its reference by 2^8; a warp that sees one
                    // raises its flag, and the MMA waits for P to be written anew
                    float m = z[0];
#pragma unroll
                    for (int h = 1; h < kBdN; ++h) m = fmaxf(m, z[h]);
                    const bool over = __any_sync(0xffffffffu, m > kRef + kBaGrow);
                    weights();
                    if (lane == 0) flags[buf * 4 + quad] = over;
                }
                if (!FP4 && __any_sync(0xffffffffu, tail)) {
                    // V rows past the last visible token: zeros, for 0 * NaN is NaN
                    const uint32_t vi = 2 * it + 1;
                    if (!(ok = warp_wait_b(vland + vi % kS, (vi / 6) & 1, abort_flag))) break;
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
                if (!first) {
                    if (!(ok = warp_wait_b(pfull + buf, (it / kBufs) & 1, abort_flag))) break;
                    const int4 f = *reinterpret_cast<const int4*>(smem + L::flags + buf * 16);
                    redo = (f.x | f.y | f.z | f.w) != 0;
                    if (redo) logits();
                }
                if (redo) {
                    // the maxima of all heads over the tile, and new references
                    float mine = 0.f;
#pragma unroll
                    for (int h = 0; h < kBdN; ++h) {
                        const float m = warp_max(z[h]);
                        if (lane == h) mine = m;
                    }
                    if (lane < kBdN) mx[quad * kBdN + lane] = mine;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(mbar + set);
                    if (!(ok = warp_wait_b(mbar + set, mn & 1, abort_flag))) break;
                    ++mn;
                    float up = 0.f;   // lane h: how far head h's reference moves
                    if (lane < kBdN) {
                        const float m = fmaxf(fmaxf(mx[lane], mx[kBdN + lane]), fmaxf(mx[2 * kBdN + lane], mx[3 * kBdN + lane]));
                        if (first) up = m > -INFINITY ? m - kRef : 0.f;
                        else up = fmaxf(m - kRef, 0.f);
                        refs[lane] += up;
                    }
                    __syncwarp();
                    if (!first) {
                        // O is free once the set's last P V is done
                        const uint32_t before = it - kSets;
                        if (!(ok = warp_wait_b(pempty + before % kBufs, (before / kBufs) & 1, abort_flag))) break;
                        tc_fence_after();
                        uint32_t o[kBdN];
                        tmem_ld16_nowait(to, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int h = 0; h < kBdN; ++h) {
                            const float a = ex2_approx(-__shfl_sync(0xffffffffu, up, h));
                            l[h] *= a;
                            o[h] = __float_as_uint(__uint_as_float(o[h]) * a);
                        }
                        tmem_st16(to, o);
                        tmem_st_wait();
                    }
#pragma unroll
                    for (int h = 0; h < kBdN; ++h) z[h] -= __shfl_sync(0xffffffffu, up, h);
                    weights();
                    fence_async_smem();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(fix + set);
                }
                if (lane == 0) mbar_arrive(sread + sb);
#pragma unroll
                for (int h = 0; h < kBdN; ++h) l[h] += z[h];
                nv = nv_next;
            }
            if (!ok) break;
            // the heads' sums over the set's threads, and the output (the area is written again
            // two segments on, when every warp has been through the next one's barrier)
            float* fin = reinterpret_cast<float*>(smem + L::fin) + (seg & 1) * kSets * 5 * kBdN;
            if (!(ok = warp_wait_b(odone + (seg & 1), (seg >> 1) & 1, abort_flag))) break;
            tc_fence_after();
            // (each thread's sums into its own set's P buffers, 64 bytes a thread, a half of the
            // threads in each; then warp w adds up threads 32 w .. of all heads)
            float* part = reinterpret_cast<float*>(smem + L::p0 + (set + (quad >> 1) * kSets) * (kBdN * 256)) + (quad & 1) * 32 * kBdN;
#pragma unroll
            for (int q = 0; q < kBdN / 4; ++q)
                *reinterpret_cast<float4*>(part + lane * kBdN + 4 * q) = make_float4(l[4 * q], l[4 * q + 1], l[4 * q + 2], l[4 * q + 3]);
            __syncwarp();
            float mysum = 0.f;
#pragma unroll 4
            for (int q = 0; q < 16; ++q) mysum += part[(2 * q + (lane >> 4)) * kBdN + (lane & 15)];
            mysum += __shfl_xor_sync(0xffffffffu, mysum, 16);
            if (lane < kBdN) fin[(set * 5 + quad) * kBdN + lane] = mysum;
            if (quad == 0 && lane < kBdN) fin[(set * 5 + 4) * kBdN + lane] = refs[lane];
            __syncwarp();
            if (lane == 0) mbar_arrive(sums);
            if (!(ok = warp_wait_b(sums, seg & 1, abort_flag))) break;
            const bool whole = sg.n == sg.T;
            const int slot = 2 * blockIdx.x + (sg.t0 == 0 ? 1 : 0);
            const size_t orow = static_cast<size_t>(sg.g) * p.Hq + sg.h * p.G;
            // lane h: head h's sum and reference over the sets, and the sets' weights
            float sum = 0.f, M = -INFINITY, wt[kSets] = {};
            if (lane < kBdN) {
                float ls[kSets], ms[kSets];
#pragma unroll
                for (int q = 0; q < kSets; ++q) {
                    const float* x = fin + q * 5 * kBdN + lane;
                    ls[q] = (x[0] + x[kBdN]) + (x[2 * kBdN] + x[3 * kBdN]);
                    ms[q] = ls[q] > 0.f ? x[4 * kBdN] : -INFINITY;
                    M = fmaxf(M, ms[q]);
                }
#pragma unroll
                for (int q = 0; q < kSets; ++q) {
                    wt[q] = ms[q] > -INFINITY ? ex2_approx(ms[q] - M) : 0.f;
                    sum += wt[q] * ls[q];
                }
                const float norm = whole ? (sum > 0.f ? p.out_mul / sum : 0.f) : 1.f;
#pragma unroll
                for (int q = 0; q < kSets; ++q) wt[q] *= norm;
            }
            // the sets share the heads out: set s writes heads 4 (s + sets i) .. + 3 (few
            // instructions rather than an unrolled loop: this code runs once a segment, cold)
            __syncwarp();
#pragma unroll 1
            for (int h0 = 4 * set; h0 < p.G; h0 += 4 * kSets) {
                uint32_t o[kSets][4];
#pragma unroll
                for (int q = 0; q < kSets; ++q) tmem_ld4_nowait(tmem + lane_off + L::tmem_o + q * kBdN + h0, o[q]);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v = 0.f;
#pragma unroll
                    for (int q = 0; q < kSets; ++q) {
                        const float w = __shfl_sync(0xffffffffu, wt[q], h0 + i);
                        if (w > 0.f) v = fmaf(w, __uint_as_float(o[q][i]), v);    // a set without a tile has nothing in O
                    }
                    if (h0 + i < p.G && tok < D) {
                        if (whole) p.out[(orow + h0 + i) * D + tok] = static_cast<uint16_t>(pack_bf16(v, 0.f));
                        else p.part_o[(static_cast<size_t>(slot) * kBdN + h0 + i) * D + tok] = v;
                    }
                }
                __syncwarp();
            }
            if (warp == 0 && lane < p.G) {
                if (!whole) p.part_ml[slot * kBdN + lane] = make_float2(M, sum);
                else if (p.lse) p.lse[orow + lane] = sum > 0.f ? (M + log2f(sum)) * 0.6931471805599453f : -INFINITY;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(oempty);
            it0 += sg.n;
            ++seg;
        }
    } else if (FP4 && warp < L::warp_vd) {
        // -------------------------------------------- queries; K into TMEM
        const int dw = warp - L::warp_kd;
        const int row = dw * 32 + lane;
        uint32_t it = 0, seg = 0;
        while (ok && cur.next<true>(p, &sg)) {
            if (seg > 0 && !(ok = warp_wait_b(qempty, (seg - 1) & 1, abort_flag))) break;
            // the softmax is done with the scales of two segments ago
            if (seg > 1 && !(ok = warp_wait_b(odone + (seg & 1), ((seg >> 1) - 1) & 1, abort_flag))) break;
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
                const uint32_t rs = it % kRaw, sb = it % kSB;
                if (!(ok = warp_wait_b(rfull + rs, (it / kRaw) & 1, abort_flag))) break;
                const uint8_t* raw = smem + L::raw0 + rs * L::raw;
                // S of tile it - kSB, the last reader of this TMEM buffer
                if (it >= kSB && !(ok = warp_wait_b(sfull + sb, (it / kSB - 1) & 1, abort_flag))) break;
                tc_fence_after();
                const uint32_t tk = tmem + (static_cast<uint32_t>(dw * 32) << 16) + L::tmem_k + sb * (D / 2);
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
                if (lane == 0) mbar_arrive(kfull + sb);
            }
        }
    } else if (FP4 && warp < L::warp_load) {
        // ------------- V into shared memory: two teams of four warps, a tile each in turn
        const int team = (warp - L::warp_vd) >> 2, dw = (warp - L::warp_vd) & 3;
        constexpr int kCh = D / 32;       // 16-byte chunks of codes (32 elements) per row
        constexpr int kRows = 32 / kCh;   // rows a warp expands at a time
        const int ch = lane % kCh, rl = lane / kCh;
        uint32_t it0 = 0;   // tiles before the segment
        while (ok && cur.next<true>(p, &sg)) {
            const int np = ba_pieces(p, sg);
            const int r = dw * 32 + lane, s = r / p.PB;
            const int j0 = (team + 2 - static_cast<int>(it0 & 1)) & 1;
            int e = (sg.t0 + j0) * p.S + s;
            bool sees = e < np && r - s * p.PB < (ba_piece(p, sg, min(e, np - 1)).x & 255);
            for (int j = j0; j < sg.n; j += 2) {
                const uint32_t it = it0 + j;
                const uint32_t seen = __ballot_sync(0xffffffffu, sees);   // the other rows become zeros
                e += 2 * p.S;
                sees = e < np && r - s * p.PB < (ba_piece(p, sg, min(e, np - 1)).x & 255);
                const uint32_t rs = it % kRaw, slot = it % kS;
                if (!(ok = warp_wait_b(rfull + rs, (it / kRaw) & 1, abort_flag))) break;
                // the slot's last reader, P V of tile it - kS (this team saw the one before it - kS + 1
                // through when it took its last tile, so the parity is that phase's)
                const uint32_t last = it - kS;
                if (it >= kS && !(ok = warp_wait_b(pempty + last % kBufs, (last / kBufs) & 1, abort_flag))) break;
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
                    mbar_arrive(pfull + it % kBufs);
                }
            }
            it0 += sg.n;
        }
    } else if (warp == L::warp_load) {
        // ------------------------------------------------------------ load
        // Lane s < S loads piece s of each tile.
        uint32_t it = 0, seg = 0, issued = 0;
        while (ok && cur.next<true>(p, &sg)) {
            const int np = ba_pieces(p, sg);
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
            int2 pc = mine && e < np ? ba_piece(p, sg, e) : make_int2(-1, 0);
            for (int j = 0; j < sg.n; ++j, ++it) {
                const int2 now = pc;
                e += p.S;
                pc = mine && j + 1 < sg.n && e < np ? ba_piece(p, sg, e) : make_int2(-1, 0);
                const bool have = now.x >= 0;
                const int bh = have ? (now.x >> 8) * p.Hkv + sg.h : 0;
                if (!FP4) {
                    const int rowc = have ? now.y * p.PB : p.cap;   // a missing piece: rows past the end, zeros
                    for (int kv = 0; kv < 2; ++kv) {
                        const uint32_t n = 2 * it + kv, slot = n % kS;
                        if (n >= kS && !(ok = warp_wait_b(empty + slot, (n / kS - 1) & 1, abort_flag))) break;
                        uint64_t* land = (kv ? vland : kland) + slot;   // n / 6: its use for this kind of tile
                        if (lane == 0) mbar_arrive_expect_tx(land, L::tile);
                        issued = n + 1;
                        __syncwarp();
                        if (mine) {
                            uint8_t* dst = smem + L::ring + slot * L::tile + lane * p.PB * 128;
#pragma unroll
                            for (int a = 0; a < D / 64; ++a) {
                                if (kv) tma_load_3d(dst + a * 16384, &v_map, land, a * 64, rowc, bh);
                                else tma_load_3d(dst + a * 16384, &k_map, land, a * 64, rowc, bh);
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
        if (!ok) {
            // the copies in flight land before the CTA gives up its shared memory
            *abort_flag = 1;
            constexpr uint32_t n = FP4 ? kRaw : kS;
            if (!FP4 && seg > 0) warp_wait_b(qfull, (seg - 1) & 1, nullptr);
            for (uint32_t i = issued > n ? issued - n : 0; i < issued; ++i)
                warp_wait_b((FP4 ? rfull : i & 1 ? vland : kland) + i % n, (i / (FP4 ? n : 6)) & 1, nullptr);
        }
    } else if (warp == L::warp_s) {
        // ------------------------------------------------------- S = K Q^T
        constexpr uint32_t id = idesc_bd(FP4, false, false);
        const uint32_t q_lo = uni(desc_lo(smem_addr(smem + L::q), 16)), k_lo = uni(desc_lo(smem_addr(smem + L::ring), 16));
        const uint32_t tm = uni(tmem);
        uint32_t it = 0, seg = 0;
        while (ok && cur.next<true>(p, &sg)) {
            if (!(ok = warp_wait_b(qfull, seg & 1, abort_flag))) break;
            for (int j = 0; j < sg.n; ++j, ++it) {
                const uint32_t sb = it % kSB, slot = (2 * it) % kS;
                if (it >= kSB && !(ok = warp_wait_b(sread + sb, (it / kSB - 1) & 1, abort_flag))) break;
                if (FP4) ok = warp_wait_b(kfull + sb, (it / kSB) & 1, abort_flag);
                else ok = warp_wait_b(kland + slot, (2 * it / 6) & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
                const uint32_t at = uni(slot * kSB + sb);
                const uint32_t td = tm + L::tmem_s + (at % kSB) * kBdN;
                const uint32_t a = FP4 ? tm + L::tmem_k + (at % kSB) * (D / 2) : k_lo + (at / kSB) * (L::tile >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int s = 0; s < D / 16; ++s) {
                        const uint64_t q = desc64(q_lo + (s >> 2) * (kBdN * 128 >> 4) + (s & 3) * 2, kHi128);
                        if (FP4) umma_f16_ts(td, a + s * 8, q, id, s > 0);
                        else umma_bf16(td, desc64(a + (s >> 2) * 1024 + (s & 3) * 2, kHi128), q, id, s > 0);
                    }
                    if (!FP4) umma_commit(empty + slot);
                    umma_commit(sfull + sb);
                    if (j + 1 == sg.n) umma_commit(qempty);
                }
                __syncwarp();
            }
            ++seg;
        }
        if (!ok) *abort_flag = 1;
        if (elect_one()) umma_commit(done);
        __syncwarp();
    } else {
        // ------------------------------------------------------ O += V^T P
        constexpr uint32_t id = idesc_bd(FP4, true, true);
        // V: MN-major A operand, atoms of 64 dims x 8 tokens; d = 64: the MMA's upper 64 rows
        // re-read bytes 1 KB further on (their results are not used)
        const uint32_t v_lo = uni(desc_lo(smem_addr(smem + L::ring), D == 128 ? 16384 : 1024));
        const uint32_t p_lo = uni(desc_lo(smem_addr(smem + L::p0), 16)), tm = uni(tmem);
        uint32_t it = 0, seg = 0, fixes[2] = {0, 0};
        while (ok && cur.next<true>(p, &sg)) {
            for (int j = 0; j < sg.n; ++j, ++it) {
                const uint32_t buf = it % kBufs, set = it % kSets, n = FP4 ? it : 2 * it + 1, slot = n % kS;
                if (!(ok = warp_wait_b(pfull + buf, (it / kBufs) & 1, abort_flag))) break;
                const int4 f = *reinterpret_cast<const int4*>(smem + L::flags + buf * 16);
                if (j < kSets || (f.x | f.y | f.z | f.w)) {
                    ok = warp_wait_b(fix + set, fixes[set] & 1, abort_flag);
                    ++fixes[set];
                }
                if (ok && j == 0 && seg > 0) ok = warp_wait_b(oempty, (seg - 1) & 1, abort_flag);
                if (!FP4) ok = ok && warp_wait_b(vland + slot, (n / 6) & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
                const uint32_t at = uni(slot * 8 + buf * 2 + (j >= kSets ? 1 : 0));   // buf's set: buf % kSets
                const uint32_t td = tm + L::tmem_o + ((at >> 1) % kSets) * kBdN, a = v_lo + (at >> 3) * (L::tile >> 4);
                const uint32_t b = p_lo + ((at >> 1) & 3) * (kBdN * 256 >> 4), more = at & 1;
                if (elect_one()) {
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        umma_bf16(td, desc64(a + s * (2048 >> 4), kHi128), desc64(b + s * (512 >> 4), kHiP), id, s > 0 ? 1u : more);
                    if (!FP4) umma_commit(empty + slot);
                    umma_commit(pempty + buf);
                    if (j + 1 == sg.n) umma_commit(odone + (seg & 1));
                }
                __syncwarp();
            }
            ++seg;
        }
        if (!ok) *abort_flag = 1;
        // every MMA done before TMEM is freed (a bounded wait that an abort does not cut short)
        if (elect_one()) umma_commit(done);
        __syncwarp();
        if (!warp_wait_b(done, 0, nullptr)) ok = false;
        __syncwarp();
    }
    if (!ok && lane == 0) {
        *abort_flag = 1;
        set_status(p.status, HISA_DEV_TIMEOUT);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == L::warp_pv) {
        tc_fence_after();
        tmem_dealloc(tmem, L::tmem_cols);
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
