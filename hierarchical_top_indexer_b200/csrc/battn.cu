// Block-sparse attention: grouped-query attention of each query row over all
// tokens of its kept blocks (or over its whole prefix), from a cache of bf16
// rows or of 4-bit rows (e2m1 codes and an e4m3 scale per 16 elements).
//
// Row i of sequence b at position t keeps the blocks j of its list; head h of
// the G = Hq / Hkv heads that share a key and value head attends to
//     z_s = scale * q . K[s],  s in a kept block, s <= t
//     out = sum_s softmax(z)_s V[s],   lse = log sum_s exp z_s.
//
// Plan.  R consecutive rows form a group whose (row, head) pairs fill the 128
// rows of one MMA: R = 128 / G for a chunk (battn_layout has the rule), else 1.
// A group reads the union of its rows' blocks once, each row masking what it
// did not keep: neighbouring rows keep much the same blocks, and a tile of
// keys then serves up to 128 (row, head) pairs instead of G.  plan_kernel
// turns a group's lists into a sorted list of pieces (up to 128 tokens of one
// block of one sequence), without duplicates; 128 / piece pieces make a tile.
// The persistent CTAs of battn_kernel add the groups' tiles up and take equal
// runs of all (key head, group, tile) slots.  A run's part of a group is
// a segment; a group that one segment covers is finished in place, the parts
// of a group that several CTAs share are joined by join_kernel.
//
// One CTA: warps 0-7 softmax (two sets of four, one thread per MMA row), warp
// 8 loads, warp 9 issues the MMAs, and for 4-bit rows warps 10-13 dequantise.
// Tiles alternate between the sets; each set has an S buffer (where P takes
// the place of S), a running maximum, sum and output accumulator of its own,
// so that neither waits for the other, and the two are merged at the end of a
// segment.  TMEM: S0, S1 (128 columns each), O0, O1.
//   S = Q K^T   (A = Q in shared memory, B = K tile)
//   P = 2^(z - m) in TMEM, unnormalised, m raised (and O rescaled) only when a
//       maximum has grown by more than 2^8: P stays below 2^8, where bf16 and
//       f16 keep their relative precision
//   O += P V    (A = P in TMEM, B = V tile, MN-major)
// bf16 rows come by TMA into the swizzled operand layout (K and V rings).
// 4-bit rows come as they are (contiguous per head); the dequantising warps
// expand them to f16, in which code * scale is exact, and the query rows are
// scaled by a power of two into f16's range, where they too are exact.
// P is rounded to bf16 (2^-8 relative) or f16 (2^-11); everything else is fp32.
// f16 P is kept 2^7 larger, so that weights down to 2^-21 of the largest keep
// all their bits and only those below 2^-32 of it vanish.
//
// Bound (d = 128): 4096 rows of one sequence, 64 of 256 blocks each, 16 heads
// over 2 key heads, 681 to 743 us: 2500 to 2700 cycles a tile, of which the 2^x
// unit takes 1024 and the MMAs 1024; the rest is the chain of each set (S,
// softmax, P V), because P takes S's place and the next S of the set waits for
// P V, and the softmax's registers: at 168 a thread it reads S twice and spills
// (352 bytes stored, 580 loaded).  4-bit rows, 2 x 512 rows causal over 8191
// keys, 32 heads over 4: 223 to 227 us; the same over bf16 rows 186 us, and
// 182 us without the expansion, whose four warps do K and then V of a tile
// (216 and 484 bytes of spills at 128 registers).
// An element-wise mask costs twice the whole tile, hence the rows that are on
// or off; a single polling lane per wait cost twice the kernel (1459 us).
#include "battn.cuh"

namespace hisa {

namespace {

constexpr int kBaSoftWarps = 8;
constexpr int kBaWarpLoad = 8;
constexpr int kBaWarpMma = 9;
constexpr int kBaWarpDeq = 10;      // 10-13 (4-bit rows)

template <int D, bool FP4>
struct BaLayout {
    static constexpr int tile = 128 * D * 2;          // one operand of 128 rows
    static constexpr int rings = FP4 ? 2 : 3;         // K and V operands in flight
    static constexpr int raw_codes = 128 * D / 2;
    static constexpr int raw_scales = 128 * D / 16;
    static constexpr int raw = FP4 ? 2 * (raw_codes + raw_scales) : 0;   // K codes, V codes, K scales, V scales
    static constexpr int raws = FP4 ? 3 : 0;
    static constexpr int q = 0;
    static constexpr int k0 = tile;
    static constexpr int v0 = k0 + rings * tile;
    static constexpr int raw0 = v0 + rings * tile;
    static constexpr int ml = raw0 + raws * raw;      // [2 sets][128] (maximum, sum)
    static constexpr int qs = ml + 2048;              // [2 segments][128] query row scales (4-bit rows)
    static constexpr int bars = qs + (FP4 ? 1024 : 0);
    static constexpr int total = bars + 256;
    static constexpr int threads = FP4 ? 448 : 320;
};

// M = 128, N = n, fp32 accumulate; f16 or bf16 inputs; B K-major or MN-major.
__host__ __device__ constexpr uint32_t idesc_ba(uint32_t n, bool f16, bool b_mn_major) {
    return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (b_mn_major ? (1u << 16) : 0u) | ((n >> 3) << 17) |
           ((128u >> 4) << 24);
}

// ------------------------------------------------------------------- plan

// One CTA per group: the visible kept blocks of the group's rows as a list of
// pieces {sequence << 8 | tokens of it any row sees, piece of the sequence},
// sequence by sequence (in the order of their first rows), pieces ascending.
// bits: per-row bitmaps of the kept blocks, in shared memory for a lone row,
// else in the workspace (the softmax masks by them).
constexpr int kPlanThreads = 256;

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const BattnParams p) {
    extern __shared__ uint32_t lone_bits[];
    __shared__ int s_seq[128], s_pos[128], s_lead[128];
    __shared__ int s_scan[kPlanThreads / 32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int g = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row0 = g * p.R;
    const int nr = min(p.R, p.n_q - row0);
    const int W = p.W;
    for (int r = tid; r < nr; r += kPlanThreads) {
        int b;
        const int t = query_position(p.q_seq, p.q_pos, p.len, p.batch, p.cap, row0 + r, &b);
        if (t < 0) set_status(p.status, HISA_DEV_BAD_QUERY);
        s_seq[r] = b;
        s_pos[r] = t;
    }
    uint32_t* bits = p.R == 1 ? lone_bits : p.bits + static_cast<size_t>(row0) * W;
    if (p.blocks)
        for (int i = tid; i < nr * W; i += kPlanThreads) bits[i] = 0u;
    __syncthreads();
    for (int r = tid; r < nr; r += kPlanThreads) {
        bool lead = s_pos[r] >= 0;
        for (int q = 0; q < r && lead; ++q) lead = !(s_pos[q] >= 0 && s_seq[q] == s_seq[r]);
        s_lead[r] = lead;
    }
    if (p.blocks)
        for (int i = tid; i < nr * p.mb; i += kPlanThreads) {
            const int r = i / p.mb, t = s_pos[r];
            const int j = p.blocks[static_cast<size_t>(row0) * p.mb + i];
            if (t >= 0 && j >= 0 && j <= t / p.B) atomicOr(bits + static_cast<size_t>(r) * W + (j >> 5), 1u << (j & 31));
        }
    __syncthreads();
    int2* list = p.list + static_cast<size_t>(g) * p.lcap;
    int base = 0;
    for (int r = 0; r < nr; ++r) {
        if (!s_lead[r]) continue;
        const int b = s_seq[r];
        int tmax = 0;
        for (int q = r; q < nr; ++q)
            if (s_seq[q] == b) tmax = max(tmax, s_pos[q]);
        if (!p.blocks) {
            const int n = tmax / p.PB + 1;
            for (int i = tid; i < n; i += kPlanThreads)
                list[base + i] = make_int2(b << 8 | min(p.PB, tmax + 1 - i * p.PB), i);
            base += n;
            continue;
        }
        const int last = tmax / p.B;                             // the last visible block
        const int last_n = (tmax - last * p.B) / p.PB + 1;       // its visible pieces
        for (int w0 = 0; w0 <= last >> 5; w0 += kPlanThreads) {
            const int w = w0 + tid;
            uint32_t u = 0;
            if (w < W)
                for (int q = r; q < nr; ++q)
                    if (s_pos[q] >= 0 && s_seq[q] == b) u |= p.R == 1 ? bits[w] : __ldcg(bits + static_cast<size_t>(q) * W + w);
            int n = __popc(u) * p.ppb;
            if (w == last >> 5 && ((u >> (last & 31)) & 1u)) n -= p.ppb - last_n;
            int x = n;   // inclusive scan over the block
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            __syncthreads();
            if (lane == 31) s_scan[warp] = x;
            __syncthreads();
            int before = 0, all = 0;
            for (int q = 0; q < kPlanThreads / 32; ++q) {
                if (q < warp) before += s_scan[q];
                all += s_scan[q];
            }
            int at = base + before + x - n;
            while (u) {
                const int j = w * 32 + __ffs(u) - 1;
                u &= u - 1;
                const int pieces = j == last ? last_n : p.ppb;
                for (int i = 0; i < pieces; ++i) {
                    const int piece = j * p.ppb + i;
                    list[at++] = make_int2(b << 8 | min(p.PB, tmax + 1 - piece * p.PB), piece);
                }
            }
            base += all;
        }
    }
    if (tid == 0) {
        p.pieces[g] = base;
        p.tiles[g] = (base + p.S - 1) / p.S;
    }
}

// -------------------------------------------------------------- attention

// One MMA row (this thread's) of one tile: S (TMEM, 128 columns at ts) to P in
// its place, with the row's reference m and sum l, and its output (TMEM, to)
// rescaled if the reference moves.  MASK: element by element as mw says; else
// the row is seen whole (on) or not at all.  first: nothing in O yet.
template <int D, bool FP4, bool MASK>
__device__ __forceinline__ void softmax_tile(uint32_t ts, uint32_t to, const uint32_t (&mw)[4], bool on, bool first, float c2,
                                             float& m, float& l) {
    constexpr float kRef = FP4 ? 7.f : 0.f;   // log2 of the largest P of a fresh maximum
    // S is read twice, 32 columns ahead of their use (all 128 would not fit the registers)
    uint32_t v[2][32];
    float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    tmem_ld32_nowait(ts, v[0]);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        tmem_ld_wait();
        if (c < 3) tmem_ld32_nowait(ts + (c + 1) * 32, v[(c + 1) & 1]);
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (!MASK || ((mw[c] >> i) & 1u)) mx4[i & 3] = fmaxf(mx4[i & 3], __uint_as_float(v[c & 1][i]));
    }
    float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
    if (!MASK && !on) mx = -INFINITY;
    if (mx > -INFINITY) mx *= c2;   // -inf where the row sees nothing
    if (first) {
        m = mx - kRef;
    } else {
        const bool grew = mx > m + (kRef + kBaGrow) || (m == -INFINITY && mx > m);
        if (__any_sync(0xffffffffu, grew)) {
            const float alpha = grew ? ex2_approx(m - (mx - kRef)) : 1.f;
            if (grew) m = mx - kRef;
            l *= alpha;
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
                uint32_t w[16];
                tmem_ld16_nowait(to + c * 16, w);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * alpha);
                tmem_st16(to + c * 16, w);
            }
        }
    }
    tmem_ld32_nowait(ts, v[0]);
    const bool off = !MASK && !on;
    const float mul = off ? 0.f : c2, sub = off ? -200.f : m == -INFINITY ? 0.f : -m;
    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t(&x)[32] = v[c & 1];
        tmem_ld_wait();
        if (c < 3) tmem_ld32_nowait(ts + (c + 1) * 32, v[(c + 1) & 1]);
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            float e[4] = {sub, sub, sub, sub};
            fma2(e[0], e[1], mul, mul, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
            fma2(e[2], e[3], mul, mul, __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]));
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                e[u] = ex2_approx(e[u]);
                if (MASK && !((mw[c] >> (i + u)) & 1u)) e[u] = 0.f;
            }
            fma2(s0, s1, 1.f, 1.f, e[0], e[1]);
            fma2(s2, s3, 1.f, 1.f, e[2], e[3]);
            w[i / 2] = FP4 ? pack_f16(e[0], e[1]) : pack_bf16(e[0], e[1]);
            w[i / 2 + 1] = FP4 ? pack_f16(e[2], e[3]) : pack_bf16(e[2], e[3]);
        }
        tmem_st16(ts + c * 16, w);
    }
    float sum = (s0 + s1) + (s2 + s3);
    tmem_st_wait();
    if (!MASK && !FP4) {
        // An off row's weights are 2^(0 S - 200) = 0, and so is their sum, unless S overflowed
        // fp32 (bf16 rows: products of 4-bit rows stay far below): 0 * inf is NaN.  Then the off
        // rows' P is cleared after all (S is gone, so the warp cannot go through the masked form
        // again; a vote a tile, no work per element).
        if (__any_sync(0xffffffffu, off && sum != 0.f)) {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t w[16];
                tmem_ld16_nowait(ts + c * 16, w);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = off ? 0u : w[i];
                tmem_st16(ts + c * 16, w);
            }
            tmem_st_wait();
            if (off) sum = 0.f;
        }
    }
    l += sum;
}

template <int D, bool FP4>
__global__ void __launch_bounds__(BaLayout<D, FP4>::threads, 1)
    battn_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                 const __grid_constant__ CUtensorMap v_map, const BattnParams p) {
    using L = BaLayout<D, FP4>;
    constexpr int kR = L::rings, kRaw = L::raws;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::bars);
    uint64_t* kfull = bars;             // [kR] K operand ready (bytes; 4-bit: 4 warps)
    uint64_t* kempty = kfull + 3;       // [kR] its S MMA is done (commit)
    uint64_t* vfull = kempty + 3;       // [kR]
    uint64_t* vempty = vfull + 3;       // [kR] its P V MMA is done (commit)
    uint64_t* rfull = vempty + 3;       // [3] 4-bit rows landed (bytes)
    uint64_t* rempty = rfull + 3;       // [3] they have been expanded (4 warps)
    uint64_t* sfull = rempty + 3;       // [2] S written, and the set's earlier P V done (commit)
    uint64_t* pfull = sfull + 2;        // [2] P written, O rescaled (4 warps)
    uint64_t* qfull = pfull + 2;        // query rows ready (bytes; 4-bit: 4 warps)
    uint64_t* qempty = qfull + 1;       // the segment's S MMAs are done (commit)
    uint64_t* odone = qempty + 1;       // the segment's P V MMAs are done (commit)
    uint64_t* oempty = odone + 1;       // its outputs have been read (8 warps)
    uint64_t* mlbar = oempty + 1;       // both sets' maxima and sums written (8 warps)
    uint64_t* done = mlbar + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == kBaWarpMma) {
        if (lane == 0) {
            for (int i = 0; i < 3; ++i) {
                mbar_init(kfull + i, FP4 ? 4 : 1);
                mbar_init(kempty + i, 1);
                mbar_init(vfull + i, FP4 ? 4 : 1);
                mbar_init(vempty + i, 1);
                mbar_init(rfull + i, 1);
                mbar_init(rempty + i, 4);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(sfull + i, 1);
                mbar_init(pfull + i, 4);
            }
            mbar_init(qfull, FP4 ? 4 : 1);
            mbar_init(qempty, 1);
            mbar_init(odone, 1);
            mbar_init(oempty, kBaSoftWarps);
            mbar_init(mlbar, kBaSoftWarps);
            mbar_init(done, 1);
            *abort_flag = 0;
            fence_barrier_init();
        }
        __syncwarp();
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    grid_dependency_wait();
    grid_launch_dependents();

    BaCursor cur = ba_start<false>(p, reinterpret_cast<int*>(smem + L::ml));
    BaSeg sg;
    bool ok = true;

    if (warp == kBaWarpLoad) {
        // ------------------------------------------------------------ load
        // Lane s < S loads piece s of each tile.
        uint32_t it = 0, seg = 0, issued[2] = {0, 0};
        while (ok && cur.next<false>(p, &sg)) {
            const int2* list = p.list + static_cast<size_t>(sg.g) * p.lcap;
            const int np = p.pieces[sg.g];
            if (!FP4) {
                if (seg > 0 && !(ok = warp_wait_b(qempty, (seg - 1) & 1, abort_flag))) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(qfull, static_cast<uint32_t>(p.R * p.G * D * 2));
#pragma unroll
                    for (int a = 0; a < D / 64; ++a)
                        tma_load_3d(smem + L::q + a * 16384, &q_map, qfull, a * 64, sg.h * p.G, sg.g * p.R);
                }
                __syncwarp();
            }
            ++seg;
            for (int j = 0; j < sg.n; ++j, ++it) {
                const int e = (sg.t0 + j) * p.S + lane;
                const bool have = lane < p.S && e < np;
                const int2 pc = have ? list[e] : make_int2(0, 0);
                const int b = pc.x >> 8;
                if (!FP4) {
                    // a missing piece loads rows past the sequence's end: zeros
                    const int rowc = have ? pc.y * p.PB : p.cap;
                    const int slot = it % kR;
                    const uint32_t use = it / kR;
                    for (int kv = 0; kv < 2; ++kv) {
                        uint64_t* full = (kv ? vfull : kfull) + slot;
                        if (use > 0 && !(ok = warp_wait_b((kv ? vempty : kempty) + slot, (use - 1) & 1, abort_flag))) break;
                        if (lane == 0) mbar_arrive_expect_tx(full, L::tile);
                        issued[kv] = it + 1;
                        __syncwarp();
                        if (lane < p.S) {
                            uint8_t* dst = smem + (kv ? L::v0 : L::k0) + slot * L::tile + lane * p.PB * 128;
#pragma unroll
                            for (int a = 0; a < D / 64; ++a)
                                tma_load_3d(dst + a * 16384, kv ? &v_map : &k_map, full, a * 64, rowc, b * p.Hkv + sg.h);
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                } else {
                    const int slot = it % (kRaw ? kRaw : 1);
                    const uint32_t use = it / (kRaw ? kRaw : 1);
                    if (use > 0 && !(ok = warp_wait_b(rempty + slot, (use - 1) & 1, abort_flag))) break;
                    const int tok = pc.y * p.PB;
                    const int rows = have ? min(p.PB, p.cap - tok) : 0;
                    const uint32_t all = __reduce_add_sync(0xffffffffu, rows);
                    if (lane == 0) mbar_arrive_expect_tx(rfull + slot, all * (D + D / 8));
                    issued[0] = it + 1;
                    __syncwarp();
                    if (rows > 0) {
                        const size_t r0 = (static_cast<size_t>(b) * p.Hkv + sg.h) * p.cap + tok;
                        uint8_t* dst = smem + L::raw0 + slot * L::raw;
                        const int at = lane * p.PB;
                        bulk_load(dst + at * (D / 2), p.k4 + r0 * (D / 2), rows * (D / 2), rfull + slot);
                        bulk_load(dst + L::raw_codes + at * (D / 2), p.v4 + r0 * (D / 2), rows * (D / 2), rfull + slot);
                        bulk_load(dst + 2 * L::raw_codes + at * (D / 16), p.k_scale + r0 * (D / 16), rows * (D / 16), rfull + slot);
                        bulk_load(dst + 2 * L::raw_codes + L::raw_scales + at * (D / 16), p.v_scale + r0 * (D / 16),
                                  rows * (D / 16), rfull + slot);
                    }
                    __syncwarp();
                }
            }
        }
        if (!ok) {
            if (lane == 0) {
                *abort_flag = 1;
                set_status(p.status, HISA_DEV_TIMEOUT);
            }
            // the copies in flight land before the CTA gives up its shared memory
            if (!FP4) {
                if (seg > 0) warp_wait_b(qfull, (seg - 1) & 1, nullptr);
                for (int kv = 0; kv < 2; ++kv)
                    for (uint32_t i = issued[kv] > kR ? issued[kv] - kR : 0; i < issued[kv]; ++i)
                        warp_wait_b((kv ? vfull : kfull) + i % kR, (i / kR) & 1, nullptr);
            } else {
                constexpr uint32_t n = kRaw ? kRaw : 1;
                for (uint32_t i = issued[0] > n ? issued[0] - n : 0; i < issued[0]; ++i)
                    warp_wait_b(rfull + i % n, (i / n) & 1, nullptr);
            }
        }
    } else if (warp == kBaWarpMma) {
        // ------------------------------------------------------------- MMA
        constexpr uint32_t id_s = idesc_ba(128, FP4, false), id_o = idesc_ba(D, FP4, true);
        const uint32_t q_lo = uni(desc_lo(smem_addr(smem + L::q), 16)), k_lo = uni(desc_lo(smem_addr(smem + L::k0), 16));
        const uint32_t v_lo = uni(desc_lo(smem_addr(smem + L::v0), 16384)), tm = uni(tmem_base);
        uint32_t kn = 0, vn = 0, seg = 0, pn[2] = {0, 0};
        auto issue_s = [&](int j) -> bool {
            const uint32_t slot = kn % kR;
            if (!warp_wait_b(kfull + slot, (kn / kR) & 1, abort_flag)) return false;
            tc_fence_after();
            const uint32_t at = uni(slot * 2 + (j & 1));
            const uint32_t td = tm + (at & 1) * 128, b = k_lo + (at >> 1) * (L::tile >> 4);
            if (elect_one()) {
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint32_t o = (s >> 2) * (16384 >> 4) + (s & 3) * 2;
                    umma_bf16(td, desc64(q_lo + o, kHi128), desc64(b + o, kHi128), id_s, s > 0);
                }
                umma_commit(kempty + slot);
                umma_commit(sfull + (j & 1));
            }
            __syncwarp();
            ++kn;
            return true;
        };
        while (ok && cur.next<false>(p, &sg)) {
            if (!(ok = warp_wait_b(qfull, seg & 1, abort_flag))) break;
            tc_fence_after();
            ok = issue_s(0) && (sg.n < 2 || issue_s(1));
            if (ok && sg.n <= 2 && elect_one()) umma_commit(qempty);
            for (int j = 0; j < sg.n && ok; ++j) {
                ok = warp_wait_b(pfull + (j & 1), pn[j & 1] & 1, abort_flag);
                ++pn[j & 1];
                if (ok && j == 0 && seg > 0) ok = warp_wait_b(oempty, (seg - 1) & 1, abort_flag);
                const uint32_t slot = vn % kR;
                ok = ok && warp_wait_b(vfull + slot, (vn / kR) & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
                const uint32_t at = uni(slot * 4 + (j > 1 ? 2 : 0) + (j & 1));
                const uint32_t ta = tm + (at & 1) * 128, b = v_lo + (at >> 2) * (L::tile >> 4), more = (at >> 1) & 1;
                if (elect_one()) {
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        umma_f16_ts(ta + 256, ta + s * 8, desc64(b + s * (2048 >> 4), kHi128), id_o, s > 0 ? 1u : more);
                    umma_commit(vempty + slot);
                    if (j + 1 == sg.n) umma_commit(odone);
                }
                __syncwarp();
                ++vn;
                if (j + 2 < sg.n) {
                    ok = issue_s(j + 2);
                    if (j + 3 == sg.n && elect_one()) umma_commit(qempty);
                }
            }
            ++seg;
        }
        if (!ok && lane == 0) {
            *abort_flag = 1;
            set_status(p.status, HISA_DEV_TIMEOUT);
        }
        // every MMA done before TMEM is freed (a bounded wait that an abort does not cut short)
        if (elect_one()) umma_commit(done);
        __syncwarp();
        if (!warp_wait_b(done, 0, nullptr) && lane == 0) set_status(p.status, HISA_DEV_TIMEOUT);
    } else if (warp < kBaSoftWarps) {
        // --------------------------------------------------------- softmax
        const int set = warp >> 2, quad = warp & 3;
        const int r = quad * 32 + lane;                       // MMA row: (row of the group, head)
        const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t ts = tmem_base + lane_off + set * 128, to = tmem_base + lane_off + 256 + set * 128;
        const int rr = r / p.G, hh = r - rr * p.G;
        const bool mine = quad * 32 < p.R * p.G;              // a warp with no row of the group only keeps step
        float2* ml = reinterpret_cast<float2*>(smem + L::ml);
        const float* qs = reinterpret_cast<const float*>(smem + L::qs);
        uint32_t sn = 0, seg = 0, vbase = 0;
        while (ok && cur.next<false>(p, &sg)) {
            const int row = sg.g * p.R + rr;
            const bool live = rr < p.R && row < p.n_q;
            int b = -1, t = -1;
            if (live) t = query_position(p.q_seq, p.q_pos, p.len, p.batch, p.cap, row, &b);
            const int2* list = p.list + static_cast<size_t>(sg.g) * p.lcap;
            const int np = p.pieces[sg.g];
            const uint32_t* bits = p.R > 1 && p.blocks && t >= 0 ? p.bits + static_cast<size_t>(row) * p.W : nullptr;
            float c2 = p.scale_log2;
            float m = -INFINITY, l = 0.f;
            // which of tile j's 128 tokens this row sees (every one in an MMA row without a
            // query, so that it costs its warp nothing), and whether the tile has tokens that
            // no row of the group sees
            uint32_t mw[4];
            bool tail = false;
            auto look = [&](int j) {
                mw[0] = mw[1] = mw[2] = mw[3] = live ? 0u : 0xffffffffu;
                tail = false;
                const int e0 = (sg.t0 + j) * p.S;
#pragma unroll 1
                for (int s = 0; s < p.S; ++s) {
                    if (e0 + s >= np) break;
                    const int2 pc = list[e0 + s];
                    tail |= (pc.x & 255) < p.PB;
                    const int start = pc.y * p.PB;
                    int n = (pc.x >> 8) == b ? min(max(t + 1 - start, 0), p.PB) : 0;
                    if (bits && n > 0) {
                        const int blk = start / p.B;
                        if (!((bits[blk >> 5] >> (blk & 31)) & 1u)) n = 0;
                    }
                    const int c0 = s * p.PB;
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int lo = max(c0 - w * 32, 0), hi = min(c0 + n - w * 32, 32);
                        if (hi > lo) mw[w] |= (hi == 32 ? 0xffffffffu : (1u << hi) - 1u) & ~((1u << lo) - 1u);
                    }
                }
            };
            look(set);
            for (int j = set; j < sg.n; j += 2, ++sn) {
                if (!(ok = warp_wait_b(sfull + set, sn & 1, abort_flag))) break;
                tc_fence_after();
                if (FP4) c2 = qs[(seg & 1) * 128 + r];
                if (!FP4 && tail) {
                    // V rows past the last token any row sees: zeros, for 0 * NaN is NaN
                    const uint32_t vi = vbase + j;
                    if (!(ok = warp_wait_b(vfull + vi % kR, (vi / kR) & 1, abort_flag))) break;
                    const int e = (sg.t0 + j) * p.S + r / p.PB;
                    if (e < np && r % p.PB >= (list[e].x & 255)) {
                        uint8_t* v = smem + L::v0 + (vi % kR) * L::tile + r * 128;
                        for (int a = 0; a < D / 64; ++a)
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                *reinterpret_cast<uint4*>(v + a * 16384 + c * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_async_smem();
                }
                if (mine) {
                    // Most rows see a whole tile or, when it is in the list for another row of
                    // the group, nothing of it: then a row is on or off, and no element is looked
                    // at alone.  An off row's elements become 2^-200 = 0.
                    const bool full = (mw[0] & mw[1] & mw[2] & mw[3]) == 0xffffffffu, none = (mw[0] | mw[1] | mw[2] | mw[3]) == 0u;
                    const bool whole_rows = __all_sync(0xffffffffu, full || none);
                    if (__all_sync(0xffffffffu, none || !live)) {
                        // no row of the warp sees the tile: P is zero
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) w[i] = 0u;
#pragma unroll
                        for (int c = 0; c < 4; ++c) tmem_st16(ts + c * 16, w);
                        tmem_st_wait();
                    } else if (whole_rows) {
                        softmax_tile<D, FP4, false>(ts, to, mw, full, j < 2, c2, m, l);
                    } else {
                        softmax_tile<D, FP4, true>(ts, to, mw, full, j < 2, c2, m, l);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(pfull + set);
                if (j + 2 < sg.n) look(j + 2);
            }
            if (!ok) break;
            vbase += sg.n;
            // the segment's output: both sets' parts merged
            // (the wait for the P V MMAs comes first: they waited for every warp to have
            // read the last segment's maxima and sums)
            if (!(ok = warp_wait_b(odone, seg & 1, abort_flag))) break;
            tc_fence_after();
            ml[set * 128 + r] = make_float2(m, l);
            __syncwarp();
            if (lane == 0) mbar_arrive(mlbar);
            if (!(ok = warp_wait_b(mlbar, seg & 1, abort_flag))) break;
            const float2 a = ml[r], c = ml[128 + r];
            const bool two = sg.n > 1;
            const float M = two ? fmaxf(a.x, c.x) : a.x;
            const float wa = a.x == -INFINITY ? 0.f : ex2_approx(a.x - M);
            const float wc = !two || c.x == -INFINITY ? 0.f : ex2_approx(c.x - M);
            const float lsum = wa * a.y + (two ? wc * c.y : 0.f);
            const bool whole = sg.n == sg.T;
            const float inv = whole ? (lsum > 0.f ? p.out_mul / lsum : 0.f) : 1.f;
            const size_t orow = static_cast<size_t>(row) * p.Hq + sg.h * p.G + hh;
            const int slot = 2 * blockIdx.x + (sg.t0 == 0 ? 1 : 0);
            if (mine) {
#pragma unroll 1
                for (int cc = set * (D / 32); cc < (set + 1) * (D / 32); ++cc) {
                    uint32_t o0[16], o1[16];
                    __syncwarp();
                    tmem_ld16_nowait(tmem_base + lane_off + 256 + cc * 16, o0);
                    if (two) tmem_ld16_nowait(tmem_base + lane_off + 384 + cc * 16, o1);
                    tmem_ld_wait();
                    float o[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        o[i] = wa > 0.f ? wa * __uint_as_float(o0[i]) : 0.f;
                        if (two && wc > 0.f) o[i] = fmaf(wc, __uint_as_float(o1[i]), o[i]);
                        o[i] *= inv;
                    }
                    if (live && whole) {
                        uint4* out = reinterpret_cast<uint4*>(p.out + orow * D + cc * 16);
                        out[0] = make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
                        out[1] = make_uint4(pack_bf16(o[8], o[9]), pack_bf16(o[10], o[11]), pack_bf16(o[12], o[13]),
                                            pack_bf16(o[14], o[15]));
                    } else if (live) {
                        float4* out = reinterpret_cast<float4*>(p.part_o + (static_cast<size_t>(slot) * 128 + r) * D + cc * 16);
#pragma unroll
                        for (int i = 0; i < 4; ++i) out[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                }
                if (set == 0 && live) {
                    if (!whole) p.part_ml[slot * 128 + r] = make_float2(M, lsum);
                    else if (p.lse) p.lse[orow] = lsum > 0.f ? (M + log2f(lsum)) * 0.6931471805599453f : -INFINITY;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(oempty);
            ++seg;
        }
        if (!ok && lane == 0) {
            *abort_flag = 1;
            set_status(p.status, HISA_DEV_TIMEOUT);
        }
    } else if (FP4) {
        // ------------------------------------------------------ dequantise
        const int dw = warp - kBaWarpDeq;
        uint32_t it = 0, seg = 0;
        while (ok && cur.next<false>(p, &sg)) {
            const int2* list = p.list + static_cast<size_t>(sg.g) * p.lcap;
            const int np = p.pieces[sg.g];
            if (seg > 0 && !(ok = warp_wait_b(qempty, (seg - 1) & 1, abort_flag))) break;
            {
                // query row r of the MMA, scaled by a power of two so that its largest element
                // lies in [2^14, 2^15): in f16 then no element loses more than 2^-40 of that
                const int r = dw * 32 + lane;
                const int rr = r / p.G, row = sg.g * p.R + rr;
                const bool live = rr < p.R && row < p.n_q;
                const uint4* src = reinterpret_cast<const uint4*>(
                    p.q + (live ? (static_cast<size_t>(row) * p.Hq + sg.h * p.G + (r - rr * p.G)) * D : 0));
                uint32_t mxb = 0;
#pragma unroll 4
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 x = live ? src[c] : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) mxb = max(mxb, max(w[i] & 0x7FFF0000u, (w[i] & 0x7FFFu) << 16));
                }
                const float mxq = __uint_as_float(mxb);
                const int ex = mxq > 0.f ? min(14 - ilogbf(mxq), 120) : 0;
                const float up = __int_as_float((ex + 127) << 23);
                reinterpret_cast<float*>(smem + L::qs)[(seg & 1) * 128 + r] = ldexpf(p.scale_log2, -ex);
#pragma unroll 4
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 x = live ? src[c] : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                    uint32_t o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o[i] = pack_f16(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xFFFF0000u) * up);
                    *reinterpret_cast<uint4*>(smem + L::q + sw128_off(r, c)) = make_uint4(o[0], o[1], o[2], o[3]);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(qfull);
            }
            ++seg;
            constexpr int kCh = D / 32;       // 16-byte chunks of codes (32 elements) per row
            constexpr int kRows = 32 / kCh;   // rows a warp expands at a time
            const int ch = lane % kCh, rl = lane / kCh;
            for (int j = 0; j < sg.n; ++j, ++it) {
                // rows that hold a token some row sees; the others become zeros
                const int r = dw * 32 + lane, s = r / p.PB, e = (sg.t0 + j) * p.S + s;
                const uint32_t seen = __ballot_sync(0xffffffffu, e < np && r - s * p.PB < (list[min(e, np - 1)].x & 255));
                const int rs = it % (kRaw ? kRaw : 1), slot = it % kR;
                const uint32_t use = it / kR;
                if (!(ok = warp_wait_b(rfull + rs, (it / (kRaw ? kRaw : 1)) & 1, abort_flag))) break;
                const uint8_t* raw = smem + L::raw0 + rs * L::raw;
                for (int kv = 0; kv < 2; ++kv) {
                    if (use > 0 && !(ok = warp_wait_b((kv ? vempty : kempty) + slot, (use - 1) & 1, abort_flag))) break;
                    uint8_t* dst = smem + (kv ? L::v0 : L::k0) + slot * L::tile;
#pragma unroll
                    for (int i = 0; i < kCh; ++i) {
                        const int rw = i * kRows + rl, row = dw * 32 + rw;
                        uint4 x = *reinterpret_cast<const uint4*>(raw + kv * L::raw_codes + row * (D / 2) + ch * 16);
                        const uint32_t sc2 = *reinterpret_cast<const uint16_t*>(raw + 2 * L::raw_codes + kv * L::raw_scales +
                                                                                row * (D / 16) + ch * 2);
                        uint32_t sch = e4m3x2_to_f16(sc2);
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
                            e2m1x8_to_f16(qq == 0 ? w[0] : qq == 1 ? w[1] : qq == 2 ? w[2] : w[3], f);
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
                    if (lane == 0) mbar_arrive((kv ? vfull : kfull) + slot);
                }
                if (!ok) break;
                if (lane == 0) mbar_arrive(rempty + rs);
            }
        }
        if (!ok && lane == 0) {
            *abort_flag = 1;
            set_status(p.status, HISA_DEV_TIMEOUT);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kBaWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
}

// ------------------------------------------------------------------- join

// The groups that no single segment covered.  Group x = (key head, group) is
// tiles [a, a + T) of all; the CTA whose run holds tile y is
// ((y + 1) * n - 1) / all with n CTAs at work, the first of them left its part
// in its slot 1, the others in their slots 0.  W warps take every W-th part of
// an MMA row (8 where few rows are split over many CTAs, whose parts one warp
// would fetch one after another: 63 parts of 4 KB took 24 us; else 1), and
// their sums are added in a fixed order.  Also the zero output of groups
// without a tile.
template <int D, int W>
__global__ void __launch_bounds__(256) join_kernel(const BattnParams p, int grid) {
    __shared__ float s_acc[W > 1 ? W : 1][D];
    __shared__ float s_sum[W];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int x = blockIdx.x;
    const int h = x / p.groups, g = x - h * p.groups;
    const int r = W > 1 ? static_cast<int>(blockIdx.y) : static_cast<int>(blockIdx.y) * 8 + warp;
    const int rr = r / p.G, row = g * p.R + rr;
    if (rr >= p.R || row >= p.n_q) return;
    const int t0 = __ldcg(p.tile0 + g), T = __ldcg(p.tile0 + g + 1) - t0;
    const long long tot = __ldcg(p.tile0 + p.groups), all = tot * p.Hkv;
    const size_t orow = static_cast<size_t>(row) * p.Hq + h * p.G + (r - rr * p.G);
    constexpr int E = D / 32;   // elements per lane
    float acc[E];
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = 0.f;
    float M = -INFINITY, sum = 0.f;
    if (T > 0) {
        const long long a = h * tot + t0, n = min(static_cast<long long>(grid), all);
        const int c0 = static_cast<int>(((a + 1) * n - 1) / all), c1 = static_cast<int>(((a + T) * n - 1) / all);
        if (c0 == c1) return;   // finished in place
        for (int c = c0 + lane; c <= c1; c += 32) M = fmaxf(M, __ldcg(p.part_ml + (2 * c + (c == c0 ? 1 : 0)) * p.prow + r).x);
        M = warp_max(M);
#pragma unroll 4
        for (int c = c0 + (W > 1 ? warp : 0); c <= c1; c += W) {
            const size_t part = static_cast<size_t>(2 * c + (c == c0 ? 1 : 0)) * p.prow + r;
            const float2 v = __ldcg(p.part_ml + part);
            const float w = v.x == -INFINITY ? 0.f : ex2_approx(v.x - M);
            sum += w * v.y;
            const float* po = p.part_o + part * D + lane * E;
            if (E == 4) {
                const float4 o = __ldcg(reinterpret_cast<const float4*>(po));
                acc[0] += w * o.x;
                acc[1] += w * o.y;
                acc[E - 2] += w * o.z;
                acc[E - 1] += w * o.w;
            } else {
                const float2 o = __ldcg(reinterpret_cast<const float2*>(po));
                acc[0] += w * o.x;
                acc[1] += w * o.y;
            }
        }
    }
    if (W > 1) {
#pragma unroll
        for (int i = 0; i < E; ++i) s_acc[warp][lane * E + i] = acc[i];
        if (lane == 0) s_sum[warp] = sum;
        __syncthreads();
        if (warp > 0) return;
#pragma unroll
        for (int w = 1; w < W; ++w) {
#pragma unroll
            for (int i = 0; i < E; ++i) acc[i] += s_acc[w][lane * E + i];
            sum += s_sum[w];
        }
    }
    const float inv = sum > 0.f ? p.out_mul / sum : 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] *= inv;
    uint32_t* out = reinterpret_cast<uint32_t*>(p.out + orow * D + lane * E);
    out[0] = pack_bf16(acc[0], acc[1]);
    if (E == 4) out[1] = pack_bf16(acc[E - 2], acc[E - 1]);
    if (lane == 0 && p.lse) p.lse[orow] = sum > 0.f ? (M + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

template <int D, bool FP4>
cudaError_t launch_typed(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm, const BattnParams& p, int grid,
                         cudaStream_t s) {
    using L = BaLayout<D, FP4>;
    cudaError_t e = smem_limit(reinterpret_cast<const void*>(battn_kernel<D, FP4>), L::total);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (!p.direct) {
        const size_t bits = p.blocks && p.R == 1 ? static_cast<size_t>(p.W) * 4 : 0;
        e = smem_limit(reinterpret_cast<const void*>(plan_kernel), bits);
        if (e != cudaSuccess) return e;
        cfg.gridDim = dim3(static_cast<unsigned>(p.groups));
        cfg.blockDim = dim3(kPlanThreads);
        cfg.dynamicSmemBytes = bits;
        e = cudaLaunchKernelEx(&cfg, plan_kernel, p);
        if (e != cudaSuccess) return e;
    }
    if (p.dec) {
        e = launch_battn_dec(qm, km, vm, p, FP4, grid, s);
    } else {
        cfg.gridDim = dim3(static_cast<unsigned>(grid));
        cfg.blockDim = dim3(L::threads);
        cfg.dynamicSmemBytes = L::total;
        e = cudaLaunchKernelEx(&cfg, battn_kernel<D, FP4>, qm, km, vm, p);
    }
    if (e != cudaSuccess) return e;
    const unsigned items = static_cast<unsigned>(p.groups) * p.Hkv;
    const bool spread = 8 * items <= static_cast<unsigned>(grid);   // eight parts or more to a (key head, group)
    cfg.gridDim = dim3(items, static_cast<unsigned>(spread ? p.R * p.G : (p.R * p.G + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return spread ? cudaLaunchKernelEx(&cfg, join_kernel<D, 8>, p, grid) : cudaLaunchKernelEx(&cfg, join_kernel<D, 1>, p, grid);
}

}  // namespace

size_t battn_layout(BattnParams& p, void* ws) {
    // Groups of rows where there are more rows than sequences.  Over whole prefixes a group
    // reads once what each of its rows would; over kept blocks it reads their union, which
    // pays with some rows to a group and some groups, and where the kernel for lone rows does
    // not serve (64 rows of G = 32: 72 and 92 us).  In groups and alone, us a call:
    //   whole prefixes, 8 sequences of 32K keys, 2 key heads, G = 8, rows of each
    //                      2          3          4          8
    //     bf16          81  89     85 116     78 158     84 255     (G = 1: 2 rows 76  86)
    //     4 bits        77  57     80  75     74  92     78 165     (G = 1: 2 rows 71  53)
    //   64 kept of 256 blocks of 128, one sequence, 2 key heads, rows
    //                     64         96        128        192        512
    //     bf16, G = 8   59  54     69  69     76  85     80 117    129 277   (4096: 676 2105)
    //     bf16, G = 1   62  51     76  67     88  83     90 115    116 274
    //     4 bits, G = 8 58  63     69  82     78 101     84 139    146 337
    //     4 bits, G = 1 63  59     77  79     93  98    102 137    117 333
    //   8 sequences, bf16, G = 8: 9 rows of each 86 and 62, 32 rows 104 and 166
    //   256 kept of 2048 blocks of 16, bf16, G = 8: 96 rows 81 and 53, 256 rows 125 and 112
    //   (4 bits 80 and 84, 116 and 188)
    // The rule takes the slower side for two or three 4-bit rows over a whole prefix, for bf16
    // chunks of a few hundred rows over small blocks, and at G = 1 from about 130 to 255 rows.
    p.G = p.Hq / p.Hkv;
    const bool sparse = p.mb > 0;
    const int most = 128 / p.G;
    const bool many = p.n_q >= 96 && p.n_q >= 2ll * most * p.batch;
    p.R = p.n_q > p.batch && (!sparse || p.G > kBattnDecHeads || many) ? most : 1;
    p.groups = (p.n_q + p.R - 1) / p.R;
    p.PB = sparse && p.B < 128 ? p.B : 128;
    p.S = 128 / p.PB;
    p.ppb = sparse && p.B > 128 ? p.B / 128 : 1;
    p.W = sparse ? ((p.cap - 1) / p.B + 32) / 32 : 0;
    const long long seqs = p.R < p.batch ? p.R : p.batch;
    long long lcap = seqs * ((p.cap - 1) / p.PB + 1);
    if (sparse) {
        const long long kept = static_cast<long long>(p.R) * p.mb * p.ppb;
        if (kept < lcap) lcap = kept;
    }
    p.lcap = lcap > 0x7fffffff ? -1 : static_cast<int>(lcap);   // -1: refused by the caller
    uint8_t* b = static_cast<uint8_t*>(ws);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        uint8_t* r = b + off;
        off += up256(bytes);
        return r;
    };
    p.list = reinterpret_cast<int2*>(take(static_cast<size_t>(p.groups) * lcap * 8));
    p.pieces = reinterpret_cast<int*>(take(static_cast<size_t>(p.groups) * 4));
    p.tiles = reinterpret_cast<int*>(take(static_cast<size_t>(p.groups) * 4));
    p.tile0 = reinterpret_cast<int*>(take(static_cast<size_t>(p.groups + 1) * 4));
    p.bits = reinterpret_cast<uint32_t*>(take(p.R > 1 ? static_cast<size_t>(p.n_q) * p.W * 4 : 0));
    // A lone row with few heads: tokens in the MMA's rows (64 rows of 8192 kept keys, G = 8:
    // 344 us, and 352 us in the 128-row kernel; G = 16: 104 and 110 us; 16 whole prefixes of
    // 64K 4-bit keys, G = 16: 101 and 187 us)
    p.dec = p.R == 1 && p.G <= kBattnDecHeads;
    p.prow = p.dec ? kBattnDecHeads : 128;
    // Whole prefixes of lone rows need no lists: every CTA works the rows' tiles out itself,
    // which saves a launch until there are many rows to go through (one row 21.5 us, 24.0 us
    // with a plan; 1024 rows 60.5 and 63.4 us; 4096 rows 215 and 199 us).
    p.direct = p.dec && !sparse && p.n_q <= kBattnDirectRows;
    const size_t parts = static_cast<size_t>(2) * kBattnMaxSms * (p.dec ? 2 : 1) * p.prow;
    p.part_o = reinterpret_cast<float*>(take(parts * p.d * 4));
    p.part_ml = reinterpret_cast<float2*>(take(parts * 8));
    return off;
}

cudaError_t launch_battn(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm, const BattnParams& p, bool fp4,
                         int sms, cudaStream_t s) {
    const int grid = (sms < kBattnMaxSms ? sms : kBattnMaxSms) * (p.dec && !fp4 ? 2 : 1);   // CTAs per SM
    if (fp4)
        return p.d == 128 ? launch_typed<128, true>(qm, km, vm, p, grid, s) : launch_typed<64, true>(qm, km, vm, p, grid, s);
    return p.d == 128 ? launch_typed<128, false>(qm, km, vm, p, grid, s) : launch_typed<64, false>(qm, km, vm, p, grid, s);
}

}  // namespace hisa
