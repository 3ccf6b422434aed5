// Rotary positions: the rotation that gives the indexer's (and the
// attention's) queries and keys their position, before they are appended,
// stored or scored.
//
// Pair i of a row's rotated part, (a, b), becomes at position p
//     (a', b') = gain * (a cos t - b sin t, b cos t + a sin t),  t = p * w_i
// (transposed: with -t, the gradient of the forward call).  The angle is kept
// as a fraction of a turn in 64-bit fixed point: turns_i = w_i / 2 pi * 2^64,
// and p * turns_i modulo 2^64 drops whole turns exactly, so a position of a
// million is as exact as position 1 (an fp32 product p * w_i would be off by
// 2^-24 p radians, 0.06 at a million).  The fraction is rounded to 32 bits
// (2^-33 of a turn; the rounding of turns_i adds up to 2^-34 at the farthest
// positions) and then to fp32's 24 for sincospi (up to 2^-26 of a turn, in
// the outer half of [-1/2, 1/2]); the rotation is computed in fp32 and rounded
// once to bf16.
//
// Bound: 4 bytes per element (read once, written once).  A block takes a few
// rows and all or some of their heads; it issues its loads first (up to four
// tasks of one or two 16-byte chunks per thread), computes the sine and cosine
// of each (row, pair) once while they are in flight, and every head of the
// row uses them.  4096 rows of 64 heads of 128, 64 of them rotated: 24.5 to
// 26.1 us, 80 to 85% of the measured copy rate.  With 256 threads a block 27.0
// us and with 64 threads of eight tasks 31.6 us where this took 24.7 (small
// blocks load while others store).
#include "hisa_kernels.cuh"

namespace hisa {

namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeTasks = 4;          // per thread
constexpr int kRopeMaxSc = 1024;       // (row, pair) sine and cosine entries per block

// Sine and cosine (times gain) of pair i at position pos.
__device__ __forceinline__ float2 rope_sc(const RopeParams& p, int pos, int i) {
    const uint64_t ph = static_cast<uint64_t>(static_cast<int64_t>(pos)) * p.turns[i];
    const int32_t top = static_cast<int32_t>(static_cast<uint32_t>((ph + 0x80000000ull) >> 32));
    float s, c;
    sincospif(static_cast<float>(top) * 4.656612873077393e-10f, &s, &c);   // 2^-31: units of pi
    if (p.transpose) s = -s;
    return make_float2(c * p.gain, s * p.gain);
}

__device__ __forceinline__ float2 unpack_bf16(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// MODE 0: half layout, 16-byte chunks (a pair of chunks, or an unrotated
// chunk, per task); MODE 1: interleaved layout, a 16-byte chunk per task.
template <int MODE>
__global__ void __launch_bounds__(kRopeThreads) rope_vec_kernel(const __grid_constant__ RopeParams p) {
    __shared__ float2 sc[kRopeMaxSc];
    grid_dependency_wait();
    grid_launch_dependents();
    const int row0 = blockIdx.x * p.rows_blk;
    const int nr = min(p.rows_blk, p.rows - row0);
    const int h0 = blockIdx.y * p.heads_blk;
    const int nh = min(p.heads_blk, p.heads - h0);
    const int np = p.rot >> 1;
    const int pair_tasks = MODE == 0 ? p.rot >> 4 : 0;
    const int th = p.tasks;   // per (row, head)
    const bool in_place = p.x == p.y;
    uint4 va[kRopeTasks], vb[kRopeTasks];
    size_t oa[kRopeTasks];
    int rel[kRopeTasks];   // first pair of the chunk's rotation (-1: copied), -2: no task
    int rr[kRopeTasks];
#pragma unroll
    for (int u = 0; u < kRopeTasks; ++u) {
        const int k = u * kRopeThreads + threadIdx.x;
        rel[u] = -2;
        // k = (row * heads_blk + head) * tasks + task, every factor below 2^10
        const int hr = static_cast<uint32_t>(k) * p.tasks_inv >> 20, t = k - hr * th;
        rr[u] = static_cast<uint32_t>(hr) * p.heads_inv >> 20;
        const int h = hr - rr[u] * p.heads_blk;
        if (rr[u] >= nr || h >= nh) continue;
        const size_t base = (static_cast<size_t>(row0 + rr[u]) * p.heads + h0 + h) * p.d;
        if (MODE == 0) {
            int e = p.off + 8 * t;
            rel[u] = 8 * t;
            if (t >= pair_tasks) {
                e = 8 * (t - pair_tasks);
                if (e >= p.off) e += p.rot;
                rel[u] = in_place ? -2 : -1;
            }
            oa[u] = base + e;
        } else {
            oa[u] = base + 8 * t;
            rel[u] = 8 * t;
        }
        if (rel[u] == -2) continue;
        va[u] = __ldcs(reinterpret_cast<const uint4*>(p.x + oa[u]));
        if (MODE == 0 && rel[u] >= 0) vb[u] = __ldcs(reinterpret_cast<const uint4*>(p.x + oa[u] + np));
    }
    for (int k = threadIdx.x; k < nr * np; k += kRopeThreads) {
        const int r = k / np;
        sc[k] = rope_sc(p, p.pos[row0 + r], k - r * np);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kRopeTasks; ++u) {
        if (rel[u] == -2) continue;
        uint32_t* a = reinterpret_cast<uint32_t*>(&va[u]);
        if (MODE == 0) {
            if (rel[u] >= 0) {
                uint32_t* b = reinterpret_cast<uint32_t*>(&vb[u]);
                const float2* t = sc + rr[u] * np + rel[u];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 x = unpack_bf16(a[i]), y = unpack_bf16(b[i]);
                    const float2 t0 = t[2 * i], t1 = t[2 * i + 1];
                    a[i] = pack_bf16(x.x * t0.x - y.x * t0.y, x.y * t1.x - y.y * t1.y);
                    b[i] = pack_bf16(y.x * t0.x + x.x * t0.y, y.y * t1.x + x.y * t1.y);
                }
                *reinterpret_cast<uint4*>(p.y + oa[u] + np) = vb[u];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = rel[u] + 2 * i - p.off;
                if (e >= 0 && e < p.rot) {
                    const float2 x = unpack_bf16(a[i]);
                    const float2 t = sc[rr[u] * np + (e >> 1)];
                    a[i] = pack_bf16(x.x * t.x - x.y * t.y, x.y * t.x + x.x * t.y);
                }
            }
        }
        *reinterpret_cast<uint4*>(p.y + oa[u]) = va[u];
    }
}

// Any sizes and offsets: a pair, or one unrotated element, per task, by
// 2-byte accesses.  Both elements of a pair belong to one thread, so x may be
// y here too.
__global__ void __launch_bounds__(kRopeThreads) rope_any_kernel(const __grid_constant__ RopeParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int np = p.rot >> 1, th = p.tasks;
    const long long total = static_cast<long long>(p.rows) * p.heads * th;
    for (long long k = static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x; k < total;
         k += static_cast<long long>(gridDim.x) * kRopeThreads) {
        const int t = static_cast<int>(k % th);
        const long long rh = k / th;
        const size_t base = static_cast<size_t>(rh) * p.d;
        if (t < np) {
            const float2 s = rope_sc(p, p.pos[rh / p.heads], t);
            const size_t ia = base + p.off + (p.interleaved ? 2 * t : t);
            const size_t ib = p.interleaved ? ia + 1 : ia + np;
            const float a = __uint_as_float(static_cast<uint32_t>(p.x[ia]) << 16);
            const float b = __uint_as_float(static_cast<uint32_t>(p.x[ib]) << 16);
            const uint32_t w = pack_bf16(a * s.x - b * s.y, b * s.x + a * s.y);
            p.y[ia] = static_cast<uint16_t>(w);
            p.y[ib] = static_cast<uint16_t>(w >> 16);
        } else {
            const int e = t - np;
            const size_t i = base + (e < p.off ? e : e + p.rot);
            if (p.x != p.y) p.y[i] = p.x[i];
        }
    }
}

}  // namespace

cudaError_t launch_rope(RopeParams& p, int sms, cudaStream_t s) {
    const bool rows16 = p.d % 8 == 0;
    const bool half_vec = !p.interleaved && rows16 && p.off % 8 == 0 && p.rot % 16 == 0;
    const bool inter_vec = p.interleaved && rows16 && p.off % 2 == 0;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (!half_vec && !inter_vec) {
        p.tasks = p.rot / 2 + p.d - p.rot;
        const long long total = static_cast<long long>(p.rows) * p.heads * p.tasks;
        const long long blocks = (total + kRopeThreads - 1) / kRopeThreads;
        cfg.gridDim = dim3(static_cast<unsigned>(blocks < 16ll * sms ? blocks : 16ll * sms));
        return cudaLaunchKernelEx(&cfg, rope_any_kernel, p);
    }
    p.tasks = half_vec ? p.rot / 16 + (p.d - p.rot) / 8 : p.d / 8;
    // Tasks per block: four per thread, fewer where the call is too small to
    // give every SM two blocks that way.
    const long long total = static_cast<long long>(p.rows) * p.heads * p.tasks;
    long long want = total / (2ll * sms);
    want = want < kRopeThreads ? kRopeThreads : want > kRopeTasks * kRopeThreads ? kRopeTasks * kRopeThreads : want;
    const int per_row = p.heads * p.tasks;
    if (per_row >= want) {
        p.rows_blk = 1;
        p.heads_blk = static_cast<int>(want / p.tasks);
    } else {
        p.heads_blk = p.heads;
        const int most = kRopeMaxSc / (p.rot / 2);
        p.rows_blk = static_cast<int>(want / per_row);
        if (p.rows_blk > most) p.rows_blk = most;
    }
    p.tasks_inv = (1u << 20) / p.tasks + 1;    // x * inv >> 20 = x / tasks for x, tasks below 2^10
    p.heads_inv = (1u << 20) / p.heads_blk + 1;
    cfg.gridDim = dim3(static_cast<unsigned>((p.rows - 1) / p.rows_blk + 1),   // (rows reach INT_MAX)
                       static_cast<unsigned>((p.heads - 1) / p.heads_blk + 1));
    return half_vec ? cudaLaunchKernelEx(&cfg, rope_vec_kernel<0>, p) : cudaLaunchKernelEx(&cfg, rope_vec_kernel<1>, p);
}

}  // namespace hisa
