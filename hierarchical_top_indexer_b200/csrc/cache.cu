// The attention cache's rows: new key and value rows stored (in 4 bits:
// quantised on the way), and rows read back.
//
// A 4-bit row keeps, for each group of 16 elements, the scale
//     s = e4m3(min(448, max |x| / (6 mul)))            (nearest, ties to even)
// and per element the e2m1 code of x / (mul s) (nearest, ties to the even
// code, saturated at 6); it stands for mul * s * code, which is exact in bf16
// (a 4-bit and a 2-bit significand, mul a power of two).  The quotient is
// taken as x * (1 / (mul s)) and cleaned of the product's rounding error by
// rounding to 16 significant bits: x has 8 significant bits, s 4 and a
// rounding boundary of e2m1 3, so a quotient is a boundary exactly or at
// least 2^-8 of it away, and the 2^-23 of the product can neither make nor
// break a tie.
//
// Bound: 2 bytes read and 0.5625 written per element (store; load the other
// way).  One thread per group of the keys and the same of the values: four
// 16-byte loads in flight before it knows its row, two 8-byte stores of codes
// and two bytes of scale; the groups of a row are neighbouring threads.  16384
// tokens of 8 heads of 128 at a random half of the positions, keys and values:
// 4 bits stored in 17.0 us and loaded in 20.0 us (at contiguous positions 16.5
// and 18.7: a token's heads lie apart, so a row is 64 bytes of codes and 8 of
// scales), bf16 21.9 and 23.4 us; both run in turn over other inputs take 40.4
// us for 4 bits, 66% of the measured copy rate.
#include "hisa_kernels.cuh"

namespace hisa {

namespace {

constexpr int kCacheThreads = 256;

// Cache row of token i's head, or -1 (sequence or position out of range).
__device__ __forceinline__ long long cache_row(const CacheParams& p, int i, int h, bool report) {
    const int b = p.seq[i];
    if (b < 0 || b >= p.batch) {
        if (report) set_status(p.status, HISA_DEV_BAD_QUERY);
        return -1;
    }
    const int t = p.pos ? p.pos[i] : p.len[b] - 1;
    if (t < 0 || t >= p.cap) {
        if (report) set_status(p.status, HISA_DEV_CAPACITY);
        return -1;
    }
    return (static_cast<long long>(b) * p.heads + h) * p.cap + t;
}

__device__ __forceinline__ float max_abs16(const uint4& a, const uint4& b) {
    // |bf16| as integers: the order of their bits is the order of the values
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, max(w[i] & 0x7FFF0000u, (w[i] & 0x7FFFu) << 16));
    return __uint_as_float(m);
}

// x * inv rounded to 16 significant bits.
__device__ __forceinline__ float snap16(float x, float inv) {
    return __uint_as_float((__float_as_uint(x * inv) + 0x80u) & 0xFFFFFF00u);
}

// Eight bf16 (four words) as e2m1 codes, the first element in the low bits.
__device__ __forceinline__ uint32_t codes8(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, float inv) {
    const uint32_t w[4] = {w0, w1, w2, w3};
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = snap16(__uint_as_float(w[i] << 16), inv);
        f[2 * i + 1] = snap16(__uint_as_float(w[i] & 0xFFFF0000u), inv);
    }
    uint32_t r;
    asm("{\n\t.reg .b8 c0, c1, c2, c3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c3, %8, %7;\n\t"
        "mov.b32 %0, {c0, c1, c2, c3};\n\t}"
        : "=r"(r)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
    return r;
}

// One row's group of 16 elements in 4 bits.
__device__ __forceinline__ void store_fp4(const uint4& a, const uint4& b, float mul, uint8_t* codes, uint8_t* scale) {
    const float want = __fdiv_rn(max_abs16(a, b), 6.f * mul);
    const __nv_fp8_storage_t s8 = __nv_cvt_float_to_fp8(want, __NV_SATFINITE, __NV_E4M3);
    const float s = __half2float(__nv_cvt_fp8_to_halfraw(s8, __NV_E4M3)) * mul;
    const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
    uint2 c;
    c.x = codes8(a.x, a.y, a.z, a.w, inv);
    c.y = codes8(b.x, b.y, b.z, b.w, inv);
    *reinterpret_cast<uint2*>(codes) = c;
    *scale = s8;
}

__device__ __forceinline__ void load_fp4(const uint2& c, uint8_t scale, float mul, uint4* out) {
    const float s = __half2float(__nv_cvt_fp8_to_halfraw(scale, __NV_E4M3)) * mul;
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t f[4];
        e2m1x8_to_f16(j ? c.y : c.x, f);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f[q]));
            w[4 * j + q] = pack_bf16(v.x * s, v.y * s);   // exact
        }
    }
    __stcs(out, make_uint4(w[0], w[1], w[2], w[3]));
    __stcs(out + 1, make_uint4(w[4], w[5], w[6], w[7]));
}

// Thread (token, head, group of 16 elements), keys and values.
template <bool FP4>
__global__ void __launch_bounds__(kCacheThreads) cache_store_kernel(const CacheParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lg = p.d == 128 ? 3 : 2, groups = 1 << lg;
    const size_t k = static_cast<size_t>(blockIdx.x) * kCacheThreads + threadIdx.x;
    const uint32_t ih = static_cast<uint32_t>(k >> lg), g = static_cast<uint32_t>(k) & (groups - 1);
    if (ih >= static_cast<uint32_t>(p.n) * p.heads) return;
    const uint4* ks = reinterpret_cast<const uint4*>(p.k_rows + k * 16);
    const uint4* vs = reinterpret_cast<const uint4*>(p.v_rows + k * 16);
    const uint4 ka = __ldcs(ks), kb = __ldcs(ks + 1), va = __ldcs(vs), vb = __ldcs(vs + 1);
    const int i = ih / static_cast<uint32_t>(p.heads), h = ih - i * p.heads;
    const long long row = cache_row(p, i, h, h == 0 && g == 0);
    if (row < 0) return;
    const size_t at = (static_cast<size_t>(row) << lg) + g;   // group of the cache
    if (FP4) {
        store_fp4(ka, kb, p.k_mul, static_cast<uint8_t*>(p.k) + 8 * at, p.k_scale + at);
        store_fp4(va, vb, p.v_mul, static_cast<uint8_t*>(p.v) + 8 * at, p.v_scale + at);
    } else {
        uint4* ko = reinterpret_cast<uint4*>(p.k) + 2 * at;
        uint4* vo = reinterpret_cast<uint4*>(p.v) + 2 * at;
        ko[0] = ka;
        ko[1] = kb;
        vo[0] = va;
        vo[1] = vb;
    }
}

// The way back: rows [n, heads, d] bf16 (zero rows where the name is bad).
template <bool FP4>
__global__ void __launch_bounds__(kCacheThreads) cache_load_kernel(const CacheParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lg = p.d == 128 ? 3 : 2, groups = 1 << lg;
    const size_t k = static_cast<size_t>(blockIdx.x) * kCacheThreads + threadIdx.x;
    const uint32_t ih = static_cast<uint32_t>(k >> lg), g = static_cast<uint32_t>(k) & (groups - 1);
    if (ih >= static_cast<uint32_t>(p.n) * p.heads) return;
    const int i = ih / static_cast<uint32_t>(p.heads), h = ih - i * p.heads;
    const long long row = cache_row(p, i, h, h == 0 && g == 0);
    uint4* ko = reinterpret_cast<uint4*>(p.k_out + k * 16);
    uint4* vo = reinterpret_cast<uint4*>(p.v_out + k * 16);
    if (row < 0) {
        const uint4 z = make_uint4(0, 0, 0, 0);
        ko[0] = ko[1] = vo[0] = vo[1] = z;
        return;
    }
    const size_t at = (static_cast<size_t>(row) << lg) + g;
    if (FP4) {
        const uint2 kc = *(reinterpret_cast<const uint2*>(p.k) + at), vc = *(reinterpret_cast<const uint2*>(p.v) + at);
        const uint8_t k8 = p.k_scale[at], v8 = p.v_scale[at];
        load_fp4(kc, k8, p.k_mul, ko);
        load_fp4(vc, v8, p.v_mul, vo);
    } else {
        const uint4* kr = reinterpret_cast<const uint4*>(p.k) + 2 * at;
        const uint4* vr = reinterpret_cast<const uint4*>(p.v) + 2 * at;
        const uint4 ka = kr[0], kb = kr[1], va = vr[0], vb = vr[1];
        __stcs(ko, ka);
        __stcs(ko + 1, kb);
        __stcs(vo, va);
        __stcs(vo + 1, vb);
    }
}

template <typename K>
cudaError_t launch_rows(K kernel, const CacheParams& p, cudaStream_t s) {
    const long long threads = static_cast<long long>(p.n) * p.heads * (p.d / 16);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((threads + kCacheThreads - 1) / kCacheThreads));
    cfg.blockDim = dim3(kCacheThreads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_cache_store(const CacheParams& p, cudaStream_t s) {
    return p.fp4 ? launch_rows(cache_store_kernel<true>, p, s) : launch_rows(cache_store_kernel<false>, p, s);
}

cudaError_t launch_cache_load(const CacheParams& p, cudaStream_t s) {
    return p.fp4 ? launch_rows(cache_load_kernel<true>, p, s) : launch_rows(cache_load_kernel<false>, p, s);
}

}  // namespace hisa
