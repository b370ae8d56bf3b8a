// Full pages of the bf16 cache written to the 8-bit cache (include/jsv.h,
// jsv_kv8_quantize).
//
// Per (page, KV head) block of 16 x D values, of K and of V:
//     scale = amax / qmax,  code = round(x * qmax / amax)
// x * qmax is exact in fp32 (8 + 7 significand bits), and the fp32 quotient
// rounds to the same code as the exact one: a code boundary is a number of at
// most 8 bits, the quotient of a 15-bit and an 8-bit number that is not equal
// to it is at least 2^-16 of its size away, and fp32 is off by 2^-24.  So the
// codes are the correctly rounded ones, ties included.
//
// One warp per block of a page: the 16 x D values (4 KB at D = 128) stay in
// registers between the maximum and the codes, so each value is read once.
// A CTA's warps take the KV heads of one page together, which makes its loads
// whole rows of the cache.  Bound by HBM traffic at prefill sizes (2 bytes in,
// 1 out a value: four prompts of 9,000 to 16,000 tokens take 59 us, 4.6 TB/s, 70% of
// the measured copy rate) and by launch latency after a verify step, where a
// request completes a page or none (6.6 us under ncu).  64 registers, for 32
// resident warps; 32-bit item indexes and the quotient from one reciprocal a
// block took prefill from 109 us to that.
#include "jsv_internal.cuh"
#include "kv_internal.cuh"
#include "sm100.cuh"

#include <cuda_fp8.h>

#include <algorithm>

namespace jsv {

namespace {

constexpr int kQuantThreads = 256;
constexpr int kQuantWarps = kQuantThreads / 32;

struct QuantParams {
    BatchArgs a;
    jsv_kv8 c;
    const uint16_t *k, *v;
    const int32_t *from_len, *to_len;
};

// Logical pages [lo, hi) of request b that are to be written; false: refused.
__device__ __forceinline__ bool quant_range(const QuantParams &p, int b, int &lo, int &hi) {
    const int f = p.from_len ? p.from_len[b] : 0, t = p.to_len[b];
    lo = f / 16;
    hi = t / 16;
    return f >= 0 && f <= t && hi <= p.a.max_pages_per_req && hi <= p.c.max_pages_per_req;
}

template <int FMT>
__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d) {
    if constexpr (FMT == JSV_KV8_E4M3) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
        return lo | (hi << 16);
    } else {
        // 1.5 * 2^23 + x: the sum is rounded to a whole number, ties to even,
        // whose low byte is the code
        constexpr float kMagic = 12582912.f;
        const uint32_t lo = __byte_perm(__float_as_uint(a + kMagic), __float_as_uint(b + kMagic), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(c + kMagic), __float_as_uint(d + kMagic), 0x0040);
        return __byte_perm(lo, hi, 0x5410);
    }
}

template <int D, int FMT>
__global__ void __launch_bounds__(kQuantThreads, 4)
kv8_quantize_kernel(const QuantParams p) {
    pdl_allow_dependents();
    pdl_wait_predecessor();
    extern __shared__ int first[];                  // [B + 1] pages before request b
    __shared__ int warp_sums[kQuantWarps];
    const BatchArgs &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // exclusive prefix of the requests' page counts, the same in every CTA
    const int per = (a.B + kQuantThreads - 1) / kQuantThreads;
    const int b_lo = min((int)threadIdx.x * per, a.B), b_hi = min(b_lo + per, a.B);
    int sum = 0;
    for (int b = b_lo; b < b_hi; ++b) {
        int lo, hi;
        if (quant_range(p, b, lo, hi)) sum += hi - lo;
        else if (blockIdx.x == 0) flag_error(a.dev_status, JSV_ERR_DEVICE_INPUT);
    }
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += u;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int at = incl - sum;
    for (int w = 0; w < warp; ++w) at += warp_sums[w];
    for (int b = b_lo; b < b_hi; ++b) {
        int lo, hi;
        first[b] = at;
        if (quant_range(p, b, lo, hi)) at += hi - lo;
    }
    if (b_hi == a.B && b_lo < a.B) first[a.B] = at;
    __syncthreads();
    const int pages = first[a.B];

    constexpr int kLanesPerRow = D / 8;             // 16-byte loads of a row
    constexpr int kRowsPerLoad = 32 / kLanesPerRow;
    constexpr int kLoads = 16 / kRowsPerLoad;
    constexpr float kQmax = FMT == JSV_KV8_E4M3 ? 448.f : 127.f;
    const int row = lane / kLanesPerRow, col = lane % kLanesPerRow;
    // items in the order page, K or V, head: neighbouring warps read
    // neighbouring heads of one page
    const long long all = (long long)pages * 2 * a.Hkv;
    if (pages > p.c.num_pages && blockIdx.x == 0 && threadIdx.x == 0)      // some page is to be written twice
        flag_error(a.dev_status, JSV_ERR_DEVICE_INPUT);
    // num_pages * Hkv * 16 is below 2^31, so these stay far inside 32 bits
    const unsigned items = pages > p.c.num_pages ? 0u : (unsigned)all, heads = (unsigned)a.Hkv;
    for (unsigned it = blockIdx.x * kQuantWarps + warp; it < items; it += gridDim.x * kQuantWarps) {
        const unsigned pk = it / heads;
        const int g = (int)(it - pk * heads), is_v = (int)(pk & 1), pr = (int)(pk >> 1);
        int b = 0, top = a.B;                       // the last b with first[b] <= pr
        while (top - b > 1) {
            const int mid = (b + top) / 2;
            if (first[mid] <= pr) b = mid;
            else top = mid;
        }
        int lo, hi;
        quant_range(p, b, lo, hi);
        const int lp = lo + pr - first[b];
        const int from = a.page_table[(size_t)b * a.max_pages_per_req + lp];
        const int to = p.c.page_table[(size_t)b * p.c.max_pages_per_req + lp];
        if (from < 0 || from >= a.num_pages || to < 0 || to >= p.c.num_pages) {
            if (lane == 0) flag_error(a.dev_status, JSV_ERR_DEVICE_INPUT);
            continue;
        }
        const uint16_t *in = (is_v ? p.v : p.k) + ((size_t)from * 16 * a.Hkv + g) * D;
        const long long in_elems = (long long)a.num_pages * 16 * a.Hkv * D;
        const size_t block = (size_t)to * a.Hkv + g;
        uint8_t *out = (is_v ? p.c.v : p.c.k) + block * 16 * D;
        uint4 x[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const size_t o = (size_t)(i * kRowsPerLoad + row) * a.Hkv * D + col * 8;
            x[i] = make_uint4(0, 0, 0, 0);
            if (JSV_IN_BOUNDS((in - (is_v ? p.v : p.k)) + o + 7, in_elems, a.dev_status))
                x[i] = __ldg(reinterpret_cast<const uint4 *>(in + o));
        }
        // largest magnitude as bf16 bits: infinities and NaN come out on top
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            m = __vmaxu2(m, __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                                     __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu)));
        m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
        const bool bad = m >= 0x7f80u;
        const float amax = __uint_as_float(m << 16);
        // at either end of the range both sides of the quotient are taken
        // 2^-32 or 2^64 times as large, so that neither x * qmax nor 1 / amax
        // overflows (exact, but for what has code 0)
        const float size = amax > 1.0e30f ? 2.3283064365386963e-10f : amax < 1.0e-30f ? 1.8446744073709552e19f : 1.f;
        const float mul = size * kQmax, div = m ? amax * size : 1.f, inv = 1.f / div;
        // y / div from the reciprocal by Markstein's correction (P. Markstein,
        // IBM Journal of Research and Development 34, 1990): the remainder of the
        // first quotient is exact in one fma, and corrects it to 2^-24 and, where the quotient is
        // a number of few bits (a tie between two codes), to that number
        auto code = [&](float x) {
            const float y = x * mul, q = y * inv;
            const float exact = fmaf(fmaf(-q, div, y), inv, q);
            return FMT == JSV_KV8_E4M3 ? copysignf(exact, x) : exact;      // the sum loses the sign of -0
        };
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            float f[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[2 * j] = code(__uint_as_float(w[j] << 16));
                f[2 * j + 1] = code(__uint_as_float(w[j] & 0xffff0000u));
            }
            uint2 c = make_uint2(code4<FMT>(f[0], f[1], f[2], f[3]), code4<FMT>(f[4], f[5], f[6], f[7]));
            if (bad) c = make_uint2(0, 0);
            const int o = (i * kRowsPerLoad + row) * D + col * 8;
            if (JSV_IN_BOUNDS(block * 16 * D + o + 7, (long long)p.c.num_pages * a.Hkv * 16 * D, a.dev_status))
                *reinterpret_cast<uint2 *>(out + o) = c;
        }
        if (lane == 0) {
            if (bad) flag_error(a.dev_status, JSV_ERR_DEVICE_INPUT);
            (is_v ? p.c.v_scale : p.c.k_scale)[block] = bad ? __uint_as_float(0x7fc00000u) : amax / kQmax;
        }
    }
}

}  // namespace

template <int D, int FMT>
static cudaError_t launch_quantize(const QuantParams &p, cudaStream_t st) {
    static PerDeviceOnce once;
    cudaError_t e = prefer_max_shared(kv8_quantize_kernel<D, FMT>, once);
    if (e != cudaSuccess) return e;
    // the pages to write are known on the device only: as many CTAs as are
    // resident at once, each walking the items
    e = launch_pdl(kv8_quantize_kernel<D, FMT>, dim3(4 * device_sm_count()), dim3(kQuantThreads),
                   (p.a.B + 1) * sizeof(int), st, p);
    count_launches(1);
    return e;
}

cudaError_t launch_kv8_quantize(const BatchArgs &a, const jsv_kv8 &c, const uint16_t *k_cache,
                                const uint16_t *v_cache, const int32_t *from_len, const int32_t *to_len,
                                cudaStream_t st) {
    QuantParams p{a, c, k_cache, v_cache, from_len, to_len};
    if (a.D == 128)
        return c.format == JSV_KV8_E4M3 ? launch_quantize<128, JSV_KV8_E4M3>(p, st)
                                        : launch_quantize<128, JSV_KV8_INT8>(p, st);
    return c.format == JSV_KV8_E4M3 ? launch_quantize<64, JSV_KV8_E4M3>(p, st)
                                    : launch_quantize<64, JSV_KV8_INT8>(p, st);
}

}  // namespace jsv
