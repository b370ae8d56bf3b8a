// Shared by the two forms of the attention over the 8-bit cache: arguments,
// geometry and the codes' conversion.
#pragma once

#include "attn_math.cuh"
#include "jsv_internal.cuh"
#include "kv_internal.cuh"
#include "sm100.cuh"

#include <math.h>

namespace jsv {

using namespace sm100;

constexpr int kMaxTreeNodes = 512;
constexpr int kTreeWords = kMaxTreeNodes / 32;
constexpr float kMaxSlack = 8.f;             // log2 units a score may pass the running maximum by
constexpr float kWeightShift = 64.f;         // 2^6: weights are held as 2^6 e vs / vref in fp16
constexpr int kMaxSplits = 64;
// V scales up to 1e-37 count as zero (the reciprocal of a reference scale stays
// finite), and none is taken as the reference below 2^-64 of the largest before
// it (an accumulator of 2^45 stays finite when it is rescaled by as much).
constexpr float kMinScale = 1.0e-37f;
constexpr float kScaleRange = 5.421010862427522e-20f;

struct Kv8Params {
    BatchArgs a;
    jsv_kv8 c;
    const uint16_t *q, *k, *v;
    uint16_t *out;
    float scale_log2;
    int S, C;                                // most splits of a request, units a split aims at
    int by_tiles;                            // a unit: 1 = a 128-slot tile, 0 = a page
    float *ws_o, *ws_ml;                     // [S][T*Hq][D], [S][T*Hq][2]
};

// The request's descriptors, with the 8-bit table's row checked too.
__device__ __forceinline__ bool load_request_kv8(const Kv8Params &p, int b, Request &r) {
    if (!load_request(p.a, b, r)) return false;
    if (r.P / 16 > p.c.max_pages_per_req) {
        flag_error(p.a.dev_status, JSV_ERR_DEVICE_INPUT);
        return false;
    }
    return true;
}

// What a request's splits share out: its pages, or its 128-slot tiles, of the
// 8-bit pages and, from the first bf16 slot on, of the others, which count
// twice (copied, masked, and Q brought back to bf16 for the first: about twice
// the cycles).
__device__ __forceinline__ int request_pages(const Request &r) { return (r.P + r.n + 15) / 16; }
__device__ __forceinline__ int prefix_tiles(const Request &r) { return (r.P / 16 + 7) / 8; }
__device__ __forceinline__ int request_units(const Kv8Params &p, const Request &r) {
    return p.by_tiles ? prefix_tiles(r) + 2 * (((r.P & 15) + r.n + 127) / 128) : request_pages(r);
}
// The tile that starts at a unit (in the middle of a bf16 tile: the next).
__device__ __forceinline__ int unit_tile(int u, int pre_tiles) {
    return u <= pre_tiles ? u : pre_tiles + (u - pre_tiles + 1) / 2;
}
// Splits of a request of `units`: about C units each, at most S.
__device__ __forceinline__ int unit_splits(int units, int C, int S) { return max(1, min(S, (units + C - 1) / C)); }

// A K scale as it is used: an infinite one makes NaN of the codes that are zero, and
// so of the scores, whatever the sign of their finished sums.
__device__ __forceinline__ float finite_or_nan(float s) { return fabsf(s) < INFINITY ? s : __uint_as_float(0x7fc00000u); }

// 1 / x to 2^-23 over the whole range of x, without a division's code.
__device__ __forceinline__ float fast_rcp(float x) {
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp16 from two fp32, the first in the low half.
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Four codes to fp16, exactly.  An int8 code u - 128 comes from the fp16
// number 1024 + u, whose low byte is u.
template <int FMT>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if constexpr (FMT == JSV_KV8_E4M3) {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t l = __byte_perm(u, 0x64646464u, 0x4140), h = __byte_perm(u, 0x64646464u, 0x4342);
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(l), "r"(0x64806480u));
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(h), "r"(0x64806480u));
    }
}

// TMEM: 32 lanes x 16 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// The tcgen05 form (tree_attention_kv8_tiles.cu).
cudaError_t launch_kv8_tiles(const Kv8Params &p, cudaStream_t st);

}  // namespace jsv
