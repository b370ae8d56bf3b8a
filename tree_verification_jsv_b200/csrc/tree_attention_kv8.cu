// Tree-causal attention over a prefix held in 8 bits (include/jsv.h,
// jsv_tree_attention_kv8).
//
// Request b's pages are one sequence: floor(P / 16) pages of codes with a
// scale per (page, KV head), then the bf16 pages that hold the rest of the
// prefix and the tree's slots.  For a row (node, query head) of KV head g
//     out = sum_j e_j v_j / sum_j e_j,   e_j = 2^(x_j - m),
//     x_j = log2(e) * scale * <q, k_j>,  k_j = code_j * ks, v_j = code_j * vs.
// A code is exact in fp16, so the products run on fp16 tensor-core operands
// accumulated in fp32: q is scaled by a power of two per row into fp16's range
// (its 8 significand bits stay), the K scale multiplies the fp32 score, and
// the V scale multiplies the fp32 weight before that is rounded to fp16 (11
// bits, 2^-11 of each weight; bf16 output rounds by 2^-8).
//
// Weights of pages with different V scales share one accumulator through a
// reference scale vref: a weight is stored as 2^6 e_j vs / vref.  The reference
// follows the pages' scales up and down: vref is set to a page's scale, and the
// accumulator rescaled, where the scale lies outside vref * [2^-6, 2].  With
// e_j <= 2^8 a stored weight stays below 2^15, inside fp16, and its step there,
// 2^-24 below 2^-14, is at most 2^-25 2^-6 2^6 = 2^-25 of vs: a row whose weight
// lies on a page of small values gets them as exactly as any others.  (A
// reference that only grew lost such pages: 5% off at 2^-27 of the largest
// scale, nothing left at 2^-31.)  The running maximum m moves only when a score
// passes it by 8 (2^8), so most pages need no reduction over the row.
#include "kv8_attention.cuh"

#include <algorithm>

namespace jsv {

using namespace sm100;

namespace {

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

}  // namespace

// ---------------------------------------------------------------------------
// Few rows: warps stream pages, each with a ring and an accumulator of its own
// ---------------------------------------------------------------------------
// With few query rows the work is reading the cache.  A CTA of four warps
// takes (request, KV head, 8*NT packed query rows, split); its warps take the
// split's pages in turn.  One lane keeps kRowStages pages of K and V in flight
// into the warp's own ring (one swizzled 16 x D box each, so that the operand
// reads below have no bank conflicts), and no warp waits for another before
// the merge at the end.
//
// The products are taken transposed, so that the padding of the rows is to 8
// (the MMA's N) and not to 16 (its M): one token of a model with four query
// heads to a KV head has four rows.  Register operands of mma.m16n8k16
// straight from the codes, lane = 4 n + t:
//   S^T = K Q^T     A: keys n and n + 8 of the page; lane t supplies the dims
//                   t*D/4 .. of its keys, four to a k-step, and of Q alike;
//                   the result has keys n, n + 8 of rows 2t, 2t + 1
//   O^T += V^T P^T  B: P as it comes from the exponentials, two 8 x 8 blocks
//                   transposed in registers (movmatrix); A: lane (t, n) reads
//                   keys 2t, 2t+1, 2t+8, 2t+9 at dims n*D/8 .. and pairs the
//                   keys' bytes; rows n and n + 8 of tile i are dims
//                   n*D/8 + 2i and + 2i + 1, so that a lane ends with D/8
//                   neighbouring dims of rows 2t and 2t + 1
//
// Bound by instruction issue and latency more than by HBM: a page costs a warp
// about 400 instructions with int8 codes (their conversion is half), and a call
// about 12 us beside the pages (a chain of dependent loads, the merges, the
// second launch).  One token of 16 requests over 512 to 8192 tokens (int8, 154
// MB) takes 36 us, 4.2 TB/s, 65% of the measured copy rate; over 4096 tokens
// each (e4m3) 32 us; both under host bounds that fit the batch (see plan_of).
// Rows to 16 by the MMA's M, as first built: 70 us for the former.  Three stages,
// eight warps a CTA, five CTAs an SM: no better.
constexpr int kRowWarps = 4;
constexpr int kRowStages = 2;

template <int D, int NT>
struct RowSmem {
    static constexpr int kBlock = 16 * D;                        // codes of one page and head
    static constexpr int kRing = kRowStages * 2 * kBlock;        // a warp's
    static constexpr int kMerge = 8 * NT * D * 4;                // a warp's, over its ring
    static constexpr int kWarp = kRing > kMerge ? kRing : kMerge;
    static constexpr int kTotal = kRowWarps * kWarp + 1024;
    // CTAs an SM that the registers are to leave room for
    static constexpr int kCtas = NT == 1 ? 4 : 3;
};

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int D, int FMT, int NT>
__global__ void __launch_bounds__(kRowWarps * 32, RowSmem<D, NT>::kCtas)
kv8_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Kv8Params p) {
    pdl_allow_dependents();
    using L = RowSmem<D, NT>;
    constexpr int kRows = 8 * NT;
    constexpr int kSteps = D / 16;               // k-steps of a score
    constexpr int kTiles = D / 16;               // 16-dim tiles of the output
    extern __shared__ uint8_t dsmem[];
    __shared__ __align__(8) uint64_t full[kRowWarps][kRowStages];
    __shared__ uint32_t anc[kRows][kTreeWords];
    __shared__ int par_sh[kMaxTreeNodes];
    __shared__ float m_sh[kRowWarps][kRows], l_sh[kRowWarps][kRows];

    const BatchArgs &a = p.a;
    const int G = a.Hq / a.Hkv;
    const int b = blockIdx.z / a.Hkv, g = blockIdx.z % a.Hkv, split = blockIdx.y;
    const int m0 = blockIdx.x * kRows;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = lane >> 2, t = lane & 3;
    if (lane == 0) {
        for (int s = 0; s < kRowStages; ++s) mbar_init(&full[warp][s], 1);
        fence_barrier_init();
    }
    __syncwarp();
    pdl_wait_predecessor();
    Request r;
    if (!load_request_kv8(p, b, r)) return;
    const int rows_total = r.n * G;
    if (m0 >= rows_total) return;
    const int pages = request_pages(r), pages8 = r.P / 16;
    const int Sb = unit_splits(pages, p.C, p.S);
    if (split >= Sb) return;
    const int t0 = (int)((long long)pages * split / Sb), t1 = (int)((long long)pages * (split + 1) / Sb);
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dsmem) + 1023) & ~uintptr_t(1023));
    uint8_t *ring = smem + warp * L::kWarp;

    // this warp's 8-bit pages: t0 + warp, then every kRowWarps-th
    const int e8 = min(t1, pages8), f8 = t0 + warp;
    const int count = e8 > f8 ? (e8 - f8 + kRowWarps - 1) / kRowWarps : 0;
    const int oob = (int)((long long)p.c.num_pages * a.Hkv * 16);          // a row past the codes: reads zeros
    // lane l holds the row coordinate and scales of the warp's page 32 grp + l;
    // `page` is the table's entry, looked up beforehand
    auto look_up = [&](int grp) -> int {
        const int i = grp * 32 + lane;
        const long long pi = (long long)b * p.c.max_pages_per_req + f8 + i * kRowWarps;
        return i < count && JSV_IN_BOUNDS(pi, (long long)a.B * p.c.max_pages_per_req, a.dev_status)
                   ? __ldg(p.c.page_table + pi) : -1;
    };
    auto load_group = [&](int grp, int page, int &row, float &ks, float &vs) {
        row = oob;
        ks = vs = 0.f;
        if (grp * 32 + lane < count) {
            if (page >= 0 && page < p.c.num_pages) {
                const size_t block = (size_t)page * a.Hkv + g;
                row = (int)block * 16;
                ks = __ldg(p.c.k_scale + block);
                vs = __ldg(p.c.v_scale + block);
            } else {
                flag_error(a.dev_status, JSV_ERR_DEVICE_INPUT);
            }
        }
    };
    // What depends on nothing but the request goes out together, before the
    // first wait for any of it: page numbers, Q, parents, the first bf16 page.
    const bool has_tail = t1 > pages8;
    const int first_tail = max(t0, pages8);
    const int tail0 = first_tail + ((warp - (first_tail - t0)) % kRowWarps + kRowWarps) % kRowWarps;
    auto tail_page = [&](int lp) -> int {
        const long long pi = (long long)b * a.max_pages_per_req + lp;
        return lp < t1 && JSV_IN_BOUNDS(pi, (long long)a.B * a.max_pages_per_req, a.dev_status)
                   ? __ldg(a.page_table + pi) : -1;
    };
    const int page_c = look_up(0);
    int page_n = look_up(1);
    int tail_next = has_tail ? tail_page(tail0) : -1;
    constexpr int kParents = kMaxTreeNodes / (kRowWarps * 32);
    int par[kParents];
#pragma unroll
    for (int k = 0; k < kParents; ++k) {
        const int i = threadIdx.x + k * (kRowWarps * 32);
        par[k] = has_tail && i < r.n && JSV_IN_BOUNDS(r.base + i, a.total_nodes, a.dev_status)
                     ? __ldg(a.parent + r.base + i) : -1;
    }
    // Q row n of each row tile, dims t*D/4 .., as bf16 pairs: words 2s, 2s+1
    // are k-step s.  Rows past the request are zero.
    uint32_t qb[NT][kSteps][2];
    auto load_q = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int rg = m0 + nt * 8 + n;
            const size_t qi = ((size_t)(r.base + rg / G) * a.Hq + g * G + rg % G) * D + t * (D / 4);
            const bool in = rg < rows_total && JSV_IN_BOUNDS(qi + D / 4 - 1, (long long)a.total_nodes * a.Hq * D,
                                                             a.dev_status);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint4 w = make_uint4(0, 0, 0, 0);
                if (in) w = __ldg(reinterpret_cast<const uint4 *>(p.q + qi) + c);
                qb[nt][2 * c][0] = w.x;
                qb[nt][2 * c][1] = w.y;
                qb[nt][2 * c + 1][0] = w.z;
                qb[nt][2 * c + 1][1] = w.w;
            }
        }
    };
    load_q();

    int row_c, row_n;
    float ks_c, vs_c, ks_n, vs_n;
    load_group(0, page_c, row_c, ks_c, vs_c);
    load_group(1, page_n, row_n, ks_n, vs_n);
    page_n = look_up(2);
    auto issue = [&](int i, int group) {             // page i of the warp, `group` the one in row_c
        const int row = __shfl_sync(0xffffffffu, (i >> 5) == group ? row_c : row_n, i & 31);
        if (lane == 0) {
            const int s = i % kRowStages;
            uint8_t *dst = ring + s * 2 * L::kBlock;
            mbar_arrive_expect_tx(&full[warp][s], 2 * L::kBlock);
            tma_load_2d(dst, &tmK, &full[warp][s], 0, row);
            tma_load_2d(dst + L::kBlock, &tmV, &full[warp][s], 0, row);
        }
    };
    for (int i = 0; i < min(count, kRowStages); ++i) issue(i, 0);

    // ancestors of the rows, where this CTA holds any of the tree's pages
    if (has_tail) {
#pragma unroll
        for (int k = 0; k < kParents; ++k) par_sh[threadIdx.x + k * (kRowWarps * 32)] = par[k];
        __syncthreads();
        if (threadIdx.x < kRows) {
            const int row = threadIdx.x, rg = m0 + row;
            for (int w = 0; w < kTreeWords; ++w) anc[row][w] = 0;
            if (rg < rows_total) {
                int j = rg / G;
                while (j != -1) {
                    anc[row][j >> 5] |= 1u << (j & 31);
                    const int pj = par_sh[j];
                    if (j == 0 ? pj != -1 : (pj < 0 || pj >= j)) {
                        flag_error(a.dev_status, JSV_ERR_DEVICE_INPUT);
                        break;
                    }
                    j = pj;
                }
            }
        }
        __syncthreads();
    }

    float fac[NT][2];                            // rows 2t, 2t + 1: score to log2 units, before the K scale
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        // the row's largest magnitude to [2^13, 2^14)
        uint32_t mx = 0;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) mx = __vmaxu2(mx, __vmaxu2(qb[nt][s][0] & 0x7fff7fffu, qb[nt][s][1] & 0x7fff7fffu));
        mx = max(mx & 0xffffu, mx >> 16);
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int ex = min(max((int)(mx >> 7), 14), 254);    // biased exponent (255: not finite, stays so)
        const float up = __uint_as_float((uint32_t)(267 - ex) << 23);
        const float down = p.scale_log2 * __uint_as_float((uint32_t)(ex - 13) << 23);
        fac[nt][0] = __shfl_sync(0xffffffffu, down, 8 * t);
        fac[nt][1] = __shfl_sync(0xffffffffu, down, 8 * t + 4);
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t w = qb[nt][s][k];
                qb[nt][s][k] = pack_f16(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up);
            }
    }

    // o[nt][i][c + 2 d]: row 2t + c, dim n*D/8 + 2i + d
    float o[NT][kTiles][4], m[NT][2], l[NT][2];
    float vmul = 0.f, vtop = 0.f;                // 2^6 / vref (0: none yet), the largest reference so far
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[nt][i][k] = 0.f;
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
    }
    auto scale_o = [&](int nt, int c, float f) {
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
            o[nt][i][c] *= f;
            o[nt][i][c + 2] *= f;
        }
    };
    // Scores in log2 units (sc[nt][c + 2 h]: row 2t + c, key n + 8 h; -inf: not
    // seen) to weights, with the running maximum and sum.
    auto softmax = [&](float (&sc)[NT][4]) {
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) grow |= fmaxf(sc[nt][c], sc[nt][c + 2]) > m[nt][c] + kMaxSlack;
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float mx = fmaxf(sc[nt][c], sc[nt][c + 2]);
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                    if (mx > m[nt][c] + kMaxSlack) {
                        const float corr = fast_exp2(m[nt][c] - mx);         // 0 from -inf
                        scale_o(nt, c, corr);
                        l[nt][c] *= corr;
                        m[nt][c] = mx;
                    }
                }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float base = m[nt][c] == -INFINITY ? 0.f : m[nt][c];
                sc[nt][c] = fast_exp2(sc[nt][c] - base);
                sc[nt][c + 2] = fast_exp2(sc[nt][c + 2] - base);
                l[nt][c] += sc[nt][c] + sc[nt][c + 2];
            }
    };
    // The reference scale follows a page's (or, for bf16 values, 1), but stays
    // within kScaleRange of the largest, so that the accumulator stays in fp32.
    auto take_scale = [&](float vs) -> float {
        const float w = fabsf(vs) * vmul;            // 2^6 vs / vref
        if ((w < 1.f || w > 2.f * kWeightShift) && fabsf(vs) > kMinScale) {
            vtop = fmaxf(vtop, fabsf(vs));
            const float inv = fast_rcp(fmaxf(fmaxf(fabsf(vs), 1.0e-36f), vtop * kScaleRange));
            const float f = vmul == 0.f ? 0.f : kWeightShift * inv * fast_rcp(vmul);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                scale_o(nt, 0, f);
                scale_o(nt, 1, f);
            }
            vmul = kWeightShift * inv;
        }
        return vs * vmul;
    };

    ks_c = finite_or_nan(ks_c);                  // here and not where it is loaded, which would wait for it
    bool ok = true;
    volatile int never = 0;
    for (int i = 0; i < count; ++i) {
        const int grp = i >> 5;
        if ((i & 31) == 0 && i > 0) {
            row_c = row_n;
            ks_c = finite_or_nan(ks_n);
            vs_c = vs_n;
            load_group(grp + 1, page_n, row_n, ks_n, vs_n);
            page_n = look_up(grp + 2);
        }
        const float ks = __shfl_sync(0xffffffffu, ks_c, i & 31), vs = __shfl_sync(0xffffffffu, vs_c, i & 31);
        const int st = i % kRowStages;
        ok = mbar_wait(&full[warp][st], (i / kRowStages) & 1, &never);
        if (__any_sync(0xffffffffu, !ok)) {
            ok = false;
            break;
        }
        const uint8_t *sk = ring + st * 2 * L::kBlock, *sv = sk + L::kBlock;

        float sc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) sc[nt][k] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
            uint32_t kw[2][4];                   // keys n, n + 8
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int at = D == 128 ? (8 * j + n) * 128 + (((2 * t + c) ^ n) << 4)
                                        : (8 * j + n) * 64 + ((t ^ (n >> 1)) << 4);
                const uint4 w = *reinterpret_cast<const uint4 *>(sk + at);
                kw[j][0] = w.x, kw[j][1] = w.y, kw[j][2] = w.z, kw[j][3] = w.w;
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                uint32_t ka[4];
                codes_to_f16<FMT>(kw[0][s], ka[0], ka[2]);
                codes_to_f16<FMT>(kw[1][s], ka[1], ka[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16(sc[nt], ka, qb[nt][4 * c + s][0], qb[nt][4 * c + s][1]);
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) sc[nt][k] *= fac[nt][k & 1] * ks;
        softmax(sc);
        const float pv = take_scale(vs);
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                pb[nt][h] = transpose_8x8(pack_f16(sc[nt][2 * h] * pv, sc[nt][2 * h + 1] * pv));
        uint32_t vw[4][D / 32];                  // keys 2t, 2t+1, 2t+8, 2t+9
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int key = 2 * t + (k & 1) + (k & 2) * 4;
            if constexpr (D == 128) {
                const uint4 w = *reinterpret_cast<const uint4 *>(sv + key * 128 + ((n ^ (key & 7)) << 4));
                vw[k][0] = w.x, vw[k][1] = w.y, vw[k][2] = w.z, vw[k][3] = w.w;
            } else {
                const uint2 w = *reinterpret_cast<const uint2 *>(sv + key * 64 + (((n >> 1) ^ ((key >> 1) & 3)) << 4) +
                                                                 (n & 1) * 8);
                vw[k][0] = w.x, vw[k][1] = w.y;
            }
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                // dims 4c + 2 half and the next, of keys (2t, 2t+1) and (2t+8, 2t+9)
                const uint32_t sel = half ? 0x7362 : 0x5140;
                uint32_t va[4];
                codes_to_f16<FMT>(__byte_perm(vw[0][c], vw[1][c], sel), va[0], va[1]);
                codes_to_f16<FMT>(__byte_perm(vw[2][c], vw[3][c], sel), va[2], va[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16(o[nt][2 * c + half], va, pb[nt][0], pb[nt][1]);
            }
        __syncwarp();
        if (i + kRowStages < count) issue(i + kRowStages, grp);
    }
    if (!ok && lane == 0) {
        flag_error(a.dev_status, JSV_ERR_TIMEOUT);
        // copies in flight land in this CTA's shared memory: wait for them, within the limit
        for (int s = 0; s < kRowStages; ++s) mbar_wait(&full[warp][s], 0, &never), mbar_wait(&full[warp][s], 1, &never);
    }

    // The bf16 pages: the rest of the prefix (seen by all) and the tree's
    // slots (seen by their descendants and themselves), on bf16 operands.
    if (ok && has_tail) {
        load_q();
        for (int lp = tail0; lp < t1; lp += kRowWarps) {
            const int page = tail_next;
            tail_next = tail_page(lp + kRowWarps);
            if (page < 0 || page >= a.num_pages) {
                if (lane == 0) flag_error(a.dev_status, JSV_ERR_DEVICE_INPUT);
                continue;
            }
            const size_t row0 = (size_t)page * 16 * a.Hkv + g;       // row of slot 0, in heads
            const long long elems = (long long)a.num_pages * 16 * a.Hkv * D;
            const int slots = min(16, r.P + r.n - lp * 16);          // slots that hold anything
            float sc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 4; ++k) sc[nt][k] = 0.f;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint4 kw[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const size_t ki = (row0 + (size_t)(8 * j + n) * a.Hkv) * D + t * (D / 4);
                    kw[j] = make_uint4(0, 0, 0, 0);
                    if (8 * j + n < slots && JSV_IN_BOUNDS(ki + c * 8 + 7, elems, a.dev_status))
                        kw[j] = *(reinterpret_cast<const uint4 *>(p.k + ki) + c);
                }
                const uint32_t k0[4] = {kw[0].x, kw[1].x, kw[0].y, kw[1].y}, k1[4] = {kw[0].z, kw[1].z, kw[0].w, kw[1].w};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_bf16(sc[nt], k0, qb[nt][2 * c][0], qb[nt][2 * c][1]);
                    mma_bf16(sc[nt], k1, qb[nt][2 * c + 1][0], qb[nt][2 * c + 1][1]);
                }
            }
            uint32_t vw[4][D / 16], key_bad = 0;                     // bit k: key k of the page is not finite
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int key = 2 * t + (k & 1) + (k & 2) * 4;
                const size_t vi = (row0 + (size_t)key * a.Hkv) * D + n * (D / 8);
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (key < slots && JSV_IN_BOUNDS(vi + c * 8 + 7, elems, a.dev_status))
                        w = *(reinterpret_cast<const uint4 *>(p.v + vi) + c);
                    vw[k][4 * c] = w.x, vw[k][4 * c + 1] = w.y, vw[k][4 * c + 2] = w.z, vw[k][4 * c + 3] = w.w;
                }
                uint32_t top = 0;
#pragma unroll
                for (int c = 0; c < D / 16; ++c) top = __vmaxu2(top, vw[k][c] & 0x7fff7fffu);
                if (max(top & 0xffffu, top >> 16) >= 0x7f80u) key_bad |= 1u << key;
            }
            // a weight of zero does not undo an infinity or NaN in the product:
            // such a key's values are taken out, and a row that sees it gets
            // NaN through its sum
            key_bad = __reduce_or_sync(0xffffffffu, key_bad);
            if (key_bad) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if ((key_bad >> (2 * t + (k & 1) + (k & 2) * 4)) & 1)
#pragma unroll
                        for (int c = 0; c < D / 16; ++c) vw[k][c] = 0;
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int row = nt * 8 + 2 * t + (k & 1), key = n + (k & 2) * 4, node = lp * 16 + key - r.P;
                    const bool seen = key < slots && (node < 0 || ((anc[row][node >> 5] >> (node & 31)) & 1u));
                    sc[nt][k] = seen ? sc[nt][k] * p.scale_log2 : -INFINITY;
                    if (seen && ((key_bad >> key) & 1)) l[nt][k & 1] = __uint_as_float(0x7fc00000u);
                }
            softmax(sc);
            const float pv = take_scale(1.f);
            uint32_t pb[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    pb[nt][h] = transpose_8x8(pack_bf16x2(sc[nt][2 * h] * pv, sc[nt][2 * h + 1] * pv));
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                const uint32_t va[4] = {__byte_perm(vw[0][c], vw[1][c], 0x5410), __byte_perm(vw[0][c], vw[1][c], 0x7632),
                                        __byte_perm(vw[2][c], vw[3][c], 0x5410), __byte_perm(vw[2][c], vw[3][c], 0x7632)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_bf16(o[nt][c], va, pb[nt][0], pb[nt][1]);
            }
        }
    }

    // This warp's rows, in fp32, without the reference scale and divided by their
    // own sum (averages of V: a sum of large values might not be finite), over
    // its ring
    float *mine = reinterpret_cast<float *>(ring);
    __syncwarp();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int row = nt * 8 + 2 * t + c;
            float sum = l[nt][c];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            const float undo = vmul == 0.f ? 0.f : fast_rcp(vmul) * (sum == 0.f ? 1.f : fast_rcp(sum));
            if (n == 0) {
                m_sh[warp][row] = ok ? m[nt][c] : -INFINITY;
                l_sh[warp][row] = ok ? sum : 0.f;
            }
#pragma unroll
            for (int i = 0; i < kTiles; i += 2)
                *reinterpret_cast<float4 *>(mine + row * D + n * (D / 8) + 2 * i) =
                    make_float4(o[nt][i][c] * undo, o[nt][i][c + 2] * undo, o[nt][i + 1][c] * undo, o[nt][i + 1][c + 2] * undo);
        }
    __syncthreads();
    const size_t rows = (size_t)a.total_nodes * a.Hq;
    for (int e = threadIdx.x; e < kRows * (D / 4); e += kRowWarps * 32) {
        const int row = e / (D / 4), c = e % (D / 4), rg = m0 + row;
        if (rg >= rows_total) break;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) M = fmaxf(M, m_sh[w][row]);
        float wt[kRowWarps], lsum = 0.f;
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) {
            const float mw = m_sh[w][row], lw = l_sh[w][row];
            // -inf: saw nothing, or NaN in what it saw
            wt[w] = lw == 0.f ? 0.f : mw == -INFINITY ? lw : fast_exp2(mw - M) * lw;
            lsum += wt[w];
        }
        // no weight at all (every score -inf): NaN, but a split's row leaves that
        // to the others
        const float inv = lsum == 0.f && Sb > 1 ? 0.f : fast_rcp(lsum);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) {
            const float f = wt[w] * inv;
            const float4 v = *reinterpret_cast<const float4 *>(smem + w * L::kWarp + (row * D + 4 * c) * 4);
            acc.x = fmaf(f, v.x, acc.x), acc.y = fmaf(f, v.y, acc.y);
            acc.z = fmaf(f, v.z, acc.z), acc.w = fmaf(f, v.w, acc.w);
        }
        const size_t row_id = (size_t)(r.base + rg / G) * a.Hq + g * G + rg % G;
        if (Sb == 1) {
            const size_t oi = row_id * D + 4 * c;
            if (JSV_IN_BOUNDS(oi + 3, (long long)rows * D, a.dev_status))
                *reinterpret_cast<uint2 *>(p.out + oi) = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
        } else {
            const size_t part = (size_t)split * rows + row_id;
            if (JSV_IN_BOUNDS(part, (long long)p.S * rows, a.dev_status)) {
                *reinterpret_cast<float4 *>(p.ws_o + part * D + 4 * c) = acc;
                if (c == 0) *reinterpret_cast<float2 *>(p.ws_ml + part * 2) = make_float2(M, lsum);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Merge of the splits' partial rows: one warp per (node, head)
// ---------------------------------------------------------------------------
constexpr int kMergeWarps = 4;

template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32, 8)
kv8_merge_kernel(const Kv8Params p) {
    pdl_allow_dependents();
    pdl_wait_predecessor();
    const BatchArgs &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.z / a.Hkv, g = blockIdx.z % a.Hkv, G = a.Hq / a.Hkv;
    const int rg = blockIdx.x * kMergeWarps + warp;
    Request r;
    if (!load_request_kv8(p, b, r) || rg >= r.n * G) return;
    const int S = unit_splits(request_units(p, r), p.C, p.S);
    if (S == 1) return;                          // written by the attention kernel
    const size_t rows = (size_t)a.total_nodes * a.Hq;
    const size_t row_id = (size_t)(r.base + rg / G) * a.Hq + g * G + rg % G;
    if (!JSV_IN_BOUNDS(row_id, rows, a.dev_status) || !JSV_IN_BOUNDS(S - 1, p.S, a.dev_status)) return;
    // lane s holds splits s and s + 32
    float ms[2], ls[2], M = -INFINITY;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int s = lane + 32 * k;
        ms[k] = -INFINITY;
        ls[k] = 0.f;
        if (s < S) {
            const float2 ml = *reinterpret_cast<const float2 *>(p.ws_ml + ((size_t)s * rows + row_id) * 2);
            ms[k] = ml.x;
            ls[k] = ml.y;
        }
        M = fmaxf(M, ms[k]);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float f[2], lsum = 0.f;                      // weights of the splits' rows
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        f[k] = ls[k] == 0.f ? 0.f : ms[k] == -INFINITY ? ls[k] : fast_exp2(ms[k] - M) * ls[k];
        lsum += f[k];
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, off);
    const float inv = 1.f / lsum;                // no weight at all: 0 * inf, NaN
#pragma unroll
    for (int k = 0; k < 2; ++k) f[k] *= inv;
    constexpr int kPer = D / 32;
    float o[kPer] = {};
    // eight splits' loads in flight at a time: no branch on a weight between
    // them (every split of the request has written its row); one after the
    // other, 37 splits took 15 us.  A weight that has underflowed to zero still
    // multiplies its row, so that an infinity or NaN in it is not lost
    const float *po = p.ws_o + row_id * D + lane * kPer;
    for (int s0 = 0; s0 < S; s0 += 8) {
        float v[8][kPer];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int x = 0; x < kPer; ++x) v[i][x] = 0.f;
            if (s0 + i < S) {
                const float *at = po + (size_t)(s0 + i) * rows * D;
                if constexpr (kPer == 4) {
                    const float4 w = *reinterpret_cast<const float4 *>(at);
                    v[i][0] = w.x, v[i][1] = w.y, v[i][2] = w.z, v[i][3] = w.w;
                } else {
                    const float2 w = *reinterpret_cast<const float2 *>(at);
                    v[i][0] = w.x, v[i][1] = w.y;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int s = s0 + i;
            const float w = __shfl_sync(0xffffffffu, s < 32 ? f[0] : f[1], s & 31);
#pragma unroll
            for (int x = 0; x < kPer; ++x) o[x] = fmaf(w, v[i][x], o[x]);
        }
    }
    uint32_t *out = reinterpret_cast<uint32_t *>(p.out + row_id * D + lane * kPer);
#pragma unroll
    for (int x = 0; x < kPer; x += 2) out[x / 2] = pack_bf16x2(o[x], o[x + 1]);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
namespace {

// The page-streaming form costs by (page, KV head, 8 rows), the tcgen05 form by
// (tile, KV head, 256 rows) and a fixed 15 us or so.  Up to 32 rows of a KV
// head the first is taken whatever the length (32 heads over 8 KV heads, us,
// streaming against tcgen05: 8 nodes over 32768 tokens 38 / 47, 16 requests of
// 8 nodes over 4096 67 / 81), above that while there are few such units (16
// nodes over 2048, 8,300 units: 17 / 21; 12 over 8192, 25,000: 25 / 28; 4 x 32
// over 1024, 34,000: 29 / 23; 32 over 8192, 66,000: 38 / 30).
constexpr int kStreamRows = 32;
constexpr double kStreamUnits = 28000.0;
// A warp takes 16 rows of a page together once there are enough units to go
// round (16 requests of 4 nodes over 4096 tokens, 66,000 units: 40 us against 48
// with 8 rows), 8 otherwise: twice the warps, and half the code to fetch, which
// is what a short call waits for (16 nodes over 128 tokens 8.2 us against 10.5;
// 12 over 2048, 6,200 units: 14 against 18).
constexpr double kWideUnits = 16000.0;

struct Kv8Plan {
    int nt;                                      // 8-row tiles of a warp, 0: the tcgen05 form
    int S, C;
};

// Splits of the largest request that minimise waves * (fixed + its share of
// the units) + what a split's partial costs, in units' times.  `load`: how
// much of B requests of the largest size the batch can hold (shorter requests
// take fewer splits, the last of them not whole).
void choose_splits(Kv8Plan &pl, long long ctas, double load, int total, int most, int slots, int per_unit,
                   double fixed, double merge, double per_split) {
    double best = 1e300;
    pl.S = 1;
    for (int s = 1; s <= kMaxSplits && s <= most; ++s) {
        const double n = (double)ctas * (load < 1.0 ? std::min(s * load + 0.5, (double)s) : s);
        const long long waves = (long long)((n + slots - 1) / slots);
        const double cost = (double)std::max(waves, 1ll) * (fixed + (double)((total + s * per_unit - 1) / (s * per_unit))) +
                            (s > 1 ? merge + per_split * s : 0.0);
        if (cost < best - 1e-9) best = cost, pl.S = s;
    }
    pl.C = (total + pl.S - 1) / pl.S;
}

// From the host-side fields: the largest request's bounds, and the pages that
// there are for all of them.  So the splits fit a batch only as well as these
// do.  A pool with pages to spare hides that a batch is ragged (one token of 16
// requests over 512 to 8192 tokens: 36 us with a pool that it fills, 51 with one
// four times as large; a ragged batch of trees 209 and 234; requests of one
// length as before), and a max_prefix far above the prefixes makes the splits
// long (four times: 64 us and 262 us for those two, 83 against 38 for 8 nodes
// over 32768 tokens).
Kv8Plan plan_of(const BatchArgs &a, const jsv_kv8 &c) {
    Kv8Plan pl;
    const int rows = a.max_nodes * (a.Hq / a.Hkv);
    const int sms = std::max(device_sm_count(), 1);
    const double load = std::min(1.0, ((double)c.num_pages + a.B) / ((double)a.B * (a.max_prefix / 16 + 1)));
    const double units = load * a.B * a.Hkv * ((a.max_prefix + (double)a.max_nodes + 15) / 16) * ((rows + 7) / 8);
    if (rows <= kStreamRows || units <= kStreamUnits) {
        pl.nt = rows <= 8 || units <= kWideUnits ? 1 : 2;
        const int tiles = (rows + 8 * pl.nt - 1) / (8 * pl.nt);
        const int total = (int)(((long long)a.max_prefix + a.max_nodes + 15) / 16);
        // a warp takes about 0.4 us (8 rows) to 0.6 us (16) for a page
        choose_splits(pl, (long long)a.B * a.Hkv * tiles, load, total, std::max(total / kRowWarps, 1),
                      sms * (pl.nt == 1 ? 4 : 3), kRowWarps, 8.0, 4.0, 0.05);
    } else {
        pl.nt = 0;
        const int tiles = (rows + 255) / 256;
        const int total = (int)(((long long)a.max_prefix / 16 + 7) / 8) + 2 * ((15 + a.max_nodes + 127) / 128);
        // a tile takes about 2.3 us, 1.7 us where the groups share out the
        // tiles; a split's fp32 partial is written and read at about 6 TB/s
        const double tile_us = rows <= 128 ? 1.7 : 2.3;
        const double per_split = (double)a.total_nodes * a.Hq * (a.D + 2) * 8.0 / 6.0e6 / tile_us;
        choose_splits(pl, (long long)a.B * a.Hkv * tiles, load, total, total, sms, 1, 9.0 / tile_us, 4.0 / tile_us,
                      per_split);
    }
    return pl;
}

template <int D, int FMT, int NT>
cudaError_t launch_rows(const Kv8Params &p, cudaStream_t st) {
    using L = RowSmem<D, NT>;
    CUtensorMap tmK, tmV;
    const uint64_t rows = (uint64_t)p.c.num_pages * p.a.Hkv * 16;
    if (!encode_tensor_map_u8_2d(&tmK, p.c.k, D, rows, 16) || !encode_tensor_map_u8_2d(&tmV, p.c.v, D, rows, 16))
        return cudaErrorInvalidValue;
    auto kernel = kv8_rows_kernel<D, FMT, NT>;
    static PerDeviceOnce once;
    cudaError_t e = once.run([&]() {
        cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kTotal);
        if (r == cudaSuccess)
            r = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     (int)cudaSharedmemCarveoutMaxShared);
        return r;
    });
    if (e != cudaSuccess) return e;
    const int G = p.a.Hq / p.a.Hkv;
    dim3 grid((p.a.max_nodes * G + 8 * NT - 1) / (8 * NT), p.S, p.a.B * p.a.Hkv);
    e = launch_pdl(kernel, grid, dim3(kRowWarps * 32), L::kTotal, st, tmK, tmV, p);
    count_launches(1);
    return e;
}

template <int D, int FMT>
cudaError_t launch_rows(const Kv8Params &p, int nt, cudaStream_t st) {
    return nt == 1 ? launch_rows<D, FMT, 1>(p, st) : launch_rows<D, FMT, 2>(p, st);
}

template <int D>
cudaError_t launch_kv8(const Kv8Params &p, int nt, cudaStream_t st) {
    cudaError_t e;
    if (nt == 0)
        e = launch_kv8_tiles(p, st);
    else
        e = p.c.format == JSV_KV8_E4M3 ? launch_rows<D, JSV_KV8_E4M3>(p, nt, st) : launch_rows<D, JSV_KV8_INT8>(p, nt, st);
    if (e != cudaSuccess || p.S == 1) return e;
    static PerDeviceOnce once;
    e = prefer_max_shared(kv8_merge_kernel<D>, once);
    if (e != cudaSuccess) return e;
    const int G = p.a.Hq / p.a.Hkv;
    e = launch_pdl(kv8_merge_kernel<D>, dim3((p.a.max_nodes * G + kMergeWarps - 1) / kMergeWarps, 1, p.a.B * p.a.Hkv),
                   dim3(kMergeWarps * 32), 0, st, p);
    count_launches(1);
    return e;
}

}  // namespace

jsv_kv8_plan attention_kv8_plan(const BatchArgs &a, const jsv_kv8 &c) {
    const Kv8Plan pl = plan_of(a, c);
    return {pl.nt ? 8 * pl.nt : 256, pl.S, pl.C};
}

size_t attention_kv8_workspace_bytes(const BatchArgs &a, const jsv_kv8 &c) {
    const Kv8Plan pl = plan_of(a, c);
    return pl.S > 1 ? (size_t)pl.S * a.total_nodes * a.Hq * ((size_t)a.D + 2) * sizeof(float) : 0;
}

cudaError_t launch_tree_attention_kv8(const BatchArgs &a, const jsv_kv8 &c, const uint16_t *q,
                                      const uint16_t *k_cache, const uint16_t *v_cache, float scale, uint16_t *out,
                                      void *ws, cudaStream_t st) {
    const Kv8Plan pl = plan_of(a, c);
    Kv8Params p;
    p.a = a;
    p.c = c;
    p.q = q;
    p.k = k_cache;
    p.v = v_cache;
    p.out = out;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.S = pl.S;
    p.C = pl.C;
    p.by_tiles = pl.nt == 0;
    p.ws_o = pl.S > 1 ? static_cast<float *>(ws) : nullptr;
    p.ws_ml = pl.S > 1 ? p.ws_o + (size_t)pl.S * a.total_nodes * a.Hq * a.D : nullptr;
    return a.D == 128 ? launch_kv8<128>(p, pl.nt, st) : launch_kv8<64>(p, pl.nt, st);
}

}  // namespace jsv
