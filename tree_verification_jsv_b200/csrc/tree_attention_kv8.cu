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
// reference scale vref: a weight is stored as 2^6 e_j vs / vref.  With
// e_j <= 2^8 and vs <= 2 vref it stays below 2^15, inside fp16; the
// accumulator is rescaled when a page's scale passes 2 vref.  The running
// maximum m moves only when a score passes it by 8 (2^8), so most pages need
// no reduction over the row.
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
// takes (request, KV head, 16*MT packed query rows, split); its warps take the
// split's pages in turn.  One lane keeps kRowStages pages of K and V in flight
// into the warp's own ring (one swizzled 16 x D box each, so that the operand
// reads below have no bank conflicts), and no warp waits for another before
// the merge at the end.
//
// Register operands of mma.m16n8k16 straight from the codes, lane = 4 n + t:
//   S = Q K^T   column n of tile j is key 8j + n; lane t supplies the dims
//               t*D/4 .. of that key, four to a k-step, and of Q alike
//   O += P V    the accumulator layout of S is the A operand layout of P;
//               lane (t, n) reads keys 2t, 2t+1, 2t+8, 2t+9 at dims n*D/8 ..,
//               pairs the keys' bytes, and tile i is dim n*D/8 + i for
//               column n, which leaves each lane D/4 neighbouring dims of O
constexpr int kRowWarps = 4;
constexpr int kRowStages = 4;

template <int D, int MT>
struct RowSmem {
    static constexpr int kBlock = 16 * D;                        // codes of one page and head
    static constexpr int kRing = kRowStages * 2 * kBlock;        // a warp's
    static constexpr int kMerge = 16 * MT * D * 4;               // a warp's, over its ring
    static constexpr int kWarp = kRing > kMerge ? kRing : kMerge;
    static constexpr int kTotal = kRowWarps * kWarp + 1024;
};

template <int D, int FMT, int MT>
__global__ void __launch_bounds__(kRowWarps * 32)
kv8_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Kv8Params p) {
    pdl_allow_dependents();
    using L = RowSmem<D, MT>;
    constexpr int kRows = 16 * MT;
    constexpr int kSteps = D / 16;               // k-steps of a score
    constexpr int kTiles = D / 8;                // column tiles of the output
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
    // lane l holds the row coordinate and scales of the warp's page 32 grp + l
    auto load_group = [&](int grp, int &row, float &ks, float &vs) {
        const int i = grp * 32 + lane;
        row = oob;
        ks = vs = 0.f;
        if (i < count) {
            const long long pi = (long long)b * p.c.max_pages_per_req + f8 + i * kRowWarps;
            int page = -1;
            if (JSV_IN_BOUNDS(pi, (long long)a.B * p.c.max_pages_per_req, a.dev_status)) page = __ldg(p.c.page_table + pi);
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
    int row_c, row_n;
    float ks_c, vs_c, ks_n, vs_n;
    load_group(0, row_c, ks_c, vs_c);
    load_group(1, row_n, ks_n, vs_n);
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
    const bool has_tail = t1 > pages8;
    if (has_tail) {
        for (int i = threadIdx.x; i < r.n; i += kRowWarps * 32)
            par_sh[i] = JSV_IN_BOUNDS(r.base + i, a.total_nodes, a.dev_status) ? __ldg(a.parent + r.base + i) : -1;
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

    // Q rows n and n + 8 of each row tile, dims t*D/4 .., as bf16 pairs:
    // words 2s, 2s+1 are k-step s.  Rows past the request are zero.
    uint32_t qa[MT][kSteps][4];
    auto load_q = [&]() {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const int rg = m0 + mt * 16 + hh * 8 + n;
                const size_t qi = ((size_t)(r.base + rg / G) * a.Hq + g * G + rg % G) * D + t * (D / 4);
                const bool in = rg < rows_total && JSV_IN_BOUNDS(qi + D / 4 - 1, (long long)a.total_nodes * a.Hq * D,
                                                                 a.dev_status);
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (in) w = __ldg(reinterpret_cast<const uint4 *>(p.q + qi) + c);
                    qa[mt][2 * c][hh] = w.x;
                    qa[mt][2 * c][hh + 2] = w.y;
                    qa[mt][2 * c + 1][hh] = w.z;
                    qa[mt][2 * c + 1][hh + 2] = w.w;
                }
            }
    };
    float fac[MT][2];                            // score to log2 units, before the K scale
    load_q();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            // the row's largest magnitude to [2^13, 2^14)
            uint32_t mx = 0;
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
                mx = __vmaxu2(mx, __vmaxu2(qa[mt][s][hh] & 0x7fff7fffu, qa[mt][s][hh + 2] & 0x7fff7fffu));
            mx = max(mx & 0xffffu, mx >> 16);
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const int ex = max((int)(mx >> 7), 14);              // biased exponent (255: not finite, stays so)
            const float up = __uint_as_float((uint32_t)(267 - min(ex, 254)) << 23);
            fac[mt][hh] = p.scale_log2 * __uint_as_float((uint32_t)(min(ex, 254) - 13) << 23);
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int k = hh; k < 4; k += 2) {
                    const uint32_t w = qa[mt][s][k];
                    qa[mt][s][k] = pack_f16(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up);
                }
        }

    float o[MT][kTiles][4], m[MT][2], l[MT][2], vref = 0.f;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[mt][i][k] = 0.f;
        m[mt][0] = m[mt][1] = -INFINITY;
        l[mt][0] = l[mt][1] = 0.f;
    }
    auto scale_o = [&](int mt, int hh, float f) {
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
            o[mt][i][2 * hh] *= f;
            o[mt][i][2 * hh + 1] *= f;
        }
    };
    // Scores in log2 units (sc[mt][j][2 hh + c]: row n + 8 hh, key 8 j + 2 t + c;
    // -inf: not seen) to weights, with the running maximum and sum.
    auto softmax = [&](float (&sc)[MT][2][4]) {
        bool grow = false;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const float mx = fmaxf(fmaxf(sc[mt][0][2 * hh], sc[mt][0][2 * hh + 1]),
                                       fmaxf(sc[mt][1][2 * hh], sc[mt][1][2 * hh + 1]));
                grow |= mx > m[mt][hh] + kMaxSlack;
            }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    float mx = fmaxf(fmaxf(sc[mt][0][2 * hh], sc[mt][0][2 * hh + 1]),
                                     fmaxf(sc[mt][1][2 * hh], sc[mt][1][2 * hh + 1]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    if (mx > m[mt][hh] + kMaxSlack) {
                        const float corr = fast_exp2(m[mt][hh] - mx);        // 0 from -inf
                        scale_o(mt, hh, corr);
                        l[mt][hh] *= corr;
                        m[mt][hh] = mx;
                    }
                }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const float base = m[mt][hh] == -INFINITY ? 0.f : m[mt][hh];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = 2 * hh; k < 2 * hh + 2; ++k) {
                        sc[mt][j][k] = fast_exp2(sc[mt][j][k] - base);
                        l[mt][hh] += sc[mt][j][k];
                    }
            }
    };
    // the reference scale takes in a page's (or, for bf16 values, 1)
    auto take_scale = [&](float vs) -> float {
        if (fabsf(vs) > 2.f * vref) {
            const float f = vref / fabsf(vs);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                scale_o(mt, 0, f);
                scale_o(mt, 1, f);
            }
            vref = fabsf(vs);
        }
        return vref > 0.f ? vs / vref * kWeightShift : vs * 0.f;
    };

    bool ok = true;
    volatile int never = 0;
    for (int i = 0; i < count; ++i) {
        const int grp = i >> 5;
        if ((i & 31) == 0 && i > 0) {
            row_c = row_n;
            ks_c = ks_n;
            vs_c = vs_n;
            load_group(grp + 1, row_n, ks_n, vs_n);
        }
        const float ks = __shfl_sync(0xffffffffu, ks_c, i & 31), vs = __shfl_sync(0xffffffffu, vs_c, i & 31);
        const int st = i % kRowStages;
        ok = mbar_wait(&full[warp][st], (i / kRowStages) & 1, &never);
        if (__any_sync(0xffffffffu, !ok)) {
            ok = false;
            break;
        }
        const uint8_t *sk = ring + st * 2 * L::kBlock, *sv = sk + L::kBlock;

        float sc[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) sc[mt][j][k] = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const int at = D == 128 ? (8 * j + n) * 128 + (((2 * t + c) ^ n) << 4)
                                        : (8 * j + n) * 64 + ((t ^ (n >> 1)) << 4);
                const uint4 w = *reinterpret_cast<const uint4 *>(sk + at);
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    uint32_t b0, b1;
                    codes_to_f16<FMT>(ws[s], b0, b1);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) mma_f16(sc[mt][j], qa[mt][4 * c + s], b0, b1);
                }
            }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const float f = fac[mt][hh] * ks;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    sc[mt][j][2 * hh] *= f;
                    sc[mt][j][2 * hh + 1] *= f;
                }
            }
        softmax(sc);
        const float pv = take_scale(vs);
        uint32_t pa[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            pa[mt][0] = pack_f16(sc[mt][0][0] * pv, sc[mt][0][1] * pv);
            pa[mt][1] = pack_f16(sc[mt][0][2] * pv, sc[mt][0][3] * pv);
            pa[mt][2] = pack_f16(sc[mt][1][0] * pv, sc[mt][1][1] * pv);
            pa[mt][3] = pack_f16(sc[mt][1][2] * pv, sc[mt][1][3] * pv);
        }
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
                const uint32_t sel = half ? 0x7362 : 0x5140;
                uint32_t b0[2], b1[2];
                codes_to_f16<FMT>(__byte_perm(vw[0][c], vw[1][c], sel), b0[0], b0[1]);
                codes_to_f16<FMT>(__byte_perm(vw[2][c], vw[3][c], sel), b1[0], b1[1]);
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) mma_f16(o[mt][4 * c + 2 * half + u], pa[mt], b0[u], b1[u]);
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
    const int first_tail = max(t0, pages8);
    if (ok && has_tail) {
        load_q();
        for (int lp = first_tail + ((warp - (first_tail - t0)) % kRowWarps + kRowWarps) % kRowWarps; lp < t1;
             lp += kRowWarps) {
            const long long pi = (long long)b * a.max_pages_per_req + lp;
            const int page = JSV_IN_BOUNDS(pi, (long long)a.B * a.max_pages_per_req, a.dev_status)
                                 ? __ldg(a.page_table + pi) : -1;
            if (page < 0 || page >= a.num_pages) {
                if (lane == 0) flag_error(a.dev_status, JSV_ERR_DEVICE_INPUT);
                continue;
            }
            const size_t row0 = (size_t)page * 16 * a.Hkv + g;       // row of slot 0, in heads
            const long long elems = (long long)a.num_pages * 16 * a.Hkv * D;
            const int slots = min(16, r.P + r.n - lp * 16);          // slots that hold anything
            float sc[MT][2][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) sc[mt][j][k] = 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const size_t ki = (row0 + (size_t)(8 * j + n) * a.Hkv) * D + t * (D / 4);
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (8 * j + n < slots && JSV_IN_BOUNDS(ki + c * 8 + 7, elems, a.dev_status))
                        w = *(reinterpret_cast<const uint4 *>(p.k + ki) + c);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        mma_bf16(sc[mt][j], qa[mt][2 * c], w.x, w.y);
                        mma_bf16(sc[mt][j], qa[mt][2 * c + 1], w.z, w.w);
                    }
                }
            }
            uint32_t vw[4][D / 16], key_bad = 0;                     // bit k: key k holds a non-finite value
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
                if (max(top & 0xffffu, top >> 16) >= 0x7f80u) key_bad |= 1u << k;
            }
            // a weight of zero does not undo an infinity or NaN in the product:
            // such a key's values are taken out, and a row that sees it gets
            // NaN through its sum
            if (__any_sync(0xffffffffu, key_bad)) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) key_bad |= __shfl_xor_sync(0xffffffffu, key_bad, off);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if ((key_bad >> k) & 1)
#pragma unroll
                        for (int c = 0; c < D / 16; ++c) vw[k][c] = 0;
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const int row = mt * 16 + hh * 8 + n;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int key = 2 * t + (k & 1) + (k & 2) * 4, node = lp * 16 + key - r.P;
                        const bool seen = key < slots && (node < 0 || ((anc[row][node >> 5] >> (node & 31)) & 1u));
                        float &s = sc[mt][k >> 1][2 * hh + (k & 1)];
                        s = seen ? s * p.scale_log2 : -INFINITY;
                        if (seen && ((key_bad >> k) & 1)) l[mt][hh] = __uint_as_float(0x7fc00000u);
                    }
                }
            softmax(sc);
            const float pv = take_scale(1.f);
            uint32_t pa[MT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                pa[mt][0] = pack_bf16x2(sc[mt][0][0] * pv, sc[mt][0][1] * pv);
                pa[mt][1] = pack_bf16x2(sc[mt][0][2] * pv, sc[mt][0][3] * pv);
                pa[mt][2] = pack_bf16x2(sc[mt][1][0] * pv, sc[mt][1][1] * pv);
                pa[mt][3] = pack_bf16x2(sc[mt][1][2] * pv, sc[mt][1][3] * pv);
            }
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint32_t sel = half ? 0x7632 : 0x5410;
                    const uint32_t b0 = __byte_perm(vw[0][c], vw[1][c], sel), b1 = __byte_perm(vw[2][c], vw[3][c], sel);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) mma_bf16(o[mt][2 * c + half], pa[mt], b0, b1);
                }
            }
        }
    }

    // This warp's rows, in fp32 and without the reference scale, over its ring
    const float undo = vref / kWeightShift;
    float *mine = reinterpret_cast<float *>(ring);
    __syncwarp();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int row = mt * 16 + hh * 8 + n;
            float sum = l[mt][hh];
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            if (t == 0) {
                m_sh[warp][row] = ok ? m[mt][hh] : -INFINITY;
                l_sh[warp][row] = ok ? sum : 0.f;
            }
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < kTiles; i += 4) {
                    float4 v = make_float4(o[mt][i][2 * hh + c], o[mt][i + 1][2 * hh + c], o[mt][i + 2][2 * hh + c],
                                           o[mt][i + 3][2 * hh + c]);
                    v.x *= undo, v.y *= undo, v.z *= undo, v.w *= undo;
                    *reinterpret_cast<float4 *>(mine + row * D + (2 * t + c) * kTiles + i) = v;
                }
        }
    __syncthreads();
    const size_t rows = (size_t)a.total_nodes * a.Hq;
    for (int e = threadIdx.x; e < kRows * (D / 4); e += kRowWarps * 32) {
        const int row = e / (D / 4), c = e % (D / 4), rg = m0 + row;
        if (rg >= rows_total) break;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) M = fmaxf(M, m_sh[w][row]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float lsum = 0.f;
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) {
            const float mw = m_sh[w][row], lw = l_sh[w][row];
            if (mw == -INFINITY && lw == 0.f) continue;          // saw nothing
            const float f = mw == -INFINITY ? 1.f : fast_exp2(mw - M);
            const float4 v = *reinterpret_cast<const float4 *>(smem + w * L::kWarp + (row * D + 4 * c) * 4);
            acc.x = fmaf(f, v.x, acc.x), acc.y = fmaf(f, v.y, acc.y);
            acc.z = fmaf(f, v.z, acc.z), acc.w = fmaf(f, v.w, acc.w);
            lsum = fmaf(f, lw, lsum);
        }
        const size_t row_id = (size_t)(r.base + rg / G) * a.Hq + g * G + rg % G;
        if (Sb == 1) {
            const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
            const size_t oi = row_id * D + 4 * c;
            if (JSV_IN_BOUNDS(oi + 3, (long long)rows * D, a.dev_status))
                *reinterpret_cast<uint2 *>(p.out + oi) = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv),
                                                                    pack_bf16x2(acc.z * inv, acc.w * inv));
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
__global__ void __launch_bounds__(kMergeWarps * 32, 16)
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
    float f[2], lsum = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        f[k] = ls[k] == 0.f ? 0.f : ms[k] == -INFINITY ? 1.f : fast_exp2(ms[k] - M);
        lsum = fmaf(f[k], ls[k], lsum);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, off);
    constexpr int kPer = D / 32;
    float o[kPer] = {};
#pragma unroll 4
    for (int s = 0; s < S; ++s) {
        const float w = __shfl_sync(0xffffffffu, s < 32 ? f[0] : f[1], s & 31);
        if (w == 0.f) continue;
        const float *po = p.ws_o + ((size_t)s * rows + row_id) * D + lane * kPer;
        if constexpr (kPer == 4) {
            const float4 v = *reinterpret_cast<const float4 *>(po);
            o[0] = fmaf(w, v.x, o[0]), o[1] = fmaf(w, v.y, o[1]), o[2] = fmaf(w, v.z, o[2]), o[3] = fmaf(w, v.w, o[3]);
        } else {
            const float2 v = *reinterpret_cast<const float2 *>(po);
            o[0] = fmaf(w, v.x, o[0]), o[1] = fmaf(w, v.y, o[1]);
        }
    }
    const float inv = lsum == 0.f ? 0.f : 1.f / lsum;
    uint32_t *out = reinterpret_cast<uint32_t *>(p.out + row_id * D + lane * kPer);
#pragma unroll
    for (int x = 0; x < kPer; x += 2) out[x / 2] = pack_bf16x2(o[x] * inv, o[x + 1] * inv);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
namespace {

// Query rows of a KV head (nodes * Hq / Hkv) up to which the page-streaming
// form is taken.
constexpr int kRowsFormMost = 32;

struct Kv8Plan {
    int mt;                                      // row tiles of a warp, 0: the tcgen05 form
    int S, C;
};

// Splits that minimise waves * (fixed + units of a split) + what a split's
// partial costs, in units' times; the estimate takes every request for the
// largest the batch may hold.
void choose_splits(Kv8Plan &pl, long long units_of_work, int total, int most, int slots, int per_unit, double fixed,
                   double merge, double per_split) {
    double best = 1e300;
    pl.S = 1;
    for (int s = 1; s <= kMaxSplits && s <= most; ++s) {
        const long long waves = (units_of_work * s + slots - 1) / slots;
        const double cost = (double)waves * (fixed + (double)((total + s * per_unit - 1) / (s * per_unit))) +
                            (s > 1 ? merge + per_split * s : 0.0);
        if (cost < best - 1e-9) best = cost, pl.S = s;
    }
    pl.C = (total + pl.S - 1) / pl.S;
}

Kv8Plan plan_of(const BatchArgs &a) {
    Kv8Plan pl;
    const int rows = a.max_nodes * (a.Hq / a.Hkv);
    const int sms = std::max(device_sm_count(), 1);
    if (rows <= kRowsFormMost) {
        pl.mt = rows <= 16 ? 1 : 2;
        const int tiles = (rows + 16 * pl.mt - 1) / (16 * pl.mt);
        const int total = (int)(((long long)a.max_prefix + a.max_nodes + 15) / 16);
        choose_splits(pl, (long long)a.B * a.Hkv * tiles, total, std::max(total / kRowWarps, 1),
                      sms * (pl.mt == 1 ? 3 : 2), kRowWarps, 8.0, 4.0, 0.05);
    } else {
        pl.mt = 0;
        const int tiles = (rows + 255) / 256;
        const int total = (int)(((long long)a.max_prefix / 16 + 7) / 8) + (15 + a.max_nodes + 127) / 128;
        // a tile takes about 2.1 us; a split's fp32 partial is written and read at about 6 TB/s
        const double per_split = (double)a.total_nodes * a.Hq * (a.D + 2) * 8.0 / 6.0e6 / 2.1;
        choose_splits(pl, (long long)a.B * a.Hkv * tiles, total, total, sms, 1, 3.0, 1.0, per_split);
    }
    return pl;
}

template <int D, int FMT, int MT>
cudaError_t launch_rows(const Kv8Params &p, cudaStream_t st) {
    using L = RowSmem<D, MT>;
    CUtensorMap tmK, tmV;
    const uint64_t rows = (uint64_t)p.c.num_pages * p.a.Hkv * 16;
    if (!encode_tensor_map_u8_2d(&tmK, p.c.k, D, rows, 16) || !encode_tensor_map_u8_2d(&tmV, p.c.v, D, rows, 16))
        return cudaErrorInvalidValue;
    auto kernel = kv8_rows_kernel<D, FMT, MT>;
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
    dim3 grid((p.a.max_nodes * G + 16 * MT - 1) / (16 * MT), p.S, p.a.B * p.a.Hkv);
    e = launch_pdl(kernel, grid, dim3(kRowWarps * 32), L::kTotal, st, tmK, tmV, p);
    count_launches(1);
    return e;
}

template <int D>
cudaError_t launch_kv8(const Kv8Params &p, int mt, cudaStream_t st) {
    cudaError_t e;
    if (mt == 0)
        e = launch_kv8_tiles(p, st);
    else if (p.c.format == JSV_KV8_E4M3)
        e = mt == 1 ? launch_rows<D, JSV_KV8_E4M3, 1>(p, st) : launch_rows<D, JSV_KV8_E4M3, 2>(p, st);
    else
        e = mt == 1 ? launch_rows<D, JSV_KV8_INT8, 1>(p, st) : launch_rows<D, JSV_KV8_INT8, 2>(p, st);
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

size_t attention_kv8_workspace_bytes(const BatchArgs &a) {
    const Kv8Plan pl = plan_of(a);
    return pl.S > 1 ? (size_t)pl.S * a.total_nodes * a.Hq * ((size_t)a.D + 2) * sizeof(float) : 0;
}

cudaError_t launch_tree_attention_kv8(const BatchArgs &a, const jsv_kv8 &c, const uint16_t *q,
                                      const uint16_t *k_cache, const uint16_t *v_cache, float scale, uint16_t *out,
                                      void *ws, cudaStream_t st) {
    const Kv8Plan pl = plan_of(a);
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
    p.by_tiles = pl.mt == 0;
    p.ws_o = pl.S > 1 ? static_cast<float *>(ws) : nullptr;
    p.ws_ml = pl.S > 1 ? p.ws_o + (size_t)pl.S * a.total_nodes * a.Hq * a.D : nullptr;
    return a.D == 128 ? launch_kv8<128>(p, pl.mt, st) : launch_kv8<64>(p, pl.mt, st);
}

}  // namespace jsv
