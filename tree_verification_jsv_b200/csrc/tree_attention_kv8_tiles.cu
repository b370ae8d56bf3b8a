// Tree-causal attention over a prefix held in 8 bits: the form for many query
// rows, on tcgen05 tensor cores (the arithmetic is described at the head of
// tree_attention_kv8.cu).
//
// One CTA per (request, KV head, 256 packed query rows, split); the rows form
// two 128-row groups that take turns on the tensor core, as in
// tree_attention.cu, whose MMA order and softmax this kernel keeps.  Where a
// CTA has 128 rows or fewer, both groups take the same rows and every other
// tile each, and their results are merged at the end: one group alone would
// leave the tensor core idle during its softmax (16 requests of 16 nodes over
// 4096 tokens: 88 us with one group, 83 with two as first built and 82 now, which
// the conversion bounds).
// Also different is where the operands come from: the codes are copied a page
// at a time to shared memory and written from there to the operand tiles as
// fp16 by seven converting warps, one 128-key tile ahead, so that the tensor
// core, the softmax and the conversion run side by side.
//
// Tiles: eight 8-bit pages each (128 keys), then 128-slot tiles of the bf16
// cache from the first slot past the full pages, copied unconverted and
// multiplied as bf16: a group's warps turn their rows of Q back to bf16 when
// they hand over the last 8-bit tile's weights.
//
//   warps 0..3    V tiles: codes -> fp16, or bf16 copied
//   warp 4        TMEM, MMA issue (one thread)
//   warps 5..7    K tiles likewise, and the tiles' scales
//   warps 8..15   softmax, one query row per thread
//
// The K scale of a page multiplies its 16 score columns (it rides on the
// multiply that brings scores to log2 units).  The V scale goes into the
// fp16 V tile as vs / vref, instead of into the weights: the converting warps
// have the instructions to spare, the softmax warps do not.  vref is the CTA's
// reference scale.  It follows the tiles' largest V scales up and down, so that
// such a page's factor lies in [16, 128], from the middle of fp16's normal
// range to where 448 times it still is finite; where it changes, O is rescaled
// with the running maximum's correction.  A factor below 2^-14 is applied in
// two steps, 2^14 times as large and then by 2^-14, so that it is never
// rounded as a subnormal number.  A value is off by two roundings, 2^-10 of it,
// and, below 2^-14 in units of vref, by fp16's step there: by up to 2^-25 vref,
// which is 2^-29 of the largest V scale of its tile.
//
// A tile took about 4,300 cycles when 256 nodes over 16384 tokens took 118 us
// (timeline of one CTA): softmax about 2,400 (scores from TMEM 230, maximum 450,
// exponentials, packing and the store 1,600), then 1,400 until the group's PV
// and next S are issued and complete, and 500 waiting for the thread that issues
// them.  The tensor pipe's share is 2,048; tree_attention.cu, whose operands
// need no conversion, takes 3,600.  All warps' code of a tile competes for the
// instruction caches, so what runs rarely is kept out of the loops: a division's
// rare cases cost 6%, the last tile's mask 3-4%, unrolled conversion 13%.
// 256 nodes over 16384 tokens (int8) take 108 us (636 TFLOP/s, 39% of the
// measured bf16 rate), four 512-node trees over 32768 1,242-1,294 us (850-885,
// by the box's clock), a ragged batch of 16 209 us.  The bf16 kernel, with twice
// the bytes to read and nothing to convert, takes 83, 1,001 and 138 on the same
// box: this form is for the bytes that the cache holds, not for time.
#include "kv8_attention.cuh"

#include <type_traits>

namespace jsv {

namespace {

constexpr int kGroups = 2;
constexpr int kGroupRows = 128;
constexpr int kRowsPerCta = kGroups * kGroupRows;
constexpr int kTileKeys = 128;
constexpr int kTilePages = kTileKeys / 16;
constexpr int kStages = 2;
constexpr int kVTeam = 4;                        // converting warps of V (0..3) and of K (5..7)
constexpr int kKTeam = 3;
constexpr int kMmaWarp = 4;
constexpr int kSoftmaxWarp0 = 8;
constexpr int kTileThreads = 512;
// registers a thread after the split, of 128 at launch: 80 + 80 + 2 * 176 =
// 4 * 128 over the four warpgroups
constexpr int kRegsConv = 80;
constexpr int kRegsMma = 80;
constexpr int kRegsSoftmax = 176;
constexpr int kSlots = 4;                        // tiles whose scales are held, see TileInfo
constexpr float kWeightLog2 = 6.f;               // weights are held as 2^6 e: e <= 2^8 stays inside fp16
constexpr float kTinyRatio = 6.103515625e-05f;   // 2^-14, the smallest normal fp16 number,
constexpr uint32_t kTinyPair = 0x04000400u;      // and a pair of them

// What the softmax warps need of a tile.  Written before the tile's K is
// handed over and once its place in the ring is free: by then S of tile j - 2
// is complete, which was issued after P of tile j - 4 arrived, so the slot's
// last tile has been read.
struct __align__(16) TileInfo {
    float ks[kTilePages];                        // read as two float4
    float vref, vinv;                            // reference scale of V and its reciprocal
    // bf16 slots whose V row is not finite, as each converting warp found them
    uint32_t bad[kVTeam][kTileKeys / 32];
};

template <int D>
struct TileSmem {
    static constexpr int kQGroup = kGroupRows * D * 2;
    static constexpr int kQ = kGroups * kQGroup;
    static constexpr int kKV = kTileKeys * D * 2;              // one K (or V) tile
    static constexpr int kStage = 2 * kKV;
    static constexpr int kRaw = kTileKeys * D;                 // one tile's codes of K (or V)
    static constexpr int kTotal = kQ + kStages * kStage + 2 * kRaw + 1024;
};

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The MMA issuer, one thread; see attention_mma_loop in tree_attention.cu for
// the order and for why everything is a constant offset from a base.  Tiles
// before `n_pre` are fp16, the others bf16.  kDual: group j % 2 takes tile j,
// and S of its next tile, j + 2, follows PV of tile j; else both groups take
// every tile.
template <int D, bool kDual>
__device__ __forceinline__ void kv8_mma_loop(uint32_t tmem, uint32_t aQ, uint32_t aKV, int ntiles, int n_pre,
                                             uint64_t *k_full, uint64_t *v_full, uint64_t *k_empty, uint64_t *v_empty,
                                             uint64_t *s_full, uint64_t *p_full, uint64_t *o_done, uint64_t *q_ready,
                                             uint64_t *drain_bar, volatile int *abort_sh, int32_t *dev_status) {
    using L = TileSmem<D>;
    constexpr uint32_t kBf16 = (1u << 7) | (1u << 10);             // operand types of the descriptor: 0 = fp16
    constexpr uint32_t id_s = idesc_bf16_f32(128, kTileKeys, false, false) & ~kBf16;
    constexpr uint32_t id_o = idesc_bf16_f32(128, D, false, true) & ~kBf16;
    constexpr uint32_t kStageStep = L::kStage >> 4;
    uint64_t dQ = desc_kmajor_sw128(aQ);
    uint64_t dK0 = desc_kmajor_sw128(aKV);
    uint64_t dV0 = desc_mnmajor_sw128(aKV + L::kKV, kTileKeys * 128, 1024);
    // the operand type is a constant of each call: a descriptor formed at run
    // time between two MMAs sits on the tensor pipe's critical path (with it the
    // 16 MMAs of a group took 3,400 cycles to issue instead of about 1,100)
    auto issue_s_typed = [&](auto grp_c, auto type_c, uint64_t dk) {
        constexpr int grp = decltype(grp_c)::value;
        constexpr uint32_t type = decltype(type_c)::value;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = grp * L::kQGroup + (kk >> 2) * (kGroupRows * 128) + (kk & 3) * 32;
            const uint32_t offk = (kk >> 2) * (kTileKeys * 128) + (kk & 3) * 32;
            mma_bf16_ss(tmem + grp * 128, dQ + (off >> 4), dk + (offk >> 4), id_s | type, kk > 0);
        }
        mma_commit(&s_full[grp]);
    };
    auto issue_pv_typed = [&](auto grp_c, auto type_c, uint64_t dv, uint32_t acc_first) {
        constexpr int grp = decltype(grp_c)::value;
        constexpr uint32_t type = decltype(type_c)::value;
#pragma unroll
        for (int kk = 0; kk < kTileKeys / 16; ++kk)
            mma_bf16_ts(tmem + 256 + grp * D, tmem + grp * 128 + kk * 8, dv + ((kk * 2048) >> 4), id_o | type,
                        kk > 0 ? 1u : acc_first);
        mma_commit(&o_done[grp]);
    };
    using F16 = std::integral_constant<uint32_t, 0u>;
    using BF16 = std::integral_constant<uint32_t, kBf16>;
    auto issue_s = [&](auto grp_c, bool codes, uint64_t dk) {
        if (codes) issue_s_typed(grp_c, F16{}, dk);
        else issue_s_typed(grp_c, BF16{}, dk);
    };
    auto issue_pv = [&](auto grp_c, bool codes, uint64_t dv, uint32_t acc_first) {
        if (codes) issue_pv_typed(grp_c, F16{}, dv, acc_first);
        else issue_pv_typed(grp_c, BF16{}, dv, acc_first);
    };
    using G0 = std::integral_constant<int, 0>;
    using G1 = std::integral_constant<int, 1>;
    bool ok = mbar_wait(q_ready, 0, abort_sh);
    if (ok) ok = mbar_wait(&k_full[0], 0, abort_sh);
    if (ok) {
        tc_fence_after();
        issue_s(G0{}, n_pre > 0, dK0);
        if constexpr (!kDual) issue_s(G1{}, n_pre > 0, dK0);
        mma_commit(&k_empty[0]);
    }
    if constexpr (kDual) {
        if (ok && ntiles > 1) {
            ok = mbar_wait(&k_full[1], 0, abort_sh);
            if (ok) {
                tc_fence_after();
                issue_s(G1{}, n_pre > 1, dK0 + kStageStep);
                mma_commit(&k_empty[1]);
            }
        }
        auto turn = [&](auto grp_c, int j) -> bool {
            constexpr int grp = decltype(grp_c)::value;
            asm volatile("" : "+l"(dQ), "+l"(dK0), "+l"(dV0));
            const uint32_t ph = (uint32_t)((j / 2) & 1);
            const bool more = j + 2 < ntiles;
            if (!mbar_wait(&v_full[grp], ph, abort_sh) || (more && !mbar_wait(&k_full[grp], ph ^ 1, abort_sh)) ||
                !mbar_wait(&p_full[grp], ph, abort_sh))
                return false;
            tc_fence_after();
            issue_pv(grp_c, j < n_pre, dV0 + grp * kStageStep, j > 1 ? 1u : 0u);
            mma_commit(&v_empty[grp]);
            if (more) {
                issue_s(grp_c, j + 2 < n_pre, dK0 + grp * kStageStep);
                mma_commit(&k_empty[grp]);
            }
            return true;
        };
        for (int j = 0; ok && j < ntiles; j += 2) ok = turn(G0{}, j) && (j + 1 >= ntiles || turn(G1{}, j + 1));
    } else {
        for (int j = 0; ok && j < ntiles; ++j) {
            asm volatile("" : "+l"(dQ), "+l"(dK0), "+l"(dV0));
            const int st = j % kStages, stn = (j + 1) % kStages;
            const uint32_t ph = (uint32_t)((j / kStages) & 1), phn = (uint32_t)(((j + 1) / kStages) & 1);
            const bool more = j + 1 < ntiles;
            const uint64_t dv = dV0 + st * kStageStep, dkn = dK0 + stn * kStageStep;
            const uint32_t acc_first = j > 0 ? 1u : 0u;
            const bool codes = j < n_pre, codes_n = j + 1 < n_pre;
            ok = mbar_wait(&v_full[st], ph, abort_sh) && (!more || mbar_wait(&k_full[stn], phn, abort_sh));
            if (!ok) break;
            ok = mbar_wait(&p_full[0], j & 1, abort_sh);
            if (!ok) break;
            tc_fence_after();
            issue_pv(G0{}, codes, dv, acc_first);
            if (more) issue_s(G0{}, codes_n, dkn);
            ok = mbar_wait(&p_full[1], j & 1, abort_sh);
            if (!ok) break;
            tc_fence_after();
            issue_pv(G1{}, codes, dv, acc_first);
            mma_commit(&v_empty[st]);
            if (more) {
                issue_s(G1{}, codes_n, dkn);
                mma_commit(&k_empty[stn]);
            }
        }
    }
    if (!ok) {
        *abort_sh = 1;
        flag_error(dev_status, JSV_ERR_TIMEOUT);
    }
    int zero = 0;
    mma_commit(drain_bar);
    mbar_wait(drain_bar, 0, (volatile int *)&zero);
}

}  // namespace

template <int D, int FMT>
__global__ void __launch_bounds__(kTileThreads, 1)
kv8_tiles_kernel(const Kv8Params p) {
    pdl_allow_dependents();
    using L = TileSmem<D>;
    extern __shared__ uint8_t dsmem[];
    __shared__ __align__(8) uint64_t k_full[kStages], v_full[kStages], k_empty[kStages], v_empty[kStages];
    __shared__ __align__(8) uint64_t s_full[kGroups], p_full[kGroups], o_done[kGroups], q_ready, tree_read, drain_bar, raw_full[kVTeam + kKTeam];
    __shared__ uint32_t tmem_base_sh;
    __shared__ volatile int abort_sh;
    __shared__ TileInfo info[kSlots];
    __shared__ float row_inv[kRowsPerCta];        // what undoes the scaling of each row of Q

    const BatchArgs &a = p.a;
    const int G = a.Hq / a.Hkv;
    const int b = blockIdx.z / a.Hkv, g = blockIdx.z % a.Hkv, split = blockIdx.y;
    const int m0 = blockIdx.x * kRowsPerCta;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dsmem) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = smem, *sKV = smem + L::kQ, *raw = sKV + kStages * L::kStage;
    // the request's parents, over the second V tile until the ancestors are found
    int *par_sh = reinterpret_cast<int *>(sKV + L::kStage + L::kKV);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&k_full[s], kKTeam);
            mbar_init(&v_full[s], kVTeam);
            mbar_init(&k_empty[s], 1);
            mbar_init(&v_empty[s], 1);
        }
        for (int s = 0; s < kGroups; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&p_full[s], 4);
            mbar_init(&o_done[s], 1);
        }
        mbar_init(&q_ready, 4 * kGroups);
        mbar_init(&tree_read, 4 * kGroups);
        mbar_init(&drain_bar, 1);
        for (int w = 0; w < kVTeam + kKTeam; ++w) mbar_init(&raw_full[w], 1);
        abort_sh = 0;
        fence_barrier_init();
    }
    pdl_wait_predecessor();
    Request r;
    if (!load_request_kv8(p, b, r)) return;
    const int rows_total = r.n * G;
    if (m0 >= rows_total) return;
    const int rows_here = min(kRowsPerCta, rows_total - m0);
    const bool dual = rows_here <= kGroupRows;

    // this split's tiles: n_pre of codes, then bf16 ones
    const int pre_tiles = prefix_tiles(r), total = request_units(p, r), pages8 = r.P / 16;
    const int Sb = unit_splits(total, p.C, p.S);
    if (split >= Sb) return;
    const int t_begin = unit_tile((int)((long long)total * split / Sb), pre_tiles);
    const int t_end = unit_tile((int)((long long)total * (split + 1) / Sb), pre_tiles);
    const int ntiles = t_end - t_begin;
    const int n_pre = max(0, min(t_end, pre_tiles) - t_begin);
    const bool has_tail = n_pre < ntiles;
    const int P0 = pages8 * 16;                  // first slot of the bf16 tiles
    auto tail_slot = [&](int j) { return P0 + (t_begin + j - pre_tiles) * kTileKeys; };

    if (warp == kMmaWarp) {
        tmem_alloc(&tmem_base_sh, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;

    // ----------------------------------------------------------- conversion
    // One team of warps fills the K tiles, another the V tiles.  `me` is the
    // warp's number in a team of kTeam.
    auto convert = [&](auto is_v_c, auto team_c, int me) {
        constexpr bool is_v = decltype(is_v_c)::value;
        constexpr int kTeam = decltype(team_c)::value;
        // A warp takes the pages me, me + kTeam, ... of each tile.  Their codes
        // come as one bulk copy each into the warp's own part of `raw`, one tile
        // ahead: no warp waits for another, and the loop over pages is short and
        // rolled, so that it and the softmax's code fit the instruction caches
        // together (unrolled it is 13% slower on 256 nodes over 16384 tokens;
        // codes copied by every lane or held in registers: 6-20%).
        // The page is read and stored in units of 512 bytes, 16 bytes a lane (4
        // rows at D = 128, 8 at D = 64).  Of eight neighbouring lanes four take
        // half a row of 128 bytes and four the other half of the next row: they
        // read all 32 banks, and the two rows' swizzled columns store to all.
        constexpr int kBlock = 16 * D;                       // codes of a page and head
        constexpr int kUnits = kBlock / 512;
        constexpr int kUnitRows = 16 / kUnits;
        const int urow = D == 128 ? ((lane >> 4) << 1) + ((lane >> 2) & 1) : lane >> 2;
        const int cc = D == 128 ? (lane & 3) | ((((lane >> 2) ^ (lane >> 3)) & 1) << 2) : lane & 3;
        const uint8_t *codes = is_v ? p.c.v : p.c.k;
        uint8_t *my_raw = raw + (is_v ? L::kRaw : 0);
        uint8_t *tiles = sKV + (is_v ? L::kKV : 0) + (cc >> 2) * (kTileKeys * 128);
        uint64_t *full = is_v ? v_full : k_full, *empty = is_v ? v_empty : k_empty;
        uint64_t *landed = &raw_full[is_v ? me : kVTeam + me];

        // lane l < 8: page l of a tile (-1: reads zeros)
        auto load_pages = [&](int j) -> int {
            int page = -1;
            const int lp = (t_begin + j) * kTilePages + lane;
            if (lane < kTilePages && j < n_pre && lp < pages8) {
                const long long pi = (long long)b * p.c.max_pages_per_req + lp;
                if (JSV_IN_BOUNDS(pi, (long long)a.B * p.c.max_pages_per_req, a.dev_status)) page = __ldg(p.c.page_table + pi);
                if (page < 0 || page >= p.c.num_pages) {
                    flag_error(a.dev_status, JSV_ERR_DEVICE_INPUT);
                    page = -1;
                }
            }
            return page;
        };
        auto fetch = [&](int pages) {                        // every lane is done with the last tile's
            const bool mine = pages >= 0 && (lane + kTeam - me) % kTeam == 0;
            const unsigned all = __ballot_sync(0xffffffffu, mine);
            if (lane == 0) mbar_arrive_expect_tx(landed, __popc(all) * kBlock);
            __syncwarp();
            if (mine)
                asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                                 smem_addr(my_raw + lane * kBlock)),
                             "l"(codes + ((size_t)pages * a.Hkv + g) * kBlock), "r"(kBlock), "r"(smem_addr(landed))
                             : "memory");
        };
        auto store = [&](uint8_t *tile, int pages, uint32_t ratios, uint32_t tiny) {
            const int chunk = (cc & 3) * 2;
#pragma unroll 1
            for (int pg = me; pg < kTilePages; pg += kTeam) {
                const bool there = __shfl_sync(0xffffffffu, pages, pg) >= 0;
                const uint32_t ratio = is_v ? __shfl_sync(0xffffffffu, ratios, pg) : 0u;
#pragma unroll 1
                for (int u0 = 0; u0 < kUnits; u0 += 2) {
                    uint4 w[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        w[u] = make_uint4(0, 0, 0, 0);
                        if (there)
                            w[u] = *reinterpret_cast<const uint4 *>(my_raw + pg * kBlock + (u0 + u) * 512 + urow * D + cc * 16);
                    }
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint32_t in[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
                        uint32_t f[8];
#pragma unroll
                        for (int k = 0; k < 4; ++k) codes_to_f16<FMT>(in[k], f[2 * k], f[2 * k + 1]);
                        if constexpr (is_v) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) f[k] = mul_f16x2(f[k], ratio);
                        }
                        // two units are 8 or 16 rows, so the swizzle goes by u alone
                        uint8_t *to = tile + pg * 2048 + u0 * (kUnitRows * 128);
                        const int row = u * kUnitRows + urow;
                        *reinterpret_cast<uint4 *>(to + sw128_offset(row, chunk)) = make_uint4(f[0], f[1], f[2], f[3]);
                        *reinterpret_cast<uint4 *>(to + sw128_offset(row, chunk + 1)) = make_uint4(f[4], f[5], f[6], f[7]);
                    }
                }
            }
            // the second step of tiny factors, by the lanes that stored the values
            // (a branch for it in the loop above cost 0.4%)
            if (is_v && tiny) {
#pragma unroll 1
                for (int i = me * kUnits; i < kTilePages * kUnits; i += (i + 1) % kUnits ? 1 : 1 + (kTeam - 1) * kUnits) {
                    if (!((tiny >> (i / kUnits)) & 1)) continue;
#pragma unroll 1
                    for (int k = 0; k < 2; ++k) {
                        uint4 *at = reinterpret_cast<uint4 *>(tile + (i & ~1) * (kUnitRows * 128) +
                                                              sw128_offset((i & 1) * kUnitRows + urow, chunk + k));
                        const uint4 x = *at;
                        *at = make_uint4(mul_f16x2(x.x, kTinyPair), mul_f16x2(x.y, kTinyPair), mul_f16x2(x.z, kTinyPair),
                                         mul_f16x2(x.w, kTinyPair));
                    }
                }
            }
        };
        // every thread's stores, then one arrival a warp
        auto hand_over = [&](uint64_t *bar) {
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        auto wait_for = [&](uint64_t *bar, uint32_t parity) -> bool {
            const bool done = mbar_wait(bar, parity, &abort_sh);
            if (__any_sync(0xffffffffu, !done)) {
                if (lane == 0) {
                    abort_sh = 1;
                    flag_error(a.dev_status, JSV_ERR_TIMEOUT);
                }
                return false;
            }
            return true;
        };
        // the second V tile's place holds the request's parents at first
        auto stage_free = [&](int j) -> bool {
            return wait_for(&empty[j % kStages], ((j / kStages) & 1) ^ 1) && (!is_v || j != 1 || wait_for(&tree_read, 0));
        };

        // Both teams keep the same reference, `want` where that lies outside
        // vref * [1/4, 2].  (A division here or in the softmax, with the code of
        // its rare cases, cost 6%.)
        float vref = 0.f, vinv = 0.f, vtop = 0.f;
        auto refer = [&](float want) {
            if (want > 2.f * vref || want < 0.25f * vref) {
                vtop = fmaxf(vtop, want);
                vref = fmaxf(want, vtop * kScaleRange);
                vinv = 1.f / vref;
            }
        };
        // page numbers two tiles ahead, scales one: neither is waited for
        int pages = load_pages(0), pages_next = load_pages(1);
        float ks, vs, ks_next, vs_next;
        auto load_scales = [&](int pages, float &ks, float &vs) {
            ks = vs = 0.f;
            if (pages >= 0) {
                const size_t block = (size_t)pages * a.Hkv + g;
                if constexpr (!is_v) ks = __ldg(p.c.k_scale + block);
                vs = __ldg(p.c.v_scale + block);
            }
        };
        fetch(pages);
        load_scales(pages, ks, vs);
        bool ok = true;
        for (int j = 0; j < n_pre; ++j) {
            load_scales(pages_next, ks_next, vs_next);
            const int pages_after = load_pages(j + 2);
            // the tile's scales: the largest V scale decides the reference
            float top = fabsf(vs);
#pragma unroll
            for (int off = 4; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            top = __shfl_sync(0xffffffffu, top, 0);
            if (top > kMinScale) refer(fmaxf(top * 0.015625f, kMinScale));
            float ratio = vs * vinv;
            const bool tiny = ratio != 0.f && fabsf(ratio) < kTinyRatio;
            if (tiny) ratio *= 1.f / kTinyRatio;
            ok = wait_for(landed, j & 1) && stage_free(j);
            if (!ok) break;
            if (!is_v && me == 0) {
                TileInfo &ti = info[j % kSlots];
                if (lane < kTilePages)                       // a page past the prefix: its columns are masked
                    ti.ks[lane] = (t_begin + j) * kTilePages + lane < pages8 ? finite_or_nan(ks) : 1.f;
                if (lane == 0) {
                    ti.vref = vref;
                    ti.vinv = vinv;
                }
            }
            store(tiles + (j % kStages) * L::kStage, pages, pack_f16(ratio, ratio), __ballot_sync(0xffffffffu, tiny));
            hand_over(&full[j % kStages]);
            pages = pages_next;
            fetch(pages);
            pages_next = pages_after;
            ks = ks_next;
            vs = vs_next;
        }
        if (!ok) {                                           // copies in flight land before this warp leaves
            int zero = 0;
            mbar_wait(landed, 0, (volatile int *)&zero);
            mbar_wait(landed, 1, (volatile int *)&zero);
        }
        // bf16 tiles, copied asynchronously to their places, all of a tile's rows
        // at once.
        constexpr int kRow16 = D / 8;                        // 16-byte chunks of a bf16 row
        constexpr int kTailUnits = kTileKeys * kRow16 / 32;  // 512 bytes each
        constexpr int kTailRows = 32 / kRow16;
        const uint16_t *cache = is_v ? p.v : p.k;
        const int trow = lane / kRow16, tc = lane % kRow16;
        auto load_tail_pages = [&](int j) -> int {           // lane l < 8: page l of tile j
            int page = -1;
            const int lp = tail_slot(j) / 16 + lane;
            if (lane < kTilePages && lp * 16 < r.P + r.n) {
                const long long pi = (long long)b * a.max_pages_per_req + lp;
                if (JSV_IN_BOUNDS(pi, (long long)a.B * a.max_pages_per_req, a.dev_status)) page = __ldg(a.page_table + pi);
                if (page < 0 || page >= a.num_pages) {
                    flag_error(a.dev_status, JSV_ERR_DEVICE_INPUT);
                    page = -1;
                }
            }
            return page;
        };
        int tail_pages = has_tail ? load_tail_pages(n_pre) : -1;
        for (int j = n_pre; ok && j < ntiles; ++j) {
            const int slot0 = tail_slot(j);
            TileInfo &ti = info[j % kSlots];
            refer(1.f);
            ok = stage_free(j);
            if (!ok) break;
            if (is_v) {
                if (lane < kTileKeys / 32) ti.bad[me][lane] = 0;
                __syncwarp();
            } else if (me == 0 && lane == 0) {
                ti.vref = vref;
                ti.vinv = vinv;
            }
            uint8_t *tile = sKV + (is_v ? L::kKV : 0) + (j % kStages) * L::kStage + (tc >> 3) * (kTileKeys * 128);
#pragma unroll 2
            for (int u = me; u < kTailUnits; u += kTeam) {
                const int row = u * kTailRows + trow;
                const int page = __shfl_sync(0xffffffffu, tail_pages, u * kTailRows / 16);
                const size_t at = (((size_t)max(page, 0) * 16 + row % 16) * a.Hkv + g) * D + tc * 8;
                const bool in = page >= 0 && slot0 + row < r.P + r.n &&
                                JSV_IN_BOUNDS(at + 7, (long long)a.num_pages * 16 * a.Hkv * D, a.dev_status);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(tile + sw128_offset(row, tc & 7))),
                             "l"(cache + (in ? at : 0)), "r"(in ? 16 : 0)
                             : "memory");
            }
            if (j + 1 < ntiles) tail_pages = load_tail_pages(j + 1);
            asm volatile("cp.async.wait_all;" ::: "memory");
            if constexpr (is_v) {
                // a weight of zero does not undo an infinity or NaN in the
                // product: such a row is zeroed here and noted
#pragma unroll 4
                for (int u = me; u < kTailUnits; u += kTeam) {
                    const int row = u * kTailRows + trow;
                    uint4 *at = reinterpret_cast<uint4 *>(tile + sw128_offset(row, tc & 7));
                    const uint4 w = *at;
                    const uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                                                __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
                    const unsigned odd = __ballot_sync(0xffffffffu, max(m & 0xffffu, m >> 16) >= 0x7f80u);
                    const unsigned mine = (kRow16 == 16 ? 0xffffu : 0xffu) << (lane / kRow16 * kRow16);
                    if (odd & mine) {
                        *at = make_uint4(0, 0, 0, 0);
                        if (tc == 0) atomicOr(&ti.bad[me][row >> 5], 1u << (row & 31));
                    }
                }
            }
            hand_over(&full[j % kStages]);
        }
    };

    if (warp < kMmaWarp) {
        setmaxnreg_dec<kRegsConv>();
        convert(std::true_type{}, std::integral_constant<int, kVTeam>{}, warp);
    } else if (warp < kSoftmaxWarp0) {
        setmaxnreg_dec<kRegsMma>();
        if (warp > kMmaWarp) {
            convert(std::false_type{}, std::integral_constant<int, kKTeam>{}, warp - kMmaWarp - 1);
        } else if (lane == 0 && ntiles > 0) {
            const uint32_t aQ = smem_addr(sQ), aKV = smem_addr(sKV);
            if (dual)
                kv8_mma_loop<D, true>(tmem, aQ, aKV, ntiles, n_pre, k_full, v_full, k_empty, v_empty, s_full, p_full,
                                      o_done, &q_ready, &drain_bar, &abort_sh, a.dev_status);
            else
                kv8_mma_loop<D, false>(tmem, aQ, aKV, ntiles, n_pre, k_full, v_full, k_empty, v_empty, s_full, p_full,
                                       o_done, &q_ready, &drain_bar, &abort_sh, a.dev_status);
        }
    } else {
        setmaxnreg_inc<kRegsSoftmax>();
        // ---------------------------------------------------------- softmax
        const int grp = (warp - kSoftmaxWarp0) >> 2, sub = warp & 3;
        const int grow = sub * 32 + lane;            // row within the group == TMEM lane
        const int first_row = dual ? 0 : grp * kGroupRows, row = first_row + grow;
        const uint32_t lane_addr = (uint32_t)(sub * 32) << 16;
        const uint32_t tS = tmem + grp * 128 + lane_addr, tO = tmem + 256 + grp * D + lane_addr;
        const int gt = threadIdx.x - 32 * (kSoftmaxWarp0 + 4 * grp);       // 0..127 in the group
        const bool row_valid = row < rows_here;
        const int rg = m0 + row, node = rg / G, head = g * G + rg % G;

        // The group's tiles: every one, or every other from its own number on.
        const int j0 = dual ? grp : 0, step = dual ? 2 : 1;

        // The group's rows of Q into its operand region, as bf16 or, scaled by a
        // power of two that brings the row's largest magnitude to [2^13, 2^14),
        // as fp16 in place.  D / 8 neighbouring threads share a row.
        constexpr int kRow16 = D / 8;
        constexpr int kQIters = kGroupRows * kRow16 / 128;
        const int qc = gt % kRow16;
        uint8_t *q_at = sQ + grp * L::kQGroup + (qc >> 3) * (kGroupRows * 128);
        {
            const float inv_g = 1.f / (float)G;              // (row + 1/2) / G truncates to the node
#pragma unroll 4
            for (int i = 0; i < kQIters; ++i) {
                const int rr = i * (128 / kRow16) + gt / kRow16, rgg = m0 + first_row + rr;
                const int nd = (int)(((float)rgg + 0.5f) * inv_g);
                const size_t qi = ((size_t)(r.base + nd) * a.Hq + g * G + (rgg - nd * G)) * D + qc * 8;
                const bool in = rgg < rows_total && JSV_IN_BOUNDS(qi + 7, (long long)a.total_nodes * a.Hq * D, a.dev_status);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(q_at + sw128_offset(rr, qc & 7))),
                             "l"(p.q + (in ? qi : 0)), "r"(in ? 16 : 0)
                             : "memory");
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            if (j0 < n_pre) {
#pragma unroll 4
                for (int i = 0; i < kQIters; ++i) {
                    const int rr = i * (128 / kRow16) + gt / kRow16;
                    uint4 *at = reinterpret_cast<uint4 *>(q_at + sw128_offset(rr, qc & 7));
                    const uint4 w = *at;
                    uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                                          __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
                    m = max(m & 0xffffu, m >> 16);
#pragma unroll
                    for (int off = 1; off < kRow16; off <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
                    const int ex = min(max((int)(m >> 7), 14), 254);
                    const float up = __uint_as_float((uint32_t)(267 - ex) << 23);
                    if (qc == 0) row_inv[grp * kGroupRows + rr] = __uint_as_float((uint32_t)(ex - 13) << 23);
                    auto two = [&](uint32_t x) {
                        return pack_f16(__uint_as_float(x << 16) * up, __uint_as_float(x & 0xffff0000u) * up);
                    };
                    *at = make_uint4(two(w.x), two(w.y), two(w.z), two(w.w));
                }
            }
            fence_async_smem();
        }
        // Back to bf16, in place.  Exact but for what lies 2^-28 and more below
        // the row's largest, which fp16 rounded to a multiple of 2^-24.
        auto q_to_bf16 = [&]() {
#pragma unroll 4
            for (int i = 0; i < kQIters; ++i) {
                const int rr = i * (128 / kRow16) + gt / kRow16;
                uint4 *at = reinterpret_cast<uint4 *>(q_at + sw128_offset(rr, qc & 7));
                const uint4 w = *at;
                const float inv = row_inv[grp * kGroupRows + rr];
                auto two = [&](uint32_t x) {
                    float lo, hi;
                    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
                        : "=f"(lo), "=f"(hi)
                        : "r"(x));
                    return pack_bf16x2(lo * inv, hi * inv);
                };
                *at = make_uint4(two(w.x), two(w.y), two(w.z), two(w.w));
            }
            fence_async_smem();
        };
        if (has_tail)
            for (int i = threadIdx.x - 32 * kSoftmaxWarp0; i < r.n; i += kGroups * 128)
                par_sh[i] = JSV_IN_BOUNDS(r.base + i, a.total_nodes, a.dev_status) ? __ldg(a.parent + r.base + i) : -1;
        named_barrier(1, kGroups * 128);         // Q, row factors and parents are in place
        if (lane == 0) mbar_arrive(&q_ready);
        // kept normal, so that a masked score stays -inf under it
        const float fac = fmaxf(p.scale_log2 * row_inv[grp * kGroupRows + grow], 1.2e-38f);
        uint32_t anc[kTreeWords];                // this row's ancestors and itself (local memory: read in bf16 tiles only)
        if (has_tail && row_valid) {
            for (int w = 0; w < kTreeWords; ++w) anc[w] = 0;
            int j = node;
            while (j != -1) {
                anc[j >> 5] |= 1u << (j & 31);
                const int pj = par_sh[j];
                if (j == 0 ? pj != -1 : (pj < 0 || pj >= j)) {
                    flag_error(a.dev_status, JSV_ERR_DEVICE_INPUT);
                    break;
                }
                j = pj;
            }
        }

        __syncwarp();
        if (lane == 0) mbar_arrive(&tree_read);

        float m_used = -INFINITY, l = 0.f, vref = 0.f;
        bool ok = true;
        const int my_tiles = max(0, (ntiles - j0 + step - 1) / step);
        int done = 0;                                // tiles of this group so far
        // Three kinds of tile, each with code of its own, so that the many of the
        // first kind run through little of it: 8-bit tiles; the group's last of
        // them, which may hold fewer pages and is followed by bf16 tiles; those.
        auto one_tile = [&](int j, auto kind_c) -> bool {
            constexpr bool is_last = decltype(kind_c)::value == 1, is_tail = decltype(kind_c)::value == 2;
            if (!mbar_wait(&s_full[grp], done & 1, &abort_sh)) ok = false;
            // what is noted about the rows of a bf16 V tile comes with the tile
            if (is_tail && !mbar_wait(&v_full[j % kStages], (j / kStages) & 1, &abort_sh)) ok = false;
            if (__any_sync(0xffffffffu, !ok)) {
                ok = false;
                return false;
            }
            tc_fence_after();
            const TileInfo &ti = info[j % kSlots];
            // The row's 128 scores, 64 columns at a time.  The weights go over the
            // first 64 columns, so the second half is read for the maximum,
            // dropped, and read again for its weights.  The weights' loop is kept
            // rolled: with the whole row unrolled, the softmax and the converting
            // warps' code did not fit the instruction caches together.
            uint32_t sv[2][32];
            auto load_half = [&](int h) {
                tmem_ld_32x32b_x32(tS + h * 64, sv[0]);
                tmem_ld_32x32b_x32(tS + h * 64 + 32, sv[1]);
            };
            load_half(1);
            // O is rescaled where the reference scale has changed since this group's last tile
            const float vnew = ti.vref, vinv = ti.vinv, vratio = vnew == vref ? 1.f : vref * vinv;
            vref = vnew;
            // columns that are not seen become -inf: by a word of the tree's
            // visibility for 32 columns, or whole pages past the prefix in its last tile
            uint32_t vis[kTileKeys / 32];
            const int nb = is_tail ? kTilePages : pages8 - (t_begin + j) * kTilePages;       // pages this tile holds
            if constexpr (is_tail) {
                const int slot0 = tail_slot(j);
#pragma unroll
                for (int c = 0; c < kTileKeys / 32; ++c) {
                    const int j0 = slot0 + c * 32 - r.P;         // tree node of column 32c (< 0: prefix, seen by all)
                    vis[c] = 0u;
                    if (row_valid) {
                        if (j0 <= -32) {
                            vis[c] = 0xffffffffu;
                        } else if (j0 < 0) {
                            vis[c] = (anc[0] << (-j0)) | ((1u << (-j0)) - 1u);
                        } else if (j0 < kMaxTreeNodes) {
                            const int w = j0 >> 5;
                            vis[c] = __funnelshift_r(anc[w], w + 1 < kTreeWords ? anc[w + 1] : 0u, j0 & 31);
                        }
                        if (vis[c] & (ti.bad[0][c] | ti.bad[1][c] | ti.bad[2][c] | ti.bad[3][c])) l = __uint_as_float(0x7fc00000u);
                    }
                }
            }
            auto mask_half = [&](int h) {
                if constexpr (is_tail) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint32_t v = h ? vis[2 + c] : vis[c];
#pragma unroll
                        for (int x = 0; x < 32; ++x) sv[c][x] = ((v >> x) & 1u) ? sv[c][x] : 0xff800000u;
                    }
                } else if (is_last && nb < kTilePages) {
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            if (h * 4 + 2 * c + x / 16 >= nb) sv[c][x] = 0xff800000u;
                }
            };
            // what brings each page's 16 columns to log2 units
            auto factors = [&](int h) -> float4 {
                if constexpr (is_tail) return make_float4(p.scale_log2, p.scale_log2, p.scale_log2, p.scale_log2);
                const float4 k = *reinterpret_cast<const float4 *>(&ti.ks[4 * h]);
                return make_float4(fac * k.x, fac * k.y, fac * k.z, fac * k.w);
            };
            // row maximum, a page at a time (scales are not negative)
            float tmax = -INFINITY;
            auto max_half = [&](int h) {
                const float4 f4 = factors(h);
                const float f[4] = {f4.x, f4.y, f4.z, f4.w};
                mask_half(h);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t *s = &sv[k / 2][(k & 1) * 16];
                    float u0 = fmax3(__uint_as_float(s[0]), __uint_as_float(s[1]), __uint_as_float(s[2]));
                    float u1 = fmax3(__uint_as_float(s[3]), __uint_as_float(s[4]), __uint_as_float(s[5]));
#pragma unroll
                    for (int x = 6; x < 14; x += 4) {
                        u0 = fmax3(u0, __uint_as_float(s[x]), __uint_as_float(s[x + 1]));
                        u1 = fmax3(u1, __uint_as_float(s[x + 2]), __uint_as_float(s[x + 3]));
                    }
                    u0 = fmax3(u0, __uint_as_float(s[14]), __uint_as_float(s[15]));
                    tmax = fmaxf(tmax, fmaxf(u0, u1) * f[k]);
                }
            };
            tmem_ld_wait();
            max_half(1);
            load_half(0);
            tmem_ld_wait();
            max_half(0);
            float m_new = m_used;
            if (tmax > m_used + kMaxSlack) m_new = tmax;
            const float corr = m_new == m_used ? 1.f : fast_exp2(m_used - m_new);     // 0 when m_used = -inf
            const float corr_o = corr * vratio;
            // O holds the earlier tiles' sum under the old maximum and reference
            // scale.  S_j was issued after PV_{j-1} and completes after it.
            if (__any_sync(0xffffffffu, corr_o != 1.f) && done > 0) {
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 16) {
                    uint32_t ov[16];
                    tmem_ld_32x32b_x16(tO + c0, ov);
                    tmem_ld_wait();
#pragma unroll
                    for (int x = 0; x < 16; ++x) ov[x] = __float_as_uint(__uint_as_float(ov[x]) * corr_o);
                    tmem_st_32x32b_x16(tO + c0, ov);
                }
                tmem_st_wait();
            }
            const float base = m_new == -INFINITY ? kWeightLog2 : kWeightLog2 - m_new;
            const uint64_t base2 = f2_pack(base, base);
            uint64_t ps2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
            // bf16 values carry no scale of their own: their weights take 1 / vref
            const float unscale = is_tail ? vinv : 1.f;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                if (h) {
                    load_half(1);
                    tmem_ld_wait();
                    mask_half(1);
                }
                const float4 f4 = factors(h);
                const float fs[4] = {f4.x, f4.y, f4.z, f4.w};
                uint32_t pk[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float f = fs[i / 8];
                    const uint64_t xa = f2_fma(f2_pack(__uint_as_float(sv[i / 16][2 * (i % 16)]),
                                                       __uint_as_float(sv[i / 16][2 * (i % 16) + 1])), f2_pack(f, f), base2);
                    float u0, u1;
                    f2_unpack(xa, u0, u1);
                    u0 = fast_exp2(u0);
                    u1 = fast_exp2(u1);
                    ps2[i & 1] = f2_add(ps2[i & 1], f2_pack(u0, u1));
                    pk[i] = is_tail ? pack_bf16x2(u0 * unscale, u1 * unscale) : pack_f16(u0, u1);
                }
                tmem_st_32x32b_x32(tS + h * 32, pk);
            }
            float q0, q1, q2, q3;
            f2_unpack(ps2[0], q0, q1);
            f2_unpack(ps2[1], q2, q3);
            l = l * corr + ((q0 + q1) + (q2 + q3));
            m_used = m_new;
            tmem_st_wait();
            // the next tile is bf16, and so is Q from here on: this group's S of the
            // last 8-bit tile is complete, and the next is issued after these
            // warps' arrivals
            if (is_last && j + step < ntiles) q_to_bf16();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[grp]);
            ++done;
            return true;
        };
        int j = j0;
        for (; ok && j + step < n_pre; j += step) one_tile(j, std::integral_constant<int, 0>{});
        if (ok && j < n_pre) {
            one_tile(j, std::integral_constant<int, 1>{});
            j += step;
        }
        for (; ok && j < ntiles; j += step) one_tile(j, std::integral_constant<int, 2>{});

        bool have_o = ok && my_tiles > 0;
        if (have_o) {
            if (!mbar_wait(&o_done[grp], (uint32_t)((my_tiles - 1) & 1), &abort_sh)) ok = false;
            if (__any_sync(0xffffffffu, !ok)) have_o = false;
        }
        if (!have_o) {
            m_used = -INFINITY;
            l = 0.f;
            if (!ok) {
                abort_sh = 1;
                flag_error(a.dev_status, JSV_ERR_TIMEOUT);
            }
        }
        // Where both groups have the same rows, the second hands its result to the
        // first through the operand ring (every product has completed once both
        // are at the barrier).
        float4 *other = reinterpret_cast<float4 *>(sKV);             // [D / 4][128 rows]
        float2 *other_ml = reinterpret_cast<float2 *>(sKV + kGroupRows * D * 4);
        // Factors of the two groups' O.  Rows are handed on divided by their own
        // sum, as averages of V: a sum of large values might not be finite.
        float mine = l == 0.f ? vref : vref / l, theirs = 0.f;
        const bool add = dual && ntiles > 1;                         // with a factor that underflowed to zero too
        if (dual) {
            named_barrier(1, kGroups * 128);
            if (grp == 1) {
                other_ml[grow] = make_float2(m_used, l);
                if (have_o) {
                    tc_fence_after();
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 16) {
                        uint32_t rr[16];
                        tmem_ld_32x32b_x16(tO + c0, rr);
                        tmem_ld_wait();
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            other[(c0 / 4 + x) * kGroupRows + grow] =
                                make_float4(__uint_as_float(rr[4 * x]) * mine, __uint_as_float(rr[4 * x + 1]) * mine,
                                            __uint_as_float(rr[4 * x + 2]) * mine, __uint_as_float(rr[4 * x + 3]) * mine);
                    }
                }
            }
            named_barrier(1, kGroups * 128);
            if (grp == 0) {
                const float2 ml = other_ml[grow];
                if (add) {
                    const float M = fmaxf(m_used, ml.x);
                    const float w0 = l == 0.f ? 0.f : m_used == -INFINITY ? l : fast_exp2(m_used - M) * l;
                    const float w1 = ml.y == 0.f ? 0.f : ml.x == -INFINITY ? ml.y : fast_exp2(ml.x - M) * ml.y;
                    l = w0 + w1;
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    mine *= w0 * inv;
                    theirs = w1 * inv;
                    m_used = M;
                }
            }
        }
        // The rows, in whole rows through this warp's slice of the group's Q
        // region (every product of the group has completed), half of D at a time.
        const size_t rows = (size_t)a.total_nodes * a.Hq;
        const size_t row_id = (size_t)(r.base + min(node, r.n - 1)) * a.Hq + head;
        constexpr int kScrCols = D / 2, kChunks = kScrCols / 4, kRowsPerStore = 32 / kChunks;
        float4 *scr = reinterpret_cast<float4 *>(sQ + grp * L::kQGroup + sub * (32 * kScrCols * 4));
        if (have_o) tc_fence_after();
        auto write_rows = [&](long long my_off, auto store) {
#pragma unroll 1
            for (int pass = 0; pass < 2; ++pass) {
#pragma unroll
                for (int c0 = 0; c0 < kScrCols; c0 += 32) {
                    uint32_t rr[32];
                    if (have_o) {
                        tmem_ld_32x32b_x32(tO + pass * kScrCols + c0, rr);
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int x = 0; x < 32; ++x) rr[x] = 0u;
                    }
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        float4 v = make_float4(__uint_as_float(rr[4 * x]) * mine, __uint_as_float(rr[4 * x + 1]) * mine,
                                               __uint_as_float(rr[4 * x + 2]) * mine, __uint_as_float(rr[4 * x + 3]) * mine);
                        if (add) {
                            const float4 u = other[((pass * kScrCols + c0) / 4 + x) * kGroupRows + grow];
                            v.x = fmaf(u.x, theirs, v.x), v.y = fmaf(u.y, theirs, v.y);
                            v.z = fmaf(u.z, theirs, v.z), v.w = fmaf(u.w, theirs, v.w);
                        }
                        scr[lane * kChunks + ((c0 / 4 + x) ^ (lane & (kChunks - 1)))] = v;
                    }
                }
                __syncwarp();
#pragma unroll 4
                for (int i = 0; i < 32; i += kRowsPerStore) {
                    const int wr = i + lane / kChunks, ch = lane % kChunks;
                    const long long off = __shfl_sync(0xffffffffu, my_off, wr);
                    const float4 v = scr[wr * kChunks + (ch ^ (wr & (kChunks - 1)))];
                    if (off >= 0) store(off + pass * kScrCols + ch * 4, v);
                }
                __syncwarp();
            }
        };
        if (dual && grp == 1) {
            // merged into the first group's rows
        } else if (Sb == 1) {
            if (l == 0.f) mine = __uint_as_float(0x7fc00000u);       // no weight at all: every score -inf
            write_rows(row_valid ? (long long)(row_id * D) : -1ll,
                       [&](long long o, const float4 &v) {
                           if (JSV_IN_BOUNDS(o + 3, (long long)rows * D, a.dev_status))
                               *reinterpret_cast<uint2 *>(p.out + o) = make_uint2(pack_bf16x2(v.x, v.y),
                                                                                  pack_bf16x2(v.z, v.w));
                       });
        } else {
            write_rows(row_valid ? (long long)(((size_t)split * rows + row_id) * D) : -1ll,
                       [&](long long o, const float4 &v) {
                           if (JSV_IN_BOUNDS(o + 3, (long long)p.S * rows * D, a.dev_status))
                               *reinterpret_cast<float4 *>(p.ws_o + o) = v;
                       });
            const size_t mi = (size_t)split * rows + row_id;
            if (row_valid && JSV_IN_BOUNDS(mi, (long long)p.S * rows, a.dev_status))
                *reinterpret_cast<float2 *>(p.ws_ml + mi * 2) = make_float2(m_used, l);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, int FMT>
static cudaError_t launch_tiles(const Kv8Params &p, cudaStream_t st) {
    using L = TileSmem<D>;
    auto kernel = kv8_tiles_kernel<D, FMT>;
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
    dim3 grid((p.a.max_nodes * G + kRowsPerCta - 1) / kRowsPerCta, p.S, p.a.B * p.a.Hkv);
    e = launch_pdl(kernel, grid, dim3(kTileThreads), L::kTotal, st, p);
    if (e != cudaSuccess) {
        cudaFuncAttributes fa;
        if (cudaFuncGetAttributes(&fa, kernel) == cudaSuccess)
            note_launch_failure("tree attention over 8-bit pages", fa.numRegs, fa.maxThreadsPerBlock, fa.sharedSizeBytes,
                                fa.maxDynamicSharedSizeBytes, kTileThreads, L::kTotal);
        return e;
    }
    count_launches(1);
    return cudaSuccess;
}

cudaError_t launch_kv8_tiles(const Kv8Params &p, cudaStream_t st) {
    const bool e4m3 = p.c.format == JSV_KV8_E4M3;
    if (p.a.D == 128) return e4m3 ? launch_tiles<128, JSV_KV8_E4M3>(p, st) : launch_tiles<128, JSV_KV8_INT8>(p, st);
    return e4m3 ? launch_tiles<64, JSV_KV8_E4M3>(p, st) : launch_tiles<64, JSV_KV8_INT8>(p, st);
}

}  // namespace jsv
