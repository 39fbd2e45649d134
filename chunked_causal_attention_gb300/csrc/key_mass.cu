// The attention weight of each key, summed over query rows and the heads of its
// key/value head, from q, k and the forward's log-sum-exp:
//
//   mass_j = sum_{h, t visible} exp(scale q_t . k_j - LSE_t)
//
// One work item is a tile of 128 keys of one key/value head; it walks every block
// of at most 128 query rows that sees the tile, for each head of the group, so a
// key's sum stays with one thread and needs no atomics: the result does not depend
// on timing. Persistent blocks take items, those with the most rows first within a
// head, from a work queue (WorkRing in tc_common.cuh). Warp roles:
//   warp 0      TMA producer: the K tile of an item, Q blocks through a ring
//   warp 1      MMA issuer and TMEM owner: S^T = K Q^T (M = 128 keys, N = rows of
//               the block) into one of four 128-column TMEM buffers
//   warp 2      the rows' -lse log2 e into shared memory, up to four blocks ahead
//   warps 4-15  three groups that take the blocks in turn: thread = key (TMEM
//               lane); it reads its row of S^T, forms 2^(s c - lse2) with the
//               block's lse2 from shared memory (two columns per instruction where
//               the pipe allows) and sums. The warps meet no barrier among
//               themselves
//   warp 3      adds up the groups' sums of a finished item, in order, and writes them
// Per block 2 * 128 * 128 * D FLOP (512 cycles of an SM at D = 128) stand against
// 128 * 128 exponentials (512 cycles at 32 a cycle): both pipes are needed whole.
// Measured, the kernel alone: 8192 tokens of 32 heads of 128 dims 245 to 260 us (1060 to
// 1120 TFLOP/s, 1060 cycles a block; a call 260), 32768 tokens 3.3 to 3.4 ms (1290 to 1340
// TFLOP/s); both pipes are 53% busy at 8192. Copies without the
// exponentials (195 us) and also without most products (154 to 179 us) show that the
// hand-over of a block from pipe to pipe is what is left; three groups hide more of it
// than two (266 us) and than four on fewer registers (299 us).
//
// Sums: 128 weights of a block in four fp32 chains, blocks with a compensated sum
// (Kahan), so that a million rows lose no more than a block does. (The kernel for few
// rows has at most eight blocks a key and adds them plainly.) A weight's own error is
// larger: scores are summed by the tensor core, 2^(s c - lse2) is one FMA and ex2.approx;
// 7e-7 of the masses at 8192 tokens, where fp32 throughout has 2e-7.
//
// Every mbarrier wait is bounded (ATTN_E_TIMEOUT); items and chunks are checked
// before use (ATTN_E_BOUNDS).
#include <algorithm>

#include "kv4.h"
#include "tc_common.cuh"

namespace attn {
namespace {

using namespace tc;

constexpr int kGroups = 3;                 // softmax warpgroups
constexpr int kThreads = 128 + 128 * kGroups;
constexpr int kBufs = 4;                   // S^T buffers in TMEM
constexpr uint32_t kTmemCols = 512;
constexpr int kRows = 128;                 // query rows of a block
constexpr int kBoxRows = 64;               // rows of a TMA box

template <int DT>
struct Layout {
    static constexpr int KST = DT == 256 ? 1 : 2, QST = DT == 256 ? 2 : DT == 128 ? 4 : 8;
    static constexpr int TILE = 128 * DT * 2;
    static constexpr int K_OFF = 0, Q_OFF = KST * TILE;
    static constexpr int LSE_OFF = Q_OFF + QST * TILE;            // [buffer][128] floats
    static constexpr int PART_OFF = LSE_OFF + kBufs * 128 * 4;   // [2][group][128] floats
    static constexpr int ITEM_OFF = PART_OFF + 2 * kGroups * 128 * 4;           // [2] items handed out
    static constexpr int TAG_OFF = ITEM_OFF + 2 * 16;                            // [buffer] tag of the block whose lse it holds
    static constexpr int BAR_OFF = TAG_OFF + kBufs * 4;
    static constexpr int B_KFULL = 0, B_KEMPTY = B_KFULL + KST;
    static constexpr int B_QFULL = B_KEMPTY + KST, B_QEMPTY = B_QFULL + QST;
    static constexpr int B_SFULL = B_QEMPTY + QST, B_SEMPTY = B_SFULL + kBufs;
    static constexpr int B_LEMPTY = B_SEMPTY + kBufs;
    static constexpr int B_PFULL = B_LEMPTY + kBufs, B_PEMPTY = B_PFULL + 2;
    static constexpr int B_RFULL = B_PEMPTY + 2, B_REMPTY = B_RFULL + 2;
    static constexpr int B_DRAIN = B_REMPTY + 2;
    static constexpr int NBAR = B_DRAIN + 1;
    static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
    static constexpr int BYTES = MISC_OFF + 16;
    static constexpr size_t ALLOC = (size_t)BYTES + 1024;
};

// The query blocks of an item in order (chunk, head of the group, 128 rows): of every
// `every` the one numbered `mine`, counting within the item, so that which group sums a
// block does not depend on the items before. f(number, context begin, head, first row,
// rows) until it returns false, the number counting on from `count`. False: f did, or a
// chunk is not one (bad).
template <typename F>
__device__ __forceinline__ bool walk_blocks(const MassArgs& a, const MassItem& it, int G, uint32_t& count, uint32_t every,
                                            uint32_t mine, bool& bad, F f) {
    const uint32_t start = count;
    for (int32_t c = it.c_lo; c < it.c_hi; ++c) {
        const attn_chunk ch = a.chunks[c];
        if (!(0 <= ch.ctx_begin && ch.ctx_begin <= ch.q_begin && ch.q_begin < ch.q_end && ch.q_end <= a.g.T)) {
            bad = true;
            return false;
        }
        if (ch.ctx_begin >= it.j1 || ch.q_end <= it.j0) continue;
        const int32_t r0 = max(ch.q_begin, it.j0), nb = (ch.q_end - r0 + kRows - 1) / kRows;
        for (int32_t g = 0; g < G; ++g) {
            for (int32_t x = every == 1 ? 0 : (int32_t)((mine + every - (count - start) % every) % every); x < nb; x += every) {
                const int32_t r = r0 + x * kRows;
                if (!f(count + x, ch.ctx_begin, g, r, min(kRows, ch.q_end - r))) return false;
            }
            count += nb;
        }
    }
    return true;
}

// A group sums the blocks x of an item with x % kGroups == turn: the first block goes to
// another group from tile to tile, for items of few blocks.
__device__ __forceinline__ uint32_t turn_of(const MassItem& it, int grp) { return (uint32_t)(grp + it.j0 / 128) % kGroups; }
// Whether any row sees a key of the item.
__device__ __forceinline__ bool seen(const MassArgs& a, const MassItem& it) {
    for (int32_t c = it.c_lo; c < it.c_hi; ++c)
        if (a.chunks[c].ctx_begin < it.j1 && a.chunks[c].q_end > it.j0) return true;
    return false;
}

// The tag of block q's log-sum-exps in a buffer, the lowest bit set where a row of the
// block has none (-inf). Such a row weighs nothing whatever its query holds, and
// 2^(s c - inf) is 0 only while the score s is not NaN or +inf: blocks with one select.
__device__ __forceinline__ uint32_t tag_of(uint32_t q, bool without) { return 2 * (q + 1) + (without ? 1u : 0u); }
__device__ __forceinline__ bool same_block(uint32_t tag, uint32_t want) { return ((tag ^ want) & ~1u) == 0; }

// Wait, for a whole warp, until *tag is the block's of `want`; bounded like an mbarrier wait.
__device__ __noinline__ bool tag_wait(volatile uint32_t* tag, uint32_t want, volatile int* abort, uint32_t* status,
                                      uint64_t limit_ns) {
    const uint64_t t0 = globaltimer();
    bool ok = true;
    while (ok && !same_block(*tag, want)) {
        if (*abort) {
            ok = false;
        } else if (globaltimer() - t0 > limit_ns) {
            *abort = 1;
            set_error(status, ATTN_E_TIMEOUT);
            ok = false;
        }
    }
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ bool item_ok(const MassItem& it, const MassArgs& a) {
    return 0 <= it.j0 && it.j0 < it.j1 && it.j1 - it.j0 <= 128 && it.j1 <= a.g.T && 0 <= it.c_lo && it.c_hi <= a.n;
}

// The MMA thread's instructions are what a block waits for: alone in its warp it issues
// one in about ten cycles, and a trace of it showed 390 cycles for eight MMAs whose
// descriptors were built one by one. So a tile's descriptor is built once; a step of 16
// dims adds to its low word (the address field: 14 bits of 16 bytes each, which the
// shared memory's 228 KB never carry out of).
struct TileDesc {
    uint32_t lo, hi;
    __device__ __forceinline__ explicit TileDesc(uint32_t saddr) {
        const uint64_t d = sdesc_sw128(saddr, 16, 1024);
        lo = (uint32_t)d;
        hi = (uint32_t)(d >> 32);
    }
    __device__ __forceinline__ uint64_t at(uint32_t bytes) const {
        uint64_t d;
        asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo + (bytes >> 4)), "r"(hi));
        return d;
    }
};

// ROWS rows x DT dims: boxes of 64 dims x 64 rows, dims in strides of 128 rows.
template <int DT>
__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap* map, uint32_t bar, const TcMaps& mp, int row,
                                          int boxes, int h, int b) {
    for (int y = 0; y < boxes; ++y) {
        const int t = row + y * kBoxRows;
        const int c1 = mp.pos_t == 1 ? t : (mp.pos_h == 1 ? h : b);
        const int c2 = mp.pos_t == 2 ? t : (mp.pos_h == 2 ? h : b);
        const int c3 = mp.pos_t == 3 ? t : (mp.pos_h == 3 ? h : b);
#pragma unroll
        for (int x = 0; x < DT / 64; ++x) tma_load_4d(dst + x * 128 * 128 + y * kBoxRows * 128, map, bar, x * 64, c1, c2, c3);
    }
}

// Weights of 64 columns that all see this thread's key, into four running sums.
__device__ __forceinline__ void weigh64(const uint32_t (&r)[2][32], const float* lse, float2 c2, float2 (&acc)[2]) {
    const float4* l4 = reinterpret_cast<const float4*>(lse);
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 8; ++y) {
            const float4 l = l4[8 * x + y];
            const float2 e0 =
                ffma2(make_float2(__uint_as_float(r[x][4 * y]), __uint_as_float(r[x][4 * y + 1])), c2, make_float2(l.x, l.y));
            const float2 e1 =
                ffma2(make_float2(__uint_as_float(r[x][4 * y + 2]), __uint_as_float(r[x][4 * y + 3])), c2, make_float2(l.z, l.w));
            acc[0] = fadd2(acc[0], make_float2(ex2(e0.x), ex2(e0.y)));
            acc[1] = fadd2(acc[1], make_float2(ex2(e1.x), ex2(e1.y)));
        }
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 1)
    key_mass_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk, const MassArgs a,
                    const TcMaps mp, const TcMaps mpkv, const int32_t n_work) {
    using L = Layout<DT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(sm);
    auto bar = [&](int i) { return sbase + L::BAR_OFF + 8u * (uint32_t)i; };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::MISC_OFF + 4);
    const WorkRing ring{reinterpret_cast<volatile int32_t*>(sm + L::MISC_OFF + 8), bar(L::B_RFULL), bar(L::B_REMPTY)};
    const int tid = threadIdx.x, warp = tid >> 5;
    const int BH = a.g.B * a.g.Hkv, G = a.g.H / a.g.Hkv;
    MassItem* s_item = reinterpret_cast<MassItem*>(sm + L::ITEM_OFF);
    volatile uint32_t* s_tag = reinterpret_cast<volatile uint32_t*>(sm + L::TAG_OFF);
    // a role that is a whole warp takes the next item: false at the end
    auto take_warp = [&](uint32_t ic, MassItem& item, int32_t& bh) {
        if (!mbar_wait_warp(ring.full + 8 * (ic & 1), (ic >> 1) & 1, abort_flag, a.status, a.wait_ns)) return false;
        bh = ring.slot[ic & 1];
        item = s_item[ic & 1];
        __syncwarp();
        if ((tid & 31) == 0) mbar_arrive(ring.empty + 8 * (ic & 1));
        return bh >= 0;
    };

    if (tid == 0) {
        for (int s = 0; s < L::KST; ++s) {
            mbar_init(bar(L::B_KFULL + s), 1);
            mbar_init(bar(L::B_KEMPTY + s), 1);
        }
        for (int s = 0; s < L::QST; ++s) {
            mbar_init(bar(L::B_QFULL + s), 1);
            mbar_init(bar(L::B_QEMPTY + s), 1);
        }
        for (int s = 0; s < kBufs; ++s) {
            mbar_init(bar(L::B_SFULL + s), 2);                 // the products and the rows' lse
            s_tag[s] = 0;
            mbar_init(bar(L::B_SEMPTY + s), 128);
            mbar_init(bar(L::B_LEMPTY + s), 128);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(L::B_PFULL + s), 128 * kGroups);
            mbar_init(bar(L::B_PEMPTY + s), 32);
            mbar_init(bar(L::B_RFULL + s), 1);
            mbar_init(bar(L::B_REMPTY + s), 3 + 4 * kGroups);
        }
        mbar_init(bar(L::B_DRAIN), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (elect_one()) {
            tma_prefetch_desc(&tmq);
            tma_prefetch_desc(&tmk);
            uint32_t kc = 0, qc = 0, ic = 0;
            // An item is read one ahead, so that the list is not waited for between
            // items. (Claiming two ahead before the loads took 259 us at 8K tokens against 251: the
            // blocks end less evenly.)
            auto item_of = [&](int32_t w, int32_t& bh) {
                int32_t i = 0;
                bh = 0;
                if (w >= n_work) return MassItem{0, 0, 0, 0};
                decode_work(w, a.n_items, BH, 1 << 30, i, bh);
                return a.items[i];
            };
            int32_t w = a.stall ? n_work : (int32_t)atomicAdd(a.counter, 1u);
            int32_t w1 = a.stall ? n_work : (int32_t)atomicAdd(a.counter, 1u);
            int32_t w2 = n_work, bh = 0, bh1 = 0;
            MassItem item = item_of(w, bh), item1 = item;
            for (; !a.stall; ++ic, w = w1, w1 = w2, item = item1, bh = bh1) {
                if (w < n_work) {
                    if (!item_ok(item, a)) {
                        set_error(a.status, ATTN_E_BOUNDS);
                        *abort_flag = 1;
                        break;
                    }
                    // the slot is free once every role has taken the item before the last (ring_put waits for it too)
                    if (!mbar_wait(bar(L::B_REMPTY + (ic & 1)), ((ic >> 1) & 1) ^ 1, abort_flag, a.status, a.wait_ns)) break;
                    s_item[ic & 1] = item;
                }
                if (!ring_put(ring, ic, w < n_work ? bh : -1, abort_flag, a.status, a.wait_ns)) break;
                if (w >= n_work || *abort_flag) break;
                item1 = item_of(w1, bh1);
                const int b = bh / a.g.Hkv, hk = bh % a.g.Hkv;
                bool ok = true, bad = false;
                if (seen(a, item)) {
                    const uint32_t s = kc % L::KST;
                    ok = mbar_wait(bar(L::B_KEMPTY + s), ((kc / L::KST) & 1) ^ 1, abort_flag, a.status, a.wait_ns);
                    if (!ok) break;
                    mbar_expect_tx(bar(L::B_KFULL + s), L::TILE);
                    load_rows<DT>(sbase + L::K_OFF + s * L::TILE, &tmk, bar(L::B_KFULL + s), mpkv, item.j0, 2, hk, b);
                    ++kc;
                }
                walk_blocks(a, item, G, qc, 1, 0, bad, [&](uint32_t q, int, int g, int r, int rows) {
                    const uint32_t s = q % L::QST;
                    ok = mbar_wait(bar(L::B_QEMPTY + s), ((q / L::QST) & 1) ^ 1, abort_flag, a.status, a.wait_ns);
                    if (!ok) return false;
                    const int boxes = rows > kBoxRows ? 2 : 1;
                    mbar_expect_tx(bar(L::B_QFULL + s), boxes * (L::TILE / 2));
                    load_rows<DT>(sbase + L::Q_OFF + s * L::TILE, &tmq, bar(L::B_QFULL + s), mp, r, boxes, hk * G + g, b);
                    return true;
                });
                if (!ok) break;
                if (bad) {
                    set_error(a.status, ATTN_E_BOUNDS);
                    *abort_flag = 1;
                    break;
                }
                w2 = (int32_t)atomicAdd(a.counter, 1u);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (elect_one()) {
            uint32_t kc = 0, qc = 0, ic = 0;
            bool ok = true;
            for (; ok; ++ic) {
                if (!mbar_wait(ring.full + 8 * (ic & 1), (ic >> 1) & 1, abort_flag, a.status, a.wait_ns)) break;
                const int32_t bh = ring.slot[ic & 1];
                const MassItem item = s_item[ic & 1];
                mbar_arrive(ring.empty + 8 * (ic & 1));
                if (bh < 0 || *abort_flag) break;
                if (!seen(a, item)) continue;
                const uint32_t ks = kc % L::KST;
                ok = mbar_wait(bar(L::B_KFULL + ks), (kc / L::KST) & 1, abort_flag, a.status, a.wait_ns);
                if (!ok) break;
                const TileDesc k0(sbase + L::K_OFF + ks * L::TILE);
                bool bad = false;
                ok = walk_blocks(a, item, G, qc, 1, 0, bad, [&](uint32_t q, int, int, int, int rows) {
                    const uint32_t qs = q % L::QST, sb = q % kBufs;
                    if (!mbar_wait(bar(L::B_QFULL + qs), (q / L::QST) & 1, abort_flag, a.status, a.wait_ns) ||
                        !mbar_wait(bar(L::B_SEMPTY + sb), ((q / kBufs) & 1) ^ 1, abort_flag, a.status, a.wait_ns))
                        return false;
                    tc_fence_after();
                    const TileDesc q0(sbase + L::Q_OFF + qs * L::TILE);
                    // as many columns as the block has rows, in steps of 16
                    const uint32_t id = idesc_bf16(128, (rows + 15) & ~15, 0, 0);
#pragma unroll
                    for (int kk = 0; kk < DT / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * (128 * 128) + (kk & 3) * 32;
                        mma_ss(tmem + sb * kRows, k0.at(off), q0.at(off), id, kk > 0);
                    }
                    mma_commit(bar(L::B_QEMPTY + qs));
                    mma_commit(bar(L::B_SFULL + sb));
                    return true;
                });
                if (!ok) break;
                mma_commit(bar(L::B_KEMPTY + ks));
                ++kc;
            }
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------ log-sum-exps
        const int lane = tid & 31;
        uint32_t qc = 0, ic = 0;
        bool ok = true;
        for (; ok; ++ic) {
            int32_t bh;
            MassItem item;
            if (!take_warp(ic, item, bh)) break;
            const int b = bh / a.g.Hkv, hk = bh % a.g.Hkv;
            bool bad = false;
            ok = walk_blocks(a, item, G, qc, 1, 0, bad, [&](uint32_t q, int, int g, int r, int n) {
                const uint32_t sb = q % kBufs;
                const float* src = a.lse + ((int64_t)b * a.g.H + hk * G + g) * a.g.T + r;
                float x[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    // weight 0: rows past the block, rows without a sum
                    x[y] = -INFINITY;
                    if (32 * y + lane < n) {
                        x[y] = src[32 * y + lane];
                        x[y] = x[y] == -INFINITY ? x[y] : -x[y] * kLog2e;
                    }
                }
                if (!mbar_wait_warp(bar(L::B_LEMPTY + sb), ((q / kBufs) & 1) ^ 1, abort_flag, a.status, a.wait_ns)) return false;
                float* dst = reinterpret_cast<float*>(sm + L::LSE_OFF) + sb * 128;
#pragma unroll
                for (int y = 0; y < 4; ++y) dst[32 * y + lane] = x[y];
                // x is -inf past the block's rows too; those are told apart by their number
                bool none = false;
#pragma unroll
                for (int y = 0; y < 4; ++y) none |= 32 * y + lane < n && x[y] == -INFINITY;
                none = __any_sync(0xffffffffu, none);
                if (lane == 0) s_tag[sb] = tag_of(q, none);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::B_SFULL + sb));
                return true;
            });
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------ sums
        const int grp = (warp >> 2) - 1, key = tid & 127;
        const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
        const float c = a.g.scale * kLog2e;
        const float2 c2 = make_float2(c, c);
        float* s_part = reinterpret_cast<float*>(sm + L::PART_OFF);
        uint32_t qc = 0, ic = 0;
        bool ok = true;
        for (; ok; ++ic) {
            int32_t bh;
            MassItem item;
            if (!take_warp(ic, item, bh)) break;
            const int j = item.j0 + key;
            float sum = 0.f, err = 0.f;                      // compensated
            bool bad = false;
            ok = walk_blocks(a, item, G, qc, kGroups, turn_of(item, grp), bad, [&](uint32_t q, int ctx, int, int row0, int n) {
                const uint32_t sb = q % kBufs;
                const float* lse = reinterpret_cast<const float*>(sm + L::LSE_OFF) + sb * 128;
                // A parity tells neighbouring phases apart only, and a group that had no block for a while may
                // come before the phase ahead of its own has ended: the buffer's tag names the block
                // whose lse it holds, written once the block before it there has been summed.
                uint32_t tag = s_tag[sb];
                if (__any_sync(0xffffffffu, !same_block(tag, tag_of(q, false)))) {
                    if (!tag_wait(s_tag + sb, tag_of(q, false), abort_flag, a.status, a.wait_ns)) return false;
                    tag = s_tag[sb];                         // stays until this block has been summed
                }
                if (!mbar_wait_warp(bar(L::B_SFULL + sb), (q / kBufs) & 1, abort_flag, a.status, a.wait_ns)) return false;
                tc_fence_after();
                // this key is seen by the columns [lo, n)
                const int lo = ctx <= j ? max(0, j - row0) : kRows;
                const bool edge = n < kRows || row0 < item.j1 - 1 || ctx > item.j0 || (tag & 1u);
                const uint32_t sa = tmem + lane_addr + sb * kRows;
                float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
                for (int half = 0; half < kRows; half += 64) {
                    uint32_t r[2][32];
                    tmem_ld32(sa + half, r[0]);              // columns past n: what an earlier block left
                    tmem_ld32(sa + half + 32, r[1]);
                    tmem_ld_wait();
                    if (half) {
                        tc_fence_before();
                        mbar_arrive(bar(L::B_SEMPTY + sb));  // the buffer has been read
                    }
                    if (!edge) {
                        weigh64(r, lse + half, c2, acc);
                    } else if (half < n) {
                        const int from = lo - half, to = n - half;
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int y = 0; y < 32; ++y) {
                                const int col = 32 * x + y;
                                const float l = lse[half + col], e = fmaf(__uint_as_float(r[x][y]), c, l);
                                const float p = col >= from && col < to && l != -INFINITY ? ex2(e) : 0.f;
                                if (y & 1) acc[(y >> 1) & 1].y += p; else acc[(y >> 1) & 1].x += p;
                            }
                    }
                }
                mbar_arrive(bar(L::B_LEMPTY + sb));
                const float part = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
                const float y = __fsub_rn(part, err), t = __fadd_rn(sum, y);
                err = t == INFINITY ? 0.f : __fsub_rn(__fsub_rn(t, sum), y);   // an infinite weight stays one: no inf - inf
                sum = t;
                return true;
            });
            if (!ok) break;
            sum -= err;
            const uint32_t slot = ic & 1;
            ok = mbar_wait_warp(bar(L::B_PEMPTY + slot), ((ic >> 1) & 1) ^ 1, abort_flag, a.status, a.wait_ns);
            if (!ok) break;
            s_part[(slot * kGroups + grp) * 128 + key] = sum;
            mbar_arrive(bar(L::B_PFULL + slot));
        }
    } else {
        // ------------------------------------------------------------ results
        const int lane = tid & 31;
        const float* s_part = reinterpret_cast<const float*>(sm + L::PART_OFF);
        for (uint32_t ic = 0;; ++ic) {
            int32_t bh;
            MassItem item;
            if (!take_warp(ic, item, bh)) break;
            float base[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int j = item.j0 + 32 * y + lane;
                base[y] = a.mass_in && j < item.j1 ? a.mass_in[(int64_t)bh * a.g.T + j] : 0.f;
            }
            const uint32_t slot = ic & 1;
            if (!mbar_wait_warp(bar(L::B_PFULL + slot), (ic >> 1) & 1, abort_flag, a.status, a.wait_ns)) break;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int key = 32 * y + lane, j = item.j0 + key;
                float sum = 0.f;
                for (int x = 0; x < kGroups; ++x) sum += s_part[(slot * kGroups + x) * 128 + key];
                if (j < item.j1) a.mass_out[(int64_t)bh * a.g.T + j] = base[y] + sum;
            }
            mbar_arrive(bar(L::B_PEMPTY + slot));
        }
    }
    // ---------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        if (*abort_flag) {
            if (elect_one()) {
                mma_commit(bar(L::B_DRAIN));
                const uint64_t t0 = globaltimer();
                while (!mbar_try_wait(bar(L::B_DRAIN), 0) && globaltimer() - t0 < a.wait_ns) {
                }
            }
            __syncwarp();
        }
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------------ few rows over many keys
//
// The rows of one chunk, a window at the end of a long prompt, are few: with all heads
// of a group (row p of w G: head p / w, token q_begin + p mod w) they fill NB blocks of
// 128, which stay in shared memory while the keys stream past. A block of the grid takes
// an equal stretch of the (head, key tile) list; at the start of each head all threads
// lay its queries out as TMA would (128-byte swizzle), with -lse log2 e and the token of
// each row. A key tile is one group's: its rows' weights are summed by one thread in
// order. The keys' bytes are the floor: 32 KB at D = 128 are 1390 cycles of an SM's share
// of the memory rate, two blocks of products and exponentials 1024. Measured: 64 rows of 4
// heads over 128K keys of 8 key/value heads 86 us (3.1 TB/s, 2500 cycles a tile; 158 us with
// the general kernel, which brings the queries from L2 again for every tile), one row 51 us
// (5.2 TB/s). A trace shows the MMA thread busy all the time at 250 to 450 cycles a step
// (wait, eight products, commit) and the groups waiting for it a third of theirs; a second
// MMA thread for every other tile gained 2% and was not kept.
template <int DT>
struct WinLayout {
    static constexpr int TILE = 128 * DT * 2;
    static constexpr int MAX_NB = DT == 64 ? 8 : DT == 128 ? 4 : 1;
    static constexpr int MAX_KST = 6;
    static constexpr int B_KFULL = 0, B_KEMPTY = B_KFULL + MAX_KST;
    static constexpr int B_SFULL = B_KEMPTY + MAX_KST, B_SEMPTY = B_SFULL + kGroups * kBufs;
    static constexpr int B_DRAIN = B_SEMPTY + kBufs, NBAR = B_DRAIN + 1;
    static constexpr int BAR_BYTES = NBAR * 8 + 16;
    static int key_stages(int nb) { return std::min(MAX_KST, (212 * 1024 - nb * (TILE + 1024)) / TILE); }
    // the tiles; -lse, token and flags (4 bytes of 32 rows each) of the rows; barriers; alignment
    static size_t most() {
        size_t m = 0;
        for (int nb = 1; nb <= MAX_NB; ++nb) m = std::max(m, bytes(nb, key_stages(nb)));
        return m;
    }
    static size_t bytes(int nb, int kst) { return (size_t)(nb + kst) * TILE + nb * 1028 + BAR_BYTES + 1024 + 8; }
};

template <int DT>
__global__ void __launch_bounds__(kThreads, 1)
    key_mass_window_kernel(const __grid_constant__ CUtensorMap tmk, const MassArgs a, const TcMaps mpkv, const attn_chunk ch,
                           const int32_t nb, const int32_t kst) {
    using L = WinLayout<DT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(sm), k_off = nb * L::TILE;
    float* s_lse = reinterpret_cast<float*>(sm + (size_t)(nb + kst) * L::TILE);
    int32_t* s_tok = reinterpret_cast<int32_t*>(s_lse + nb * 128);
    // a byte for 32 rows, set where one of them weighs nothing
    uint8_t* s_none = reinterpret_cast<uint8_t*>(s_tok + nb * 128);
    uint8_t* s_bar = s_none + ((nb * 4 + 7) & ~7);
    const uint32_t bar0 = smem_u32(s_bar);
    auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    uint8_t* misc = s_bar + L::NBAR * 8;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 4);
    const int tid = threadIdx.x, warp = tid >> 5;
    const int G = a.g.H / a.g.Hkv, w = ch.q_end - ch.q_begin, R = w * G;
    const int tiles = (a.g.T + 127) / 128;

    if (tid == 0) {
        for (int s = 0; s < kst; ++s) {
            mbar_init(bar(L::B_KFULL + s), 1);
            mbar_init(bar(L::B_KEMPTY + s), 1);
        }
        for (int s = 0; s < kGroups * kBufs; ++s) mbar_init(bar(L::B_SFULL + s), 1);
        for (int s = 0; s < kBufs; ++s) mbar_init(bar(L::B_SEMPTY + s), 128);
        mbar_init(bar(L::B_DRAIN), 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const int64_t total = (int64_t)a.g.B * a.g.Hkv * tiles;
    const int64_t begin = blockIdx.x * total / gridDim.x, end = (blockIdx.x + 1) * total / gridDim.x;
    // whether any row sees a key of the tile, and whether all rows see all of its keys
    auto seen_tile = [&](int j0) { return j0 < ch.q_end && j0 + 128 > ch.ctx_begin; };
    uint32_t ks = 0, kp = 0;                                    // stage of the next key tile, and its parity
    uint32_t qc = 0, turn = 0, dealt = 0, mine = 0;             // blocks; the next tile's group; blocks of each group, of this one
    auto next_stage = [&]() {
        if (++ks == (uint32_t)kst) {
            ks = 0;
            kp ^= 1;
        }
    };
    auto next_turn = [&]() { turn = turn + 1 == kGroups ? 0 : turn + 1; };
    const TileDesc qd(sbase);
    bool ok = true;
    for (int64_t x0 = begin; x0 < end;) {
        const int bh = (int)(x0 / tiles), first = (int)(x0 - (int64_t)bh * tiles);
        const int count = (int)min((int64_t)(tiles - first), end - x0);
        const int b = bh / a.g.Hkv, hk = bh % a.g.Hkv;
        // ---------------------------------------------------------------- queries of the head
        for (int i = tid; i < nb * 128 * (DT / 8); i += kThreads) {
            const int p = i / (DT / 8), c16 = i % (DT / 8);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (p < R && c16 * 8 < a.g.D)
                v = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.q) + (int64_t)b * a.g.sb +
                                                    (int64_t)(hk * G + p / w) * a.g.sh +
                                                    (int64_t)(ch.q_begin + p % w) * a.g.st + c16 * 8);
            const int row = p & 127;
            *reinterpret_cast<uint4*>(sm + (p >> 7) * L::TILE + (c16 >> 3) * (128 * 128) + row * 128 +
                                      (((c16 & 7) ^ (row & 7)) << 4)) = v;
        }
        for (int p = tid; p < nb * 128; p += kThreads) {
            float l = -INFINITY;                        // weight 0: rows past the last, rows without a sum
            const int t = ch.q_begin + p % w;
            if (p < R) {
                l = a.lse[((int64_t)b * a.g.H + hk * G + p / w) * a.g.T + t];
                l = l == -INFINITY ? l : -l * kLog2e;
            }
            s_lse[p] = l;
            // 2^(s c - inf) is 0 only while the score s is not NaN or +inf, which the zero queries of a row
            // past the last make of a key that is not finite, and a row without a sum may be: no key is theirs
            s_tok[p] = l == -INFINITY ? -1 : t;
            const bool none = __any_sync(0xffffffffu, l == -INFINITY);
            if ((tid & 31) == 0) s_none[p >> 5] = none;
        }
        fence_proxy_async_smem();
        __syncthreads();
        if (warp == 0) {
            // ------------------------------------------------------------ producer
            if (elect_one() && !a.stall) {
                for (int i = 0; i < count && ok; ++i) {
                    const int j0 = (first + i) * 128;
                    if (!seen_tile(j0)) continue;
                    ok = mbar_wait(bar(L::B_KEMPTY + ks), kp ^ 1, abort_flag, a.status, a.wait_ns);
                    if (!ok) break;
                    mbar_expect_tx(bar(L::B_KFULL + ks), L::TILE);
                    load_rows<DT>(sbase + k_off + ks * L::TILE, &tmk, bar(L::B_KFULL + ks), mpkv, j0, 2, hk, b);
                    next_stage();
                }
            }
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA issuer
            if (elect_one()) {
                for (int i = 0; i < count && ok; ++i, next_turn()) {
                    if (!seen_tile((first + i) * 128)) continue;
                    const uint32_t grp = turn;
                    ok = mbar_wait(bar(L::B_KFULL + ks), kp, abort_flag, a.status, a.wait_ns);
                    const TileDesc kd(sbase + k_off + ks * L::TILE);
                    for (int x = 0; x < nb && ok; ++x, ++qc) {
                        const uint32_t sb = qc % kBufs;
                        ok = mbar_wait(bar(L::B_SEMPTY + sb), ((qc / kBufs) & 1) ^ 1, abort_flag, a.status, a.wait_ns);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t id = idesc_bf16(128, (min(128, R - 128 * x) + 15) & ~15, 0, 0);
#pragma unroll
                        for (int kk = 0; kk < DT / 16; ++kk) {
                            const uint32_t off = (kk >> 2) * (128 * 128) + (kk & 3) * 32;
                            mma_ss(tmem + sb * 128, kd.at(off), qd.at(off + x * L::TILE), id, kk > 0);
                        }
                        // a group's barriers in its own turn: at most kBufs of its blocks are ahead of it
                        const uint32_t m = dealt >> (8 * grp) & 3u;
                        dealt = (dealt & ~(3u << (8 * grp))) | ((m + 1) & 3u) << (8 * grp);
                        mma_commit(bar(L::B_SFULL + grp * kBufs + m));
                    }
                    if (!ok) break;
                    mma_commit(bar(L::B_KEMPTY + ks));
                    next_stage();
                }
            }
        } else if (warp >= 4) {
            // ------------------------------------------------------------ sums
            const int grp = (warp >> 2) - 1, key = tid & 127;
            const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
            const float c = a.g.scale * kLog2e;
            const float2 c2 = make_float2(c, c);
            uint32_t without = 0;                       // a bit for 64 rows of the head, set where one weighs nothing
            for (int y = 0; y < 2 * nb; ++y)
                without |= (reinterpret_cast<const uint16_t*>(s_none)[y] ? 1u : 0u) << y;
            for (int i = 0; i < count && ok; ++i, next_turn()) {
                const int j0 = (first + i) * 128, j = j0 + key;
                const bool sees = seen_tile(j0);
                if (turn != (uint32_t)grp) {
                    if (sees) qc += nb;
                    continue;
                }
                const int64_t at = (int64_t)bh * a.g.T + j;
                const float base = a.mass_in && j < a.g.T ? a.mass_in[at] : 0.f;
                const bool edge = j0 + 127 > ch.q_begin || j0 < ch.ctx_begin;
                float sum = 0.f;
                for (int x = 0; x < nb && ok && sees; ++x, ++qc, ++mine) {
                    ok = mbar_wait_warp(bar(L::B_SFULL + grp * kBufs + mine % kBufs), (mine / kBufs) & 1, abort_flag, a.status,
                                        a.wait_ns);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t sb = qc % kBufs, sa = tmem + lane_addr + sb * 128;
                    const int cols = (min(128, R - 128 * x) + 15) & ~15;
                    float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
                    for (int half = 0; half < cols; half += 64) {
                        const float* lse = s_lse + 128 * x + half;
                        const int left = cols - half;                    // columns of this half
                        uint32_t r[2][32];
                        if (left >= 64) {
                            tmem_ld32(sa + half, r[0]);
                            tmem_ld32(sa + half + 32, r[1]);
                        } else {
                            // in sixteens: the columns past `cols` were never written
                            uint32_t(&q16)[4][16] = reinterpret_cast<uint32_t(&)[4][16]>(r);
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                if (16 * y < left) tmem_ld16(sa + half + 16 * y, q16[y]);
                        }
                        tmem_ld_wait();
                        if (left <= 64) {
                            tc_fence_before();
                            mbar_arrive(bar(L::B_SEMPTY + sb));          // the buffer has been read
                        }
                        const bool pick = edge || (without >> (2 * x + half / 64) & 1u);
                        if (left >= 64 && !pick) {
                            weigh64(r, lse, c2, acc);
                        } else {
                            const int32_t* tok = s_tok + 128 * x + half;
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                if (16 * y >= left) break;
#pragma unroll
                                for (int z = 0; z < 16; ++z) {
                                    const float e = fmaf(__uint_as_float(r[y >> 1][16 * (y & 1) + z]), c, lse[16 * y + z]);
                                    const bool on = !pick || (j >= ch.ctx_begin && j <= tok[16 * y + z]);
                                    const float p = on ? ex2(e) : 0.f;
                                    if (z & 1) acc[(z >> 1) & 1].y += p; else acc[(z >> 1) & 1].x += p;
                                }
                            }
                        }
                    }
                    sum += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
                }
                if (ok && j < a.g.T) a.mass_out[at] = base + sum;
            }
        }
        __syncwarp();
        tc_fence_before();
        __syncthreads();                                // the head's queries have been read
        tc_fence_after();
        x0 += count;
    }
    // ---------------------------------------------------------------- teardown
    if (warp == 1) {
        __syncwarp();
        if (*abort_flag) {
            if (elect_one()) {
                mma_commit(bar(L::B_DRAIN));
                const uint64_t t0 = globaltimer();
                while (!mbar_try_wait(bar(L::B_DRAIN), 0) && globaltimer() - t0 < a.wait_ns) {
                }
            }
            __syncwarp();
        }
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Whether the window kernel takes these rows: one chunk whose rows of a group fit. It lays
// them out first, 7 us for each 128 (above 128 dims 11), and then takes nb blocks a key
// tile, where the general kernel takes a block of each head, 0.72 us each; a tile costs the
// general kernel no less than 1.8 us and this one 0.95. So the tiles of an SM decide. Both
// measured, general / window, us, at w rows, G heads a group, key/value heads x keys:
//   128 dims, w 1,   G 4:  8 x 1K 12 / 9,  8 x 16K 27 / 13,  8 x 128K 157 / 52
//             w 64,  G 4:  8 x 1K 12 / 25, 8 x 16K 27 / 31,  8 x 32K 45 / 38,  8 x 128K 158 / 86
//             w 128, G 4:  8 x 1K 14 / 39, 8 x 16K 29 / 54,  8 x 128K 162 / 181
//             w 128, G 1:  8 x 4K 10 / 17, 8 x 16K 20 / 21,  8 x 32K 31 / 25,  32 x 64K 192 / 101
//             w 64,  G 8:  4 x 8K 16 / 41, 4 x 64K 72 / 72,  4 x 128K 134 / 113
//   64 dims,  w 256, G 4:  8 x 1K 17 / 64, 8 x 128K 238 / 376
//   256 dims, w 32,  G 4:  8 x 8K 20 / 21, 8 x 16K 31 / 25;  w 128, G 1: 32 x 8K 40 / 47, 32 x 16K 69 / 64
template <int DT>
bool window(const MassArgs& a, const attn_chunk* chunks) {
    if (a.n != 1) return false;
    const int64_t w = chunks[0].q_end - chunks[0].q_begin, G = a.g.H / a.g.Hkv, rows = w * G, nb = (rows + 127) / 128;
    if (nb > WinLayout<DT>::MAX_NB) return false;
    const int64_t tiles = (int64_t)a.g.B * a.g.Hkv * ((a.g.T + 127) / 128), sms = device_sm_count(), n = (tiles + sms - 1) / sms;
    const int64_t blocks = G * ((w + 127) / 128);
    // in tenths of a block: what is saved a tile, against the rows' layout and two blocks
    return n * (std::max<int64_t>(10 * blocks, 25) - std::max<int64_t>(10 * nb, 13)) > (DT > 128 ? 150 : 100) * rows / 128 + 20;
}

template <int DT>
cudaError_t launch_window(const MassArgs& a, const attn_chunk& ch, cudaStream_t s) {
    using L = WinLayout<DT>;
    CUtensorMap mk;
    TcMaps mpkv{1, 2, 3};
    if (!make_tile_map(&mk, a.k, a.g.kv(), mpkv, kBoxRows)) return cudaErrorInvalidValue;
    const int nb = ((ch.q_end - ch.q_begin) * (a.g.H / a.g.Hkv) + 127) / 128, kst = L::key_stages(nb);
    const size_t smem = L::bytes(nb, kst);
    // always the most that any call takes: the limit is the function's, and a call of another thread may be
    // between its own limit and its launch
    cudaError_t e = cudaFuncSetAttribute(key_mass_window_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)L::most());
    if (e != cudaSuccess) return e;
    const int64_t total = (int64_t)a.g.B * a.g.Hkv * ((a.g.T + 127) / 128);
    const int grid = (int)std::min<int64_t>(total, device_sm_count());
    key_mass_window_kernel<DT><<<grid, kThreads, smem, s>>>(mk, a, mpkv, ch, nb, kst);
    return counted(cudaGetLastError());
}

template <int DT>
cudaError_t launch_d(const MassArgs& a, cudaStream_t s) {
    CUtensorMap mq, mk;
    TcMaps mp{1, 2, 3}, mpkv{1, 2, 3};
    const Geom gkv = a.g.kv();
    if (!make_tile_map(&mq, a.q, a.g, mp, kBoxRows) || !make_tile_map(&mk, a.k, gkv, mpkv, kBoxRows))
        return cudaErrorInvalidValue;
    const int64_t work = (int64_t)a.n_items * a.g.B * a.g.Hkv;
    if (work > INT32_MAX) return cudaErrorInvalidValue;
    const size_t smem = Layout<DT>::ALLOC;
    static_assert(Layout<DT>::ALLOC <= 232448, "shared memory of the key mass kernel");
    cudaError_t e = cudaFuncSetAttribute(key_mass_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int grid = (int)std::min<int64_t>(work, device_sm_count());
    key_mass_kernel<DT><<<grid, kThreads, smem, s>>>(mq, mk, a, mp, mpkv, (int32_t)work);
    return counted(cudaGetLastError());
}

}  // namespace

bool key_mass_window(const MassArgs& a, const attn_chunk* chunks) {
    return a.g.D > 128 ? window<256>(a, chunks) : a.g.D > 64 ? window<128>(a, chunks) : window<64>(a, chunks);
}

cudaError_t launch_key_mass_window(const MassArgs& a, const attn_chunk& ch, cudaStream_t s) {
    return a.g.D > 128 ? launch_window<256>(a, ch, s) : a.g.D > 64 ? launch_window<128>(a, ch, s) : launch_window<64>(a, ch, s);
}

cudaError_t launch_key_mass(const MassArgs& a, cudaStream_t s) {
    return a.g.D > 128 ? launch_d<256>(a, s) : a.g.D > 64 ? launch_d<128>(a, s) : launch_d<64>(a, s);
}

}  // namespace attn
